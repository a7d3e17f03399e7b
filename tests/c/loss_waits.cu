// The losses' kernel for rows that two CTAs share, as shipped, launched by a test that
// has it wait for more sums than the CTAs send, so that its waits run out.
#include "zero_loss.cu"

namespace zero {
// Defined in translation units that this one does without.
bool pdl_launches() { return false; }
zero_status_t require_device(const void* const*, int) { return ZERO_OK; }
cudaError_t launch_loss_f16(const LossArgs&, LossOp, bool, bool, int, void*) { return cudaErrorNotSupported; }
cudaError_t launch_loss_bf16(const LossArgs&, LossOp, bool, bool, int, void*) { return cudaErrorNotSupported; }
}  // namespace zero

// The cross-entropy of bfloat16 rows with its gradient; missing: bytes that the kernel
// waits for and nothing sends.
extern "C" int loss_waits(const zero_mat_t* logits, const zero_ids_t* targets, float* loss, const zero_mat_t* d_logits,
                          uint64_t wait_ns, uint32_t missing)
{
    constexpr int NT = 256;
    LossArgs a;
    const zero_status_t st = check_rows(logits, targets, d_logits, 1.0f, 1.0f, a);
    if (st != ZERO_OK)
        return st;
    a.loss = loss;
    a.hard = 1.0f;
    const auto kernel = k_loss_rows<ZERO_BF16, kDistill, true, false, 0, NT>;
    RowShape sh = shape_of<false, 0, NT>(a, 2);
    const size_t smem = smem_of<NT>(sh);
    sh.sent += missing;
    sh.wait_ns = wait_ns;
    static std::atomic<uint64_t> allowed{0};
    allow_smem(kernel, kMostSmem, allowed);
    return train_status(launch_train(kernel, dim3(2 * (a.rows < 8 ? a.rows : 8)), NT, smem, 2, nullptr, a, sh));
}
