// The weight gradient's kernel, as shipped, launched by a test with other
// arguments than the entry point's: its longest wait, one pair of CTAs for all
// tiles, and copies that bring less than the kernel waits for (boxes of half as
// many tokens), so that its waits run out.
#include "zero_wgrad.cu"

namespace zero {
// Defined in a translation unit that this one does without.
bool pdl_launches() { return false; }
zero_status_t require_device(const void* const*, int) { return ZERO_OK; }
}  // namespace zero

// short_dy, short_q: that operand's copies bring half their bytes.
// one_pair: tiles are not cut, and one pair of CTAs takes them all.
extern "C" int wgrad_waits(const zero_mat_t* dy, const zero_act8_t* x, uint32_t accumulate, const zero_mat_t* dw,
                           void* workspace, uint64_t workspace_bytes, uint64_t wait_ns, uint32_t short_dy,
                           uint32_t short_q, uint32_t one_pair)
{
    Plan plan;
    if (!make_plan(dy->rows, dy->cols, x->cols, &plan))
        return ZERO_ERR_UNSUPPORTED;
    if (one_pair) {
        plan.splits = 1;
        plan.full = plan.units = plan.tiles_i * plan.tiles_o;
    }
    if (plan_workspace(plan) > workspace_bytes)
        return ZERO_ERR_INVALID_ARG;
    WgradArgs a = make_args(x, nullptr, accumulate, dw, workspace, plan);
    a.wait_ns = wait_ns;
    const EncodeTiled encode = encode_tiled();
    CUtensorMap ymap, qmap;
    if (!encode || !encode_operands(encode, &ymap, &qmap, dy, x, short_dy ? kStepT / 2 : kStepT,
                                    short_q ? kStepT / 2 : kStepT))
        return ZERO_ERR_CUDA;
    const uint32_t pairs = one_pair ? 1 : kPairs;
    return train_status(dy->dtype == ZERO_F16 ? launch_products<ZERO_F16>(ymap, qmap, a, nullptr, pairs)
                                              : launch_products<ZERO_BF16>(ymap, qmap, a, nullptr, pairs));
}
