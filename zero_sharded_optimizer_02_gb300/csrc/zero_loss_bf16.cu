// The losses' row kernels for bfloat16 logits.
#include "zero_loss.cuh"

cudaError_t zero::launch_loss_bf16(const LossArgs& a, LossOp op, bool grad, bool top, int dual, void* stream)
{
    return launch_loss<ZERO_BF16>(a, op, grad, top, dual, stream);
}
