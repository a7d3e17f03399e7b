// Weight gradient of a linear layer from an 8-bit checkpoint of its input
// (sm_103a):  dw[o][i] = gain[i] * sum over t of dy[t][o] * xhat[t][i].
#include "zero_train_device.cuh"

namespace zero {
namespace {

constexpr int kTileO = 64, kTileI = 64, kTileT = 16;
constexpr int kThreads = 256;

struct WgradArgs {
    const uint16_t* dy;
    const int8_t* q;
    const uint8_t* scale;
    const uint16_t* gain;
    uint16_t* dw;
    uint64_t dy_pitch, q_pitch, scale_pitch, dw_pitch;
    uint64_t tokens, outs, ins;
    uint32_t add;
};

// One CTA sums a 64 x 64 tile of dw over all tokens in fp32, 4 x 4 a thread.
template <int DT>
__global__ void __launch_bounds__(kThreads) k_weight_grad(const WgradArgs a)
{
    __shared__ float sy[kTileT][kTileO];
    __shared__ float sx[kTileT][kTileI];
    pdl_entry();
    const uint64_t o0 = (uint64_t)blockIdx.y * kTileO, i0 = (uint64_t)blockIdx.x * kTileI;
    const int to = threadIdx.x / 16, ti = threadIdx.x % 16;
    float acc[4][4] = {};
    for (uint64_t t0 = 0; t0 < a.tokens; t0 += kTileT) {
        for (int k = threadIdx.x; k < kTileT * kTileO; k += kThreads) {
            const uint64_t t = t0 + k / kTileO, o = o0 + k % kTileO;
            sy[k / kTileO][k % kTileO] =
                t < a.tokens && o < a.outs ? widen1<DT>(a.dy[t * a.dy_pitch + o]) : 0.0f;
        }
        for (int k = threadIdx.x; k < kTileT * kTileI; k += kThreads) {
            const uint64_t t = t0 + k / kTileI, i = i0 + k % kTileI;
            float x = 0.0f;
            if (t < a.tokens && i < a.ins)
                x = (float)a.q[t * a.q_pitch + i] *
                    act8_step(a.scale[t * a.scale_pitch + i / ZERO_ACT8_BLOCK]);
            sx[k / kTileI][k % kTileI] = widen1<DT>(narrow1<DT>(x));
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTileT; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[r][c] += sy[k][to * 4 + r] * sx[k][ti * 4 + c];
        __syncthreads();
    }
    for (int r = 0; r < 4; ++r)
        for (int c = 0; c < 4; ++c) {
            const uint64_t o = o0 + to * 4 + r, i = i0 + ti * 4 + c;
            if (o < a.outs && i < a.ins) {
                float x = a.gain ? acc[r][c] * widen1<DT>(a.gain[i]) : acc[r][c];
                uint16_t* w = a.dw + o * a.dw_pitch + i;
                *w = narrow1<DT>(a.add ? widen1<DT>(*w) + x : x);
            }
        }
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" uint64_t zero_act_weight_grad_workspace(uint64_t tokens, uint64_t outs, uint64_t ins)
{
    (void)tokens;
    (void)outs;
    (void)ins;
    return 0;
}

extern "C" zero_status_t zero_act_weight_grad(const zero_mat_t* dy, const zero_act8_t* x,
                                              const void* gain, uint32_t accumulate,
                                              const zero_mat_t* dw, void* workspace,
                                              uint64_t workspace_bytes, void* stream)
{
    zero_status_t st = check_mat(dy, true);
    if (st == ZERO_OK)
        st = check_act8(x);
    if (st == ZERO_OK)
        st = check_mat(dw, false);
    if (st != ZERO_OK)
        return st;
    if (dy->rows != x->rows || dw->rows != dy->cols || dw->cols != x->cols ||
        dw->dtype != dy->dtype || accumulate > 1)
        return ZERO_ERR_INVALID_ARG;
    if ((uintptr_t)gain % 2 != 0)
        return ZERO_ERR_ALIGNMENT;
    if (dw->rows == 0 || dw->cols == 0 || (dy->rows == 0 && accumulate))
        return ZERO_OK;
    const uint64_t need = zero_act_weight_grad_workspace(dy->rows, dy->cols, x->cols);
    if (need && (!workspace || workspace_bytes < need))
        return ZERO_ERR_INVALID_ARG;
    if (need && (uintptr_t)workspace % 16 != 0)
        return ZERO_ERR_ALIGNMENT;
    const Span outs[2] = {span_of(dw), span_of(workspace, need)};
    const Span ins[4] = {span_of(dy), span_of_q(x), span_of_scale(x), span_of(gain, 2 * x->cols)};
    if (any_overlap(outs, 2, ins, 4))
        return ZERO_ERR_INVALID_ARG;
    const void* p[6];
    int n = 0;
    const bool some = dy->rows > 0;
    const void* all[6] = {some ? dy->base : nullptr, some ? x->q : nullptr,
                          some ? x->scale : nullptr, gain, dw->base, need ? workspace : nullptr};
    for (const void* q : all)
        if (q)
            p[n++] = q;
    st = require_device(p, n);
    if (st != ZERO_OK)
        return st;
    if ((dw->rows + kTileO - 1) / kTileO > 65535 || (dw->cols + kTileI - 1) / kTileI > 0x7FFFFFFFull)
        return ZERO_ERR_UNSUPPORTED;

    WgradArgs a = {};
    a.dy = static_cast<const uint16_t*>(dy->base);
    a.q = x->q;
    a.scale = x->scale;
    a.gain = static_cast<const uint16_t*>(gain);
    a.dw = static_cast<uint16_t*>(dw->base);
    a.dy_pitch = dy->pitch;
    a.q_pitch = x->q_pitch;
    a.scale_pitch = x->scale_pitch;
    a.dw_pitch = dw->pitch;
    a.tokens = dy->rows;
    a.outs = dw->rows;
    a.ins = dw->cols;
    a.add = accumulate;
    const dim3 grid((unsigned)((a.ins + kTileI - 1) / kTileI), (unsigned)((a.outs + kTileO - 1) / kTileO));
    return train_status(launch_train(dy->dtype == ZERO_F16 ? k_weight_grad<ZERO_F16> : k_weight_grad<ZERO_BF16>,
                                     grid, kThreads, 0, 1, stream, a));
}
