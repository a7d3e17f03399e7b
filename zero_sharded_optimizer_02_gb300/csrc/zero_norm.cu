// Residual addition with the root-mean-square norm, its backward pass from an
// 8-bit checkpoint, and the checkpoint's own pack and unpack (sm_103a).
//
// All four are bound by memory: the floor is each operand once.
#include "zero_train_device.cuh"

namespace zero {
namespace {

// -- norm ---------------------------------------------------------------------------

// A row is held in registers by a group of G threads (whole warps), V vectors
// of 8 elements a thread: vector j of thread i covers columns (j*G + i)*8, so
// four neighbouring lanes hold one block of the checkpoint.
struct NormShape {
    uint32_t group;   // G
    uint32_t vecs;    // V: 1, 2 or 4
    uint32_t rows;    // rows per CTA
    uint32_t threads() const { return group * rows; }
};

constexpr uint32_t kNormMinThreads = 128;

// The least V whose group fits 256 threads, else 4.
NormShape norm_shape(uint64_t cols)
{
    const uint32_t nv = (uint32_t)((cols + 7) / 8);
    uint32_t v = 1;
    while (v < 4 && (nv + v - 1) / v > 256)
        v *= 2;
    const uint32_t g = ((nv + v - 1) / v + 31) / 32 * 32;
    return NormShape{g, v, g >= kNormMinThreads ? 1 : kNormMinThreads / g};
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int d = 16; d; d >>= 1)
        x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    return x;
}

// Sum of x over the calling thread's group; the same bits in every thread.
// sums: 32 floats of shared memory that no thread still reads.
__device__ __forceinline__ float group_sum(float x, uint32_t group, float* sums)
{
    x = warp_sum(x);
    if (group > 32) {
        const uint32_t warp = threadIdx.x / 32, per = group / 32;
        if (threadIdx.x % 32 == 0)
            sums[warp] = x;
        __syncthreads();
        const uint32_t w0 = warp / per * per;
        x = 0.0f;
        for (uint32_t w = 0; w < per; ++w)
            x += sums[w0 + w];
    }
    return x;
}

struct NormFwdArgs {
    const uint16_t* x;
    const uint16_t* res;
    const uint16_t* gain;
    uint16_t* h;
    uint16_t* y;
    float* rstd;
    int8_t* q;
    uint8_t* scale;
    uint64_t x_pitch, res_pitch, h_pitch, y_pitch, q_pitch, scale_pitch;
    uint64_t rows, cols;
    uint32_t group, rows_per_cta;
    uint32_t gain_vec;   // the gain lies on a 16-byte boundary
    float eps;
};

template <int DT>
__device__ __forceinline__ void load_gain(const uint16_t* gain, bool vec, uint64_t c,
                                          uint64_t cols, float (&g)[8])
{
    if (!gain) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            g[i] = 1.0f;
        return;
    }
    set8<DT>(g, vec ? load8<true>(gain, c, cols) : load8<false>(gain, c, cols));
}

template <int DT, int V>
__global__ void __launch_bounds__(1024) k_norm_forward(const NormFwdArgs a)
{
    __shared__ float sums[32];
    pdl_entry();
    const uint32_t lane = threadIdx.x % a.group;
    const uint64_t row = (uint64_t)blockIdx.x * a.rows_per_cta + threadIdx.x / a.group;
    const bool live = row < a.rows;
    float s[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        set8<DT>(s[j], live ? load8<true>(a.x + row * a.x_pitch, c, a.cols) : make_uint4(0, 0, 0, 0));
        if (a.res && live)
            add8<DT>(s[j], load8<true>(a.res + row * a.res_pitch, c, a.cols));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss += s[j][i] * s[j][i];
    }
    ss = group_sum(ss, a.group, sums);
    const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.cols) + a.eps);
    if (live && lane == 0 && a.rstd)
        a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        if (a.h && live && c < a.cols)
            store8_row<true>(a.h + row * a.h_pitch, c, a.cols, narrow8<DT>(s[j]));
        float xhat[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            xhat[i] = s[j][i] * rstd;
        if (a.y && live && c < a.cols) {
            float g[8], y[8];
            load_gain<DT>(a.gain, a.gain_vec, c, a.cols, g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = xhat[i] * g[i];
            store8_row<true>(a.y + row * a.y_pitch, c, a.cols, narrow8<DT>(y));
        }
        if (a.q) {
            if (c >= a.cols) {   // past the row's end: not part of its last block
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    xhat[i] = 0.0f;
            } else if (c + 8 > a.cols) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i >= a.cols)
                        xhat[i] = 0.0f;
            }
            uint32_t sc;
            const uint2 q = act8_pack8<DT>(xhat, sc);
            if (live && c < a.cols) {
                store8_q(a.q + row * a.q_pitch, c, a.cols, q);
                if (c % ZERO_ACT8_BLOCK == 0)
                    a.scale[row * a.scale_pitch + c / ZERO_ACT8_BLOCK] = (uint8_t)sc;
            }
        }
    }
}

// Most CTAs of the backward kernel, each of which leaves one partial row of
// the gain's gradient: 8 CTAs of 128 threads on each of 152 SMs.
constexpr uint32_t kNormMaxParts = 1216;

struct NormBwdArgs {
    const uint16_t* dy;
    const int8_t* q;
    const uint8_t* scale;
    const float* rstd;
    const uint16_t* gain;
    const uint16_t* dres;
    uint16_t* dx;
    float* parts;        // [gridDim.x][part_pitch], or null: no gain gradient
    uint64_t dy_pitch, q_pitch, scale_pitch, dres_pitch, dx_pitch, part_pitch;
    uint64_t rows, cols;
    uint32_t group, rows_per_cta;
    uint32_t gain_vec;
};

template <int DT, int V>
__global__ void __launch_bounds__(1024) k_norm_backward(const NormBwdArgs a)
{
    __shared__ float sums[2][32];
    __shared__ float fold[kNormMinThreads * 4 * 8];   // only CTAs of several groups
    pdl_entry();
    const uint32_t lane = threadIdx.x % a.group, mine = threadIdx.x / a.group;
    float dg[V][8], g[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        load_gain<DT>(a.gain, a.gain_vec, ((uint64_t)j * a.group + lane) * 8, a.cols, g[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dg[j][i] = 0.0f;
    }
    int flip = 0;
    for (uint64_t r0 = (uint64_t)blockIdx.x * a.rows_per_cta; r0 < a.rows;
         r0 += (uint64_t)gridDim.x * a.rows_per_cta) {
        const uint64_t row = r0 + mine;
        const bool live = row < a.rows;
        float u[V][8], xhat[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
            const bool in = live && c < a.cols;
            set8<DT>(u[j], in ? load8<true>(a.dy + row * a.dy_pitch, c, a.cols)
                              : make_uint4(0, 0, 0, 0));
            const uint2 q = in ? load8_q(a.q + row * a.q_pitch, c, a.cols) : make_uint2(0, 0);
            const float step =
                in ? act8_step(a.scale[row * a.scale_pitch + c / ZERO_ACT8_BLOCK]) : 0.0f;
            act8_unpack8(q, step, xhat[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (c + i >= a.cols)
                    xhat[j][i] = 0.0f;   // the step may be NaN there
                dg[j][i] += u[j][i] * xhat[j][i];
                u[j][i] *= g[j][i];
                dot += u[j][i] * xhat[j][i];
            }
        }
        dot = group_sum(dot, a.group, sums[flip]);
        flip ^= 1;
        if (live) {
            const float mean = __fdiv_rn(dot, (float)a.cols), rstd = a.rstd[row];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
                if (c >= a.cols)
                    continue;
                float r[8];
                set8<DT>(r, a.dres ? load8<true>(a.dres + row * a.dres_pitch, c, a.cols)
                                   : make_uint4(0, 0, 0, 0));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] += rstd * (u[j][i] - xhat[j][i] * mean);
                store8_row<true>(a.dx + row * a.dx_pitch, c, a.cols, narrow8<DT>(r));
            }
        }
    }
    if (!a.parts)
        return;
    if (a.rows_per_cta > 1) {   // fold the groups' sums in group order
        const uint32_t width = a.group * V * 8;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                fold[mine * width + ((uint32_t)j * a.group + lane) * 8 + i] = dg[j][i];
        __syncthreads();
        if (mine != 0)
            return;
        for (uint32_t m = 1; m < a.rows_per_cta; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dg[j][i] += fold[m * width + ((uint32_t)j * a.group + lane) * 8 + i];
    }
    float* part = a.parts + blockIdx.x * a.part_pitch;   // part_pitch: cols rounded up to 8
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        if (c < a.cols) {
            reinterpret_cast<float4*>(part + c)[0] = make_float4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]);
            reinterpret_cast<float4*>(part + c)[1] = make_float4(dg[j][4], dg[j][5], dg[j][6], dg[j][7]);
        }
    }
}

// d_gain[c] = rnd((add ? d_gain[c] : 0) + sum of the parts, in a fixed order).
constexpr int kFoldSlices = 8;
template <int DT>
__global__ void __launch_bounds__(32 * kFoldSlices)
    k_norm_gain(const float* parts, uint32_t nparts, uint64_t part_pitch, uint64_t cols,
                uint32_t add, uint16_t* dgain)
{
    __shared__ float s[kFoldSlices][32];
    pdl_entry();
    const uint64_t c = (uint64_t)blockIdx.x * 32 + threadIdx.x % 32;
    const uint32_t slice = threadIdx.x / 32;
    float acc = 0.0f;
    if (c < cols)
#pragma unroll 8
        for (uint32_t p = slice; p < nparts; p += kFoldSlices)
            acc += parts[p * part_pitch + c];
    s[slice][threadIdx.x % 32] = acc;
    __syncthreads();
    if (slice == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < kFoldSlices; ++i)
            acc += s[i][threadIdx.x];
        dgain[c] = narrow1<DT>(add ? widen1<DT>(dgain[c]) + acc : acc);
    }
}

template <int DT>
cudaError_t launch_forward(const NormFwdArgs& a, const NormShape& sh, void* stream)
{
    const dim3 grid((unsigned)((a.rows + sh.rows - 1) / sh.rows));
    switch (sh.vecs) {
    case 1: return launch_train(k_norm_forward<DT, 1>, grid, sh.threads(), 0, 1, stream, a);
    case 2: return launch_train(k_norm_forward<DT, 2>, grid, sh.threads(), 0, 1, stream, a);
    default: return launch_train(k_norm_forward<DT, 4>, grid, sh.threads(), 0, 1, stream, a);
    }
}

template <int DT>
cudaError_t launch_backward(const NormBwdArgs& a, const NormShape& sh, uint32_t grid,
                            void* stream)
{
    switch (sh.vecs) {
    case 1: return launch_train(k_norm_backward<DT, 1>, dim3(grid), sh.threads(), 0, 1, stream, a);
    case 2: return launch_train(k_norm_backward<DT, 2>, dim3(grid), sh.threads(), 0, 1, stream, a);
    default: return launch_train(k_norm_backward<DT, 4>, dim3(grid), sh.threads(), 0, 1, stream, a);
    }
}

uint64_t backward_parts(uint64_t rows, const NormShape& sh)
{
    const uint64_t ctas = (rows + sh.rows - 1) / sh.rows;
    return ctas < kNormMaxParts ? ctas : kNormMaxParts;
}

// -- pack and unpack -------------------------------------------------------------------

constexpr int kPackThreads = 256;
constexpr int kPackUnroll = 4;

struct PackArgs {
    uint16_t* x;
    int8_t* q;
    uint8_t* scale;
    uint64_t x_pitch, q_pitch, scale_pitch;
    uint64_t cols;
    uint32_t slots;   // 8-element slots a row: 4 per block, so a block is 4 neighbouring lanes
    uint32_t items;   // slots * rows of this launch
};

template <int DT>
__global__ void __launch_bounds__(kPackThreads) k_act_pack(const PackArgs a)
{
    pdl_entry();
    const uint32_t i0 = blockIdx.x * (kPackThreads * kPackUnroll) + threadIdx.x;
    uint4 w[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        const uint32_t i = i0 + u * kPackThreads;
        w[u] = make_uint4(0, 0, 0, 0);
        if (i < a.items) {
            const uint32_t row = i / a.slots;
            const uint64_t c = (uint64_t)(i - row * a.slots) * 8;
            if (c < a.cols)
                w[u] = load8<true>(a.x + row * a.x_pitch, c, a.cols);
        }
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        const uint32_t i = i0 + u * kPackThreads;
        float x[8];
        set8<DT>(x, w[u]);
        uint32_t sc;
        const uint2 q = act8_pack8<DT>(x, sc);
        if (i < a.items) {
            const uint32_t row = i / a.slots;
            const uint64_t c = (uint64_t)(i - row * a.slots) * 8;
            if (c < a.cols) {
                store8_q(a.q + row * a.q_pitch, c, a.cols, q);
                if (c % ZERO_ACT8_BLOCK == 0)
                    a.scale[row * a.scale_pitch + c / ZERO_ACT8_BLOCK] = (uint8_t)sc;
            }
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kPackThreads) k_act_unpack(const PackArgs a)
{
    pdl_entry();
    const uint32_t i0 = blockIdx.x * (kPackThreads * kPackUnroll) + threadIdx.x;
    uint2 q[kPackUnroll];
    uint32_t sc[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        const uint32_t i = i0 + u * kPackThreads;
        q[u] = make_uint2(0, 0);
        sc[u] = 0;
        if (i < a.items) {
            const uint32_t row = i / a.slots;
            const uint64_t c = (uint64_t)(i - row * a.slots) * 8;
            if (c < a.cols) {
                q[u] = load8_q(a.q + row * a.q_pitch, c, a.cols);
                sc[u] = a.scale[row * a.scale_pitch + c / ZERO_ACT8_BLOCK];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        const uint32_t i = i0 + u * kPackThreads;
        if (i < a.items) {
            const uint32_t row = i / a.slots;
            const uint64_t c = (uint64_t)(i - row * a.slots) * 8;
            if (c < a.cols) {
                float x[8];
                act8_unpack8(q[u], act8_step(sc[u]), x);
                store8_row<true>(a.x + row * a.x_pitch, c, a.cols, narrow8<DT>(x));
            }
        }
    }
}

// Pack and unpack run in launches of at most 2^30 slots, so that item numbers
// stay in 32 bits.
zero_status_t launch_pack(const zero_mat_t* x, const zero_act8_t* c, bool pack, void* stream)
{
    if (x->rows == 0 || x->cols == 0)
        return ZERO_OK;
    const uint64_t slots = (x->cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK * 4;
    if (slots > (1ull << 30))
        return ZERO_ERR_UNSUPPORTED;
    const uint64_t step = (1ull << 30) / slots;
    cudaError_t e = cudaSuccess;
    for (uint64_t r = 0; r < x->rows && e == cudaSuccess; r += step) {
        const uint64_t rows = x->rows - r < step ? x->rows - r : step;
        PackArgs a;
        a.x = static_cast<uint16_t*>(x->base) + r * x->pitch;
        a.q = c->q + r * c->q_pitch;
        a.scale = c->scale + r * c->scale_pitch;
        a.x_pitch = x->pitch;
        a.q_pitch = c->q_pitch;
        a.scale_pitch = c->scale_pitch;
        a.cols = x->cols;
        a.slots = (uint32_t)slots;
        a.items = (uint32_t)(slots * rows);
        const dim3 grid((a.items + kPackThreads * kPackUnroll - 1) / (kPackThreads * kPackUnroll));
        const bool f16 = x->dtype == ZERO_F16;
        if (pack)
            e = launch_train(f16 ? k_act_pack<ZERO_F16> : k_act_pack<ZERO_BF16>, grid,
                             kPackThreads, 0, 1, stream, a);
        else
            e = launch_train(f16 ? k_act_unpack<ZERO_F16> : k_act_unpack<ZERO_BF16>, grid,
                             kPackThreads, 0, 1, stream, a);
    }
    return train_status(e);
}

// Argument checks that pack and unpack share.
zero_status_t check_pack(const zero_mat_t* x, const zero_act8_t* c, bool pack)
{
    zero_status_t st = check_mat(x, true);
    if (st == ZERO_OK)
        st = check_act8(c);
    if (st != ZERO_OK)
        return st;
    if (x->rows != c->rows || x->cols != c->cols)
        return ZERO_ERR_INVALID_ARG;
    if (x->rows == 0 || x->cols == 0)
        return ZERO_OK;
    const Span m[1] = {span_of(x)}, q[2] = {span_of_q(c), span_of_scale(c)};
    if (pack ? any_overlap(q, 2, m, 1) : any_overlap(m, 1, q, 2))
        return ZERO_ERR_INVALID_ARG;
    const void* p[3] = {x->base, c->q, c->scale};
    return require_device(p, 3);
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status_t zero_act_pack(const zero_mat_t* x, const zero_act8_t* out, void* stream)
{
    const zero_status_t st = check_pack(x, out, true);
    return st != ZERO_OK ? st : launch_pack(x, out, true, stream);
}

extern "C" zero_status_t zero_act_unpack(const zero_act8_t* in, const zero_mat_t* out,
                                         void* stream)
{
    const zero_status_t st = check_pack(out, in, false);
    return st != ZERO_OK ? st : launch_pack(out, in, false, stream);
}

extern "C" zero_status_t zero_norm_forward(const zero_mat_t* x, const zero_mat_t* residual,
                                           const void* gain, float eps, const zero_mat_t* h,
                                           const zero_mat_t* y, float* rstd,
                                           const zero_act8_t* checkpoint, void* stream)
{
    zero_status_t st = check_mat(x, true);
    if (st != ZERO_OK)
        return st;
    if ((!h && !y && !rstd && !checkpoint) || !(eps > 0.0f) || !(eps < 3.0e38f))
        return ZERO_ERR_INVALID_ARG;
    const zero_mat_t* mats[3] = {residual, h, y};
    for (const zero_mat_t* m : mats) {
        if (!m)
            continue;
        st = check_mat(m, true);
        if (st != ZERO_OK)
            return st;
        if (!same_shape(m, x))
            return ZERO_ERR_INVALID_ARG;
    }
    if (checkpoint) {
        st = check_act8(checkpoint);
        if (st != ZERO_OK)
            return st;
        if (checkpoint->rows != x->rows || checkpoint->cols != x->cols)
            return ZERO_ERR_INVALID_ARG;
    }
    if ((uintptr_t)gain % 2 != 0 || (uintptr_t)rstd % 4 != 0)
        return ZERO_ERR_ALIGNMENT;
    if (x->cols > ZERO_NORM_MAX_COLS)
        return ZERO_ERR_UNSUPPORTED;
    if (x->rows == 0 || x->cols == 0)
        return ZERO_OK;
    const Span none = span_of(nullptr, 0);
    const Span outs[5] = {h ? span_of(h) : none, y ? span_of(y) : none,
                          span_of(rstd, 4 * x->rows), checkpoint ? span_of_q(checkpoint) : none,
                          checkpoint ? span_of_scale(checkpoint) : none};
    // h may stand in for an input that it replaces
    const Span ins[3] = {h && same_place(h, x) ? none : span_of(x),
                         !residual || (h && same_place(h, residual)) ? none : span_of(residual),
                         span_of(gain, 2 * x->cols)};
    const Span whole[2] = {span_of(x), residual ? span_of(residual) : none};
    if (any_overlap(outs, 5, ins, 3) || any_overlap(outs + 1, 4, whole, 2))
        return ZERO_ERR_INVALID_ARG;
    const void* p[8];
    int n = 0;
    const void* all[8] = {x->base, residual ? residual->base : nullptr, gain,
                          h ? h->base : nullptr, y ? y->base : nullptr, rstd,
                          checkpoint ? checkpoint->q : nullptr,
                          checkpoint ? checkpoint->scale : nullptr};
    for (const void* q : all)
        if (q)
            p[n++] = q;
    st = require_device(p, n);
    if (st != ZERO_OK)
        return st;

    const NormShape sh = norm_shape(x->cols);
    if ((x->rows + sh.rows - 1) / sh.rows > 0x7FFFFFFFull)
        return ZERO_ERR_UNSUPPORTED;
    NormFwdArgs a = {};
    a.x = static_cast<const uint16_t*>(x->base);
    a.x_pitch = x->pitch;
    if (residual) {
        a.res = static_cast<const uint16_t*>(residual->base);
        a.res_pitch = residual->pitch;
    }
    a.gain = static_cast<const uint16_t*>(gain);
    a.gain_vec = aligned16(gain);
    if (h) {
        a.h = static_cast<uint16_t*>(h->base);
        a.h_pitch = h->pitch;
    }
    if (y) {
        a.y = static_cast<uint16_t*>(y->base);
        a.y_pitch = y->pitch;
    }
    a.rstd = rstd;
    if (checkpoint) {
        a.q = checkpoint->q;
        a.scale = checkpoint->scale;
        a.q_pitch = checkpoint->q_pitch;
        a.scale_pitch = checkpoint->scale_pitch;
    }
    a.rows = x->rows;
    a.cols = x->cols;
    a.group = sh.group;
    a.rows_per_cta = sh.rows;
    a.eps = eps;
    return train_status(x->dtype == ZERO_F16 ? launch_forward<ZERO_F16>(a, sh, stream)
                                             : launch_forward<ZERO_BF16>(a, sh, stream));
}

extern "C" uint64_t zero_norm_backward_workspace(uint64_t rows, uint64_t cols)
{
    if (cols > ZERO_NORM_MAX_COLS)
        return UINT64_MAX;
    if (rows == 0 || cols == 0)
        return 0;
    return backward_parts(rows, norm_shape(cols)) * ((cols + 7) / 8 * 8) * sizeof(float);
}

extern "C" zero_status_t zero_norm_backward(const zero_mat_t* dy, const zero_act8_t* checkpoint,
                                            const float* rstd, const void* gain,
                                            const zero_mat_t* d_residual, const zero_mat_t* dx,
                                            void* d_gain, uint32_t accumulate, void* workspace,
                                            uint64_t workspace_bytes, void* stream)
{
    zero_status_t st = check_mat(dy, true);
    if (st == ZERO_OK)
        st = check_mat(dx, true);
    if (st == ZERO_OK)
        st = check_act8(checkpoint);
    if (st == ZERO_OK && d_residual)
        st = check_mat(d_residual, true);
    if (st != ZERO_OK)
        return st;
    if (!same_shape(dy, dx) || (d_residual && !same_shape(dy, d_residual)) ||
        checkpoint->rows != dy->rows || checkpoint->cols != dy->cols || accumulate > 1 ||
        (!rstd && dy->rows && dy->cols))
        return ZERO_ERR_INVALID_ARG;
    if ((uintptr_t)gain % 2 != 0 || (uintptr_t)d_gain % 2 != 0 || (uintptr_t)rstd % 4 != 0)
        return ZERO_ERR_ALIGNMENT;
    if (dy->cols > ZERO_NORM_MAX_COLS)
        return ZERO_ERR_UNSUPPORTED;
    if (dy->cols == 0)
        return ZERO_OK;
    const uint64_t need = d_gain ? zero_norm_backward_workspace(dy->rows, dy->cols) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return ZERO_ERR_INVALID_ARG;
    if (need && !aligned16(workspace))
        return ZERO_ERR_ALIGNMENT;
    const Span none = span_of(nullptr, 0);
    const Span outs[3] = {span_of(dx), span_of(d_gain, 2 * dy->cols), span_of(workspace, need)};
    const Span ins[6] = {same_place(dx, dy) ? none : span_of(dy),
                         !d_residual || same_place(dx, d_residual) ? none : span_of(d_residual),
                         span_of_q(checkpoint), span_of_scale(checkpoint),
                         span_of(rstd, 4 * dy->rows), span_of(gain, 2 * dy->cols)};
    const Span whole[2] = {span_of(dy), d_residual ? span_of(d_residual) : none};
    if (any_overlap(outs, 3, ins, 6) || any_overlap(outs + 1, 2, whole, 2))
        return ZERO_ERR_INVALID_ARG;
    const void* p[9];
    int n = 0;
    const void* all[9] = {dy->base, checkpoint->q, checkpoint->scale, rstd, gain,
                          d_residual ? d_residual->base : nullptr, dx->base, d_gain,
                          need ? workspace : nullptr};
    for (const void* q : all)
        if (q)
            p[n++] = q;
    st = require_device(p, n);
    if (st != ZERO_OK)
        return st;

    const NormShape sh = norm_shape(dy->cols);
    const bool f16 = dy->dtype == ZERO_F16;
    const uint64_t pitch = (dy->cols + 7) / 8 * 8;
    cudaError_t e = cudaSuccess;
    uint32_t grid = 0;
    if (dy->rows) {
        const uint64_t room = (uint64_t)sm_count() * (2048 / sh.threads());
        if (room == 0)
            return ZERO_ERR_CUDA;
        const uint64_t parts = backward_parts(dy->rows, sh);
        grid = (uint32_t)(parts < room ? parts : room);
        NormBwdArgs a = {};
        a.dy = static_cast<const uint16_t*>(dy->base);
        a.dy_pitch = dy->pitch;
        a.q = checkpoint->q;
        a.scale = checkpoint->scale;
        a.q_pitch = checkpoint->q_pitch;
        a.scale_pitch = checkpoint->scale_pitch;
        a.rstd = rstd;
        a.gain = static_cast<const uint16_t*>(gain);
        a.gain_vec = aligned16(gain);
        if (d_residual) {
            a.dres = static_cast<const uint16_t*>(d_residual->base);
            a.dres_pitch = d_residual->pitch;
        }
        a.dx = static_cast<uint16_t*>(dx->base);
        a.dx_pitch = dx->pitch;
        a.parts = d_gain ? static_cast<float*>(workspace) : nullptr;
        a.part_pitch = pitch;
        a.rows = dy->rows;
        a.cols = dy->cols;
        a.group = sh.group;
        a.rows_per_cta = sh.rows;
        e = f16 ? launch_backward<ZERO_F16>(a, sh, grid, stream)
                : launch_backward<ZERO_BF16>(a, sh, grid, stream);
    }
    if (e == cudaSuccess && d_gain)
        e = launch_train(f16 ? k_norm_gain<ZERO_F16> : k_norm_gain<ZERO_BF16>,
                         dim3((unsigned)((dy->cols + 31) / 32)), 32 * kFoldSlices, 0, 1, stream,
                         static_cast<const float*>(workspace), grid, pitch, dy->cols, accumulate,
                         static_cast<uint16_t*>(d_gain));
    return train_status(e);
}
