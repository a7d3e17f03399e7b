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
// four neighbouring lanes hold one block of the checkpoint.  A CTA takes rows
// in turn and loads the next one while it works on one.
struct NormShape {
    uint32_t group;   // G
    uint32_t vecs;    // V: 1, 2 or 4
    uint32_t rows;    // rows per CTA
    uint32_t threads() const { return group * rows; }
};

constexpr uint32_t kNormMinThreads = 128;
constexpr uint32_t kNormGroup = 512;   // most threads of a row of one or two vectors a thread
constexpr uint32_t kNormWideGroup = 1024;

// One vector a thread as far as kNormGroup threads go, then two, then four.
NormShape norm_shape(uint64_t cols)
{
    const uint32_t nv = (uint32_t)((cols + 7) / 8);
    const uint32_t v = nv <= kNormGroup ? 1 : nv <= 2 * kNormGroup ? 2 : 4;
    const uint32_t g = ((nv + v - 1) / v + 31) / 32 * 32;
    return NormShape{g, v, g >= kNormMinThreads ? 1 : kNormMinThreads / g};
}

template <int V>
struct NormLimits {   // threads of a CTA
    static constexpr int threads = V == 4 ? (int)kNormWideGroup : (int)kNormGroup;
};

// Resident CTAs an SM that a grid of rows-in-turn CTAs is sized for.
uint32_t norm_ctas_per_sm(const NormShape& sh, uint32_t threads_per_sm)
{
    return sh.threads() < threads_per_sm ? threads_per_sm / sh.threads() : 1;
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

// One vector of a row, as it is loaded.
struct FwdRaw {
    uint4 x, res;
};

template <int V>
__device__ __forceinline__ void load_forward(const NormFwdArgs& a, uint64_t row, uint32_t lane, FwdRaw (&r)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        const bool in = row < a.rows && c < a.cols;
        r[j].x = in ? load8<true>(a.x + row * a.x_pitch, c, a.cols) : make_uint4(0, 0, 0, 0);
        r[j].res = in && a.res ? load8<true>(a.res + row * a.res_pitch, c, a.cols) : make_uint4(0, 0, 0, 0);
    }
}

// Bound by memory.  16,384 x 4,096 with residual, h, y and checkpoint: 606 MB.
template <int DT, int V>
__global__ void __launch_bounds__(NormLimits<V>::threads, V == 4 ? 1 : 2) k_norm_forward(const NormFwdArgs a)
{
    __shared__ float sums[2][32];
    pdl_entry();
    const uint32_t lane = threadIdx.x % a.group;
    uint64_t row = (uint64_t)blockIdx.x * a.rows_per_cta + threadIdx.x / a.group;
    const uint64_t hop = (uint64_t)gridDim.x * a.rows_per_cta;
    uint4 gain[V];   // of this thread's columns, 16-bit
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        gain[j] = !a.gain ? make_uint4(0, 0, 0, 0)
                          : a.gain_vec ? load8<true>(a.gain, c, a.cols) : load8<false>(a.gain, c, a.cols);
    }
    FwdRaw next[V];
    load_forward<V>(a, row, lane, next);
    int flip = 0;
    // the same number of turns in every group of the CTA
    for (uint64_t r0 = (uint64_t)blockIdx.x * a.rows_per_cta; r0 < a.rows; r0 += hop, row += hop) {
        const bool live = row < a.rows;
        float s[V][8];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            set8<DT>(s[j], next[j].x);
            if (a.res)
                add8<DT>(s[j], next[j].res);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss += s[j][i] * s[j][i];
        }
        if (r0 + hop < a.rows)
            load_forward<V>(a, row + hop, lane, next);
        ss = group_sum(ss, a.group, sums[flip]);
        flip ^= 1;
        const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.cols) + a.eps);
        if (live && lane == 0 && a.rstd)
            a.rstd[row] = rstd;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
            const bool in = live && c < a.cols;
            if (a.h && in)
                store8_row<true>(a.h + row * a.h_pitch, c, a.cols, narrow8<DT>(s[j]));
            float xhat[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                xhat[i] = s[j][i] * rstd;
            if (a.y && in) {
                float y[8];
                if (a.gain) {
                    set8<DT>(y, gain[j]);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] *= xhat[i];
                    store8_row<true>(a.y + row * a.y_pitch, c, a.cols, narrow8<DT>(y));
                } else {
                    store8_row<true>(a.y + row * a.y_pitch, c, a.cols, narrow8<DT>(xhat));
                }
            }
            if (a.q) {
                // elements past the row's end are zero: loaded as zero
                uint32_t sc;
                uint2 q;
                if (nonfinite(ss)) {   // the same in the whole group
                    q = act8_pack8<DT>(xhat, sc);
                } else {   // |xhat| <= sqrt(cols): far below the exponent's upper limit
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        m = fmaxf(m, fabsf(xhat[i]));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                    sc = act8_scale<DT>(__float_as_uint(m));
                    const float inv = act8_inverse(sc);
                    q = make_uint2(act8_pack4(xhat[0], xhat[1], xhat[2], xhat[3], inv),
                                   act8_pack4(xhat[4], xhat[5], xhat[6], xhat[7], inv));
                }
                if (in) {
                    store8_q(a.q + row * a.q_pitch, c, a.cols, q);
                    if (c % ZERO_ACT8_BLOCK == 0)
                        a.scale[row * a.scale_pitch + c / ZERO_ACT8_BLOCK] = (uint8_t)sc;
                }
            }
        }
    }
}

// Most CTAs of the backward kernel, each of which leaves one partial row of
// the gain's gradient: 8 CTAs of 128 threads on each of 152 SMs.
constexpr uint32_t kNormMaxParts = 1216;
constexpr uint32_t kNormBackThreads = 1024;   // resident threads an SM it is sized for

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

struct BwdRaw {
    uint4 dy, dres;
    uint2 q;
    uint32_t s;
};

template <int V>
__device__ __forceinline__ void load_backward(const NormBwdArgs& a, uint64_t row, uint32_t lane, BwdRaw (&r)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        const bool in = row < a.rows && c < a.cols;
        r[j].dy = in ? load8<true>(a.dy + row * a.dy_pitch, c, a.cols) : make_uint4(0, 0, 0, 0);
        r[j].q = in ? load8_q(a.q + row * a.q_pitch, c, a.cols) : make_uint2(0, 0);
        r[j].s = in ? a.scale[row * a.scale_pitch + c / ZERO_ACT8_BLOCK] : 127;
        r[j].dres = in && a.dres ? load8<true>(a.dres + row * a.dres_pitch, c, a.cols) : make_uint4(0, 0, 0, 0);
    }
}

// Bound by memory.  What lies past a row's end is loaded as zero; the sums that
// a lost block's NaN step makes of it there are not read.
template <int DT, int V>
__global__ void __launch_bounds__(NormLimits<V>::threads, V == 1 ? 2 : 1) k_norm_backward(const NormBwdArgs a)
{
    __shared__ float sums[2][32];
    __shared__ float fold[kNormMinThreads * 8];   // only CTAs of several groups, which hold one vector a thread
    pdl_entry();
    const uint32_t lane = threadIdx.x % a.group, mine = threadIdx.x / a.group;
    const uint64_t hop = (uint64_t)gridDim.x * a.rows_per_cta;
    float dg[V][8];
    uint4 gain[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
        gain[j] = !a.gain ? make_uint4(0, 0, 0, 0)
                          : a.gain_vec ? load8<true>(a.gain, c, a.cols) : load8<false>(a.gain, c, a.cols);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dg[j][i] = 0.0f;
    }
    uint64_t row = (uint64_t)blockIdx.x * a.rows_per_cta + mine;
    BwdRaw next[V];
    load_backward<V>(a, row, lane, next);
    float next_rstd = row < a.rows ? a.rstd[row] : 0.0f;
    int flip = 0;
    for (uint64_t r0 = (uint64_t)blockIdx.x * a.rows_per_cta; r0 < a.rows; r0 += hop, row += hop) {
        const bool live = row < a.rows;
        const float rstd = next_rstd;
        float u[V][8], xhat[V][8];
        uint4 dres[V];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float step = act8_step(next[j].s);
            dres[j] = next[j].dres;
            act8_whole8(next[j].q, xhat[j]);
            float g[8];
            set8<DT>(g, gain[j]);
            set8<DT>(u[j], next[j].dy);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xhat[j][i] *= step;
                const float t = u[j][i] * xhat[j][i];
                dg[j][i] += t;
                dot += a.gain ? g[i] * t : t;
                if (a.gain)
                    u[j][i] *= g[i];
            }
        }
        if (r0 + hop < a.rows) {
            load_backward<V>(a, row + hop, lane, next);
            next_rstd = row + hop < a.rows ? a.rstd[row + hop] : 0.0f;
        }
        dot = group_sum(dot, a.group, sums[flip]);
        flip ^= 1;
        if (live) {
            const float mean = __fdiv_rn(dot, (float)a.cols) * rstd;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint64_t c = ((uint64_t)j * a.group + lane) * 8;
                if (c >= a.cols)
                    continue;
                float r[8];
                set8<DT>(r, dres[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] += rstd * u[j][i] - mean * xhat[j][i];
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
constexpr int kFoldSlices = 32;
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
cudaError_t launch_forward(const NormFwdArgs& a, const NormShape& sh, uint32_t grid, void* stream)
{
    switch (sh.vecs) {
    case 1: return launch_train(k_norm_forward<DT, 1>, dim3(grid), sh.threads(), 0, 1, stream, a);
    case 2: return launch_train(k_norm_forward<DT, 2>, dim3(grid), sh.threads(), 0, 1, stream, a);
    default: return launch_train(k_norm_forward<DT, 4>, dim3(grid), sh.threads(), 0, 1, stream, a);
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
constexpr int kPackUnroll = 2;

struct PackArgs {
    uint16_t* x;
    int8_t* q;
    uint8_t* scale;
    uint64_t x_pitch, q_pitch, scale_pitch;
    uint64_t cols;
    uint32_t slots;   // 16-element slots a row: 2 per block, so a block is 2 neighbouring lanes
    uint32_t items;   // slots * rows of this launch
};

// 16 elements of a row from c on, as two vectors.
struct Half {
    uint4 lo, hi;
};

// Bound by memory: 3.03 bytes an element, of which pack writes 1.03 and unpack 2.
template <int DT>
__global__ void __launch_bounds__(kPackThreads) k_act_pack(const PackArgs a)
{
    pdl_entry();
    const uint32_t i0 = blockIdx.x * (kPackThreads * kPackUnroll) + threadIdx.x;
    Half w[kPackUnroll];
    uint32_t row[kPackUnroll];
    uint64_t col[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        const uint32_t i = i0 + u * kPackThreads;
        w[u].lo = w[u].hi = make_uint4(0, 0, 0, 0);
        row[u] = i / a.slots;
        col[u] = (uint64_t)(i - row[u] * a.slots) * 16;
        if (i < a.items && col[u] < a.cols) {
            const uint16_t* p = a.x + row[u] * a.x_pitch;
            w[u].lo = load8<true>(p, col[u], a.cols);
            w[u].hi = load8<true>(p, col[u] + 8, a.cols);
        }
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        float x[2][8];
        set8<DT>(x[0], w[u].lo);
        set8<DT>(x[1], w[u].hi);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, max(mag_bits(x[0][i]), mag_bits(x[1][i])));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const uint32_t sc = act8_scale<DT>(m);
        const float inv = act8_inverse(sc);
        uint32_t q[4];
        if (sc < Act8Limits<DT>::hi + 127) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float(&v)[8] = x[k / 2];
                const int o = k % 2 * 4;
                q[k] = act8_pack4(v[o], v[o + 1], v[o + 2], v[o + 3], inv);
            }
        } else {   // held down by the exponent's limit, or lost
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                q[k] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[k] |= act8_quant(x[k / 2][k % 2 * 4 + i], inv, sc == kAct8Bad) << (8 * i);
            }
        }
        if (i0 + u * kPackThreads < a.items && col[u] < a.cols) {
            int8_t* p = a.q + row[u] * a.q_pitch;
            if (col[u] + 16 <= a.cols) {
                *reinterpret_cast<uint4*>(p + col[u]) = make_uint4(q[0], q[1], q[2], q[3]);
            } else {
                store8_q(p, col[u], a.cols, make_uint2(q[0], q[1]));
                store8_q(p, col[u] + 8, a.cols, make_uint2(q[2], q[3]));
            }
            if (col[u] % ZERO_ACT8_BLOCK == 0)
                a.scale[row[u] * a.scale_pitch + col[u] / ZERO_ACT8_BLOCK] = (uint8_t)sc;
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kPackThreads) k_act_unpack(const PackArgs a)
{
    pdl_entry();
    const uint32_t i0 = blockIdx.x * (kPackThreads * kPackUnroll) + threadIdx.x;
    uint4 q[kPackUnroll];
    uint32_t sc[kPackUnroll], row[kPackUnroll];
    uint64_t col[kPackUnroll];
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u) {
        const uint32_t i = i0 + u * kPackThreads;
        q[u] = make_uint4(0, 0, 0, 0);
        sc[u] = 127;
        row[u] = i / a.slots;
        col[u] = (uint64_t)(i - row[u] * a.slots) * 16;
        if (i < a.items && col[u] < a.cols) {
            const int8_t* p = a.q + row[u] * a.q_pitch;
            if (col[u] + 16 <= a.cols) {
                q[u] = *reinterpret_cast<const uint4*>(p + col[u]);
            } else {
                const uint2 lo = load8_q(p, col[u], a.cols), hi = load8_q(p, col[u] + 8, a.cols);
                q[u] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
            sc[u] = a.scale[row[u] * a.scale_pitch + col[u] / ZERO_ACT8_BLOCK];
        }
    }
#pragma unroll
    for (int u = 0; u < kPackUnroll; ++u)
        if (i0 + u * kPackThreads < a.items && col[u] < a.cols) {
            uint16_t* p = a.x + row[u] * a.x_pitch;
            store8_row<true>(p, col[u], a.cols, act8_values8<DT>(make_uint2(q[u].x, q[u].y), sc[u]));
            store8_row<true>(p, col[u] + 8, a.cols, act8_values8<DT>(make_uint2(q[u].z, q[u].w), sc[u]));
        }
}

// Pack and unpack run in launches of at most 2^30 slots, so that item numbers
// stay in 32 bits.
zero_status_t launch_pack(const zero_mat_t* x, const zero_act8_t* c, bool pack, void* stream)
{
    if (x->rows == 0 || x->cols == 0)
        return ZERO_OK;
    const uint64_t slots = (x->cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK * 2;
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
    const uint64_t ctas = (x->rows + sh.rows - 1) / sh.rows;
    const uint64_t room = (uint64_t)sm_count() * norm_ctas_per_sm(sh, 1024);
    if (room == 0)
        return ZERO_ERR_CUDA;
    const uint32_t grid = (uint32_t)(ctas < room ? ctas : room);
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
    return train_status(x->dtype == ZERO_F16 ? launch_forward<ZERO_F16>(a, sh, grid, stream)
                                             : launch_forward<ZERO_BF16>(a, sh, grid, stream));
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
        const uint64_t room = (uint64_t)sm_count() * norm_ctas_per_sm(sh, kNormBackThreads);
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
