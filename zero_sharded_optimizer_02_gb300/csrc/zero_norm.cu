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
// in turn.  Each thread copies its own pieces of the next row to a ring in
// shared memory of its own (cp.async: no barrier, no registers).
//
// V = 4 where there are rows enough to fill the GPU: what a thread does once a
// row (the reduction, addresses, the square root) is then spread over 32
// elements.  With one vector a thread the kernels were bound by issuing
// instructions (73% of all slots, 59 an element): forward 117 us and backward
// 113 us at 16,384 x 4,096.  Few rows take V = 1: more threads a row, less
// latency.
struct NormShape {
    uint32_t group;   // G
    uint32_t vecs;    // V: 1, 2 or 4
    uint32_t rows;    // rows per CTA
    uint32_t threads() const { return group * rows; }
};

constexpr uint32_t kNormMinThreads = 128;
constexpr uint32_t kNormGroup = 512;        // most threads of a row of one vector a thread
constexpr uint32_t kNormMidGroup = 256;     // of two, or of four with registers for two CTAs an SM
constexpr uint32_t kNormWideGroup = 1024;   // of four
constexpr uint64_t kNormManyRows = 608;     // 4 rows an SM

NormShape norm_shape(uint64_t rows, uint64_t cols, bool backward)
{
    const uint32_t nv = (uint32_t)((cols + 7) / 8);
    uint32_t v = nv <= kNormGroup ? 1 : 4;
    if (rows >= kNormManyRows && nv >= 64)
        v = nv < 128 || (backward && nv <= 2 * kNormMidGroup) ? 2 : 4;
    const uint32_t g = ((nv + v - 1) / v + 31) / 32 * 32;
    return NormShape{g, v, g >= kNormMinThreads ? 1 : kNormMinThreads / g};
}

template <int V, bool WIDE, bool BACK>
struct NormLimits {
    static constexpr int threads = V == 1 ? (int)kNormGroup : (int)(WIDE ? kNormWideGroup : kNormMidGroup);
    // CTAs an SM that the registers are limited for.  16,384 x 4,096: forward
    // 101 us with 2, 98 with 3 (x 1,600: 52, 46); backward 117 with 3, 95 with 2,
    // 145 with 1 (more than two spill; four vectors spill 52 to 64 bytes with two).
    // WIDE: 1,024 threads leave 64 registers, of which the backward kernel spills
    // about 750 bytes, and no room for a row ahead: 2,048 x 16,384 forward 54 us
    // (5.7 TB/s), backward 141 (1.7 TB/s), where 4,096 x 8,192 take 53 and 63.
    static constexpr int ctas = WIDE ? 1 : V == 1 || BACK ? 2 : 3;
    static constexpr int ahead = V == 1 ? 3 : WIDE ? 0 : 1;   // rows
};

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
    uint64_t rows;
    uint32_t cols, group, rows_per_cta;
    uint32_t gain_vec;   // the gain lies on a 16-byte boundary
    float eps, inv_cols;
};

// Elements of vector j of this thread that the row has: 8, fewer at its end, 0
// past it.  FULL: the group's vectors cover exactly the row.
template <bool FULL>
__device__ __forceinline__ uint32_t have(uint32_t c, uint32_t cols)
{
    return FULL || c + 8 <= cols ? 8u : c < cols ? cols - c : 0u;
}

template <bool FULL>
__device__ __forceinline__ void store_have(uint16_t* p, uint32_t n, uint4 v)
{
    if (FULL || n == 8) {
        *reinterpret_cast<uint4*>(p) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
        if (i < n)
            p[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}

template <bool FULL>
__device__ __forceinline__ void store_have_q(int8_t* p, uint32_t n, uint2 v)
{
    if (FULL || n == 8) {
        *reinterpret_cast<uint2*>(p) = v;
        return;
    }
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i)
        if (i < n)
            p[i] = (int8_t)(w[i / 4] >> (8 * (i & 3)));
}

// The gain at columns [c, c + 8); it stays in L1.
template <int DT, bool FULL>
__device__ __forceinline__ void load_gain(const uint16_t* gain, uint32_t vec, uint32_t c, uint32_t cols, float (&g)[8])
{
    if (vec && (FULL || c + 8 <= cols))
        set8<DT>(g, __ldg(reinterpret_cast<const uint4*>(gain + c)));
    else
        set8<DT>(g, load8<false>(gain, c, cols));
}

// The ring: [stage][array][vector][thread] of 16 bytes.
template <int V>
__device__ __forceinline__ uint4* ring_at(uint4* ring, int stage, int array, int j)
{
    return ring + ((stage * 2 + array) * V + j) * blockDim.x + threadIdx.x;
}

// Copies this thread's pieces of one row; p, r: the row at its first column.
template <int V, bool FULL>
__device__ __forceinline__ void fetch_pair(uint4* ring, int stage, const uint16_t* p, const uint16_t* r, uint32_t group8,
                                           uint32_t c, uint32_t cols)
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t n = 2 * have<FULL>(c + j * group8, cols), o = n ? j * group8 : 0;
        cp_async16_part(ring_at<V>(ring, stage, 0, j), p + o, n);
        if (r)
            cp_async16_part(ring_at<V>(ring, stage, 1, j), r + o, n);
    }
}

// Bound by memory.  16,384 x 4,096 with residual, h, y and checkpoint: 606 MB in
// 98 us (6.2 TB/s), 337 of them written (a memset writes 4.0 TB/s at most).
template <int DT, int V, bool WIDE, bool FULL>
__global__ void __launch_bounds__(NormLimits<V, WIDE, false>::threads, NormLimits<V, WIDE, false>::ctas) k_norm_forward(const NormFwdArgs a)
{
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ float sums[2][32];
    constexpr int kAhead = NormLimits<V, WIDE, false>::ahead;
    pdl_entry();
    const uint32_t lane = threadIdx.x % a.group, mine = threadIdx.x / a.group;
    const uint32_t c0 = lane * 8, group8 = a.group * 8;
    const uint64_t hop = (uint64_t)gridDim.x * a.rows_per_cta;
    uint64_t row = (uint64_t)blockIdx.x * a.rows_per_cta + mine;
    // the row that is copied next, and its first column of this thread (a thread
    // wholly past the row's end stays at column 0 and copies nothing)
    const uint32_t at = have<FULL>(c0, a.cols) ? c0 : 0;
    uint64_t ahead = row;
    const uint16_t* px = a.x + row * a.x_pitch + at;
    const uint16_t* pr = a.res ? a.res + row * a.res_pitch + at : nullptr;
    auto fetch = [&](int stage) {
        if (ahead < a.rows)
            fetch_pair<V, FULL>(ring, stage, px, pr, group8, c0, a.cols);
        cp_async_commit();
        ahead += hop;
        px += hop * a.x_pitch;
        if (pr)
            pr += hop * a.res_pitch;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        fetch(k);
    int flip = 0, stage = 0;
    // the same number of turns in every group of the CTA
    for (uint64_t r0 = (uint64_t)blockIdx.x * a.rows_per_cta; r0 < a.rows; r0 += hop, row += hop) {
        const bool live = row < a.rows;   // the ring of a group past the last row holds any values
        if (kAhead == 0)
            fetch(0);
        cp_async_wait<kAhead ? kAhead - 1 : 0>();
        float s[V][8];
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            set8<DT>(s[j], *ring_at<V>(ring, stage, 0, j));
            if (pr)
                add8<DT>(s[j], *ring_at<V>(ring, stage, 1, j));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                ss += s[j][i] * s[j][i];
        }
        if (kAhead)
            fetch(stage ? stage - 1 : kAhead);   // the stage that the last row freed
        stage = stage == kAhead ? 0 : stage + 1;
        ss = group_sum(ss, a.group, sums[flip]);
        flip ^= 1;
        const float rstd = __frsqrt_rn(ss * a.inv_cols + a.eps);
        if (live && lane == 0 && a.rstd)
            a.rstd[row] = rstd;
        if (a.h && live) {
            uint16_t* p = a.h + row * a.h_pitch + c0;
#pragma unroll
            for (int j = 0; j < V; ++j)
                store_have<FULL>(p + j * group8, have<FULL>(c0 + j * group8, a.cols), narrow8<DT>(s[j]));
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[j][i] *= rstd;   // xhat
        if (a.q) {
            int8_t* p = a.q + row * a.q_pitch + c0;
            uint8_t* sp = a.scale + row * a.scale_pitch + c0 / ZERO_ACT8_BLOCK;
            const bool lost = nonfinite(ss);   // the same in the whole group
#pragma unroll
            for (int j = 0; j < V; ++j) {
                // elements past the row's end are zero: copied as zero
                uint32_t sc;
                uint2 q;
                if (lost) {
                    q = act8_pack8<DT>(s[j], sc);
                } else {   // |xhat| <= sqrt(cols): far below the exponent's upper limit
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        m = fmaxf(m, fabsf(s[j][i]));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
                    sc = act8_scale<DT>(__float_as_uint(m));
                    const float inv = act8_inverse(sc);
                    q = make_uint2(act8_pack4(s[j][0], s[j][1], s[j][2], s[j][3], inv),
                                   act8_pack4(s[j][4], s[j][5], s[j][6], s[j][7], inv));
                }
                const uint32_t n = have<FULL>(c0 + j * group8, a.cols);
                if (live && (FULL || n)) {
                    store_have_q<FULL>(p + j * group8, n, q);
                    if (lane % 4 == 0)   // group8 is a multiple of the block
                        sp[j * (group8 / ZERO_ACT8_BLOCK)] = (uint8_t)sc;
                }
            }
        }
        if (a.y && live) {
            uint16_t* p = a.y + row * a.y_pitch + c0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t c = c0 + j * group8;
                float g[8];
                if (a.gain) {
                    load_gain<DT, FULL>(a.gain, a.gain_vec, c, a.cols, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        s[j][i] *= g[i];
                }
                store_have<FULL>(p + j * group8, have<FULL>(c, a.cols), narrow8<DT>(s[j]));
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
    uint64_t rows;
    uint32_t cols, group, rows_per_cta;
    uint32_t gain_vec;
    float inv_cols;
};

// 16,384 x 4,096 with a residual's gradient: 472 MB in 94 us (5.0 TB/s), bound by
// the latency that two CTAs an SM can cover.  The gain's gradient stays in
// registers over a CTA's rows and leaves one partial row a CTA.  What lies past a row's end is copied as zero; the sums that a lost block's NaN step
// makes of it there are not read.
template <int DT, int V, bool WIDE, bool FULL>
__global__ void __launch_bounds__(NormLimits<V, WIDE, true>::threads, NormLimits<V, WIDE, true>::ctas) k_norm_backward(const NormBwdArgs a)
{
    extern __shared__ __align__(16) uint4 ring[];
    __shared__ float sums[2][32];
    constexpr int kAhead = NormLimits<V, WIDE, true>::ahead;
    pdl_entry();
    const uint32_t lane = threadIdx.x % a.group, mine = threadIdx.x / a.group;
    const uint32_t c0 = lane * 8, group8 = a.group * 8;
    const uint64_t hop = (uint64_t)gridDim.x * a.rows_per_cta;
    uint64_t row = (uint64_t)blockIdx.x * a.rows_per_cta + mine;
    float dg[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dg[j][i] = 0.0f;
    // behind the ring of dy and dres, one of the checkpoint's bytes, 8 a vector
    uint2* qring = reinterpret_cast<uint2*>(ring + (kAhead + 1) * 2 * V * blockDim.x) + threadIdx.x;
    const uint32_t at = have<FULL>(c0, a.cols) ? c0 : 0;
    uint64_t ahead = row;
    const uint16_t* pd = a.dy + row * a.dy_pitch + at;
    const uint16_t* pr = a.dres ? a.dres + row * a.dres_pitch + at : nullptr;
    const int8_t* pq = a.q + row * a.q_pitch + at;
    const uint8_t* ps = a.scale + row * a.scale_pitch + at / ZERO_ACT8_BLOCK;
    auto fetch = [&](int stage) {
        if (ahead < a.rows) {
            fetch_pair<V, FULL>(ring, stage, pd, pr, group8, c0, a.cols);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const uint32_t n = have<FULL>(c0 + j * group8, a.cols);
                cp_async8_part(qring + (stage * V + j) * blockDim.x, pq + (n ? j * group8 : 0), n);
            }
        }
        cp_async_commit();
        ahead += hop;
        pd += hop * a.dy_pitch;
        pq += hop * a.q_pitch;
        if (pr)
            pr += hop * a.dres_pitch;
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        fetch(k);
    // scale bytes and rstd: one row ahead, in registers
    uint32_t next_s[V], next_rstd;
    auto scales = [&](uint64_t r) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            next_s[j] = load_byte(ps + j * (group8 / ZERO_ACT8_BLOCK),
                                  r < a.rows && have<FULL>(c0 + j * group8, a.cols), 127);
        next_rstd = load_word(a.rstd + r, r < a.rows, 0);
        ps += hop * a.scale_pitch;
    };
    scales(row);
    int flip = 0, stage = 0;
    for (uint64_t r0 = (uint64_t)blockIdx.x * a.rows_per_cta; r0 < a.rows; r0 += hop, row += hop) {
        const bool live = row < a.rows;
        if (kAhead == 0)
            fetch(0);
        cp_async_wait<kAhead ? kAhead - 1 : 0>();
        const float rstd = __uint_as_float(next_rstd);
        float u[V][8], xhat[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float step = act8_step(next_s[j]);
            act8_whole8(qring[(stage * V + j) * blockDim.x], xhat[j]);
            set8<DT>(u[j], *ring_at<V>(ring, stage, 0, j));
            if (!live)   // the ring holds any values: not to be summed
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    u[j][i] = xhat[j][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                xhat[j][i] *= step;
                dg[j][i] += u[j][i] * xhat[j][i];
            }
            if (a.gain) {
                float g[8];
                load_gain<DT, FULL>(a.gain, a.gain_vec, c0 + j * group8, a.cols, g);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    u[j][i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dot += u[j][i] * xhat[j][i];
        }
        if (kAhead)
            fetch(stage ? stage - 1 : kAhead);
        scales(row + hop);
        dot = group_sum(dot, a.group, sums[flip]);
        flip ^= 1;
        if (live) {
            const float mean = dot * a.inv_cols * rstd;
            uint16_t* p = a.dx + row * a.dx_pitch + c0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float r[8];
                if (pr)
                    set8<DT>(r, *ring_at<V>(ring, stage, 1, j));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = rstd * u[j][i] - mean * xhat[j][i];
                    r[i] = pr ? r[i] + d : d;
                }
                store_have<FULL>(p + j * group8, have<FULL>(c0 + j * group8, a.cols), narrow8<DT>(r));
            }
        }
        stage = stage == kAhead ? 0 : stage + 1;
    }
    if (!a.parts)
        return;
    if (a.rows_per_cta > 1) {   // fold the groups' sums in group order
        const uint32_t width = group8 * V;
        float* fold = reinterpret_cast<float*>(ring);   // 32 of the ring's 40 bytes a vector and stage
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                fold[mine * width + j * group8 + c0 + i] = dg[j][i];
        __syncthreads();
        if (mine != 0)
            return;
        for (uint32_t m = 1; m < a.rows_per_cta; ++m)
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dg[j][i] += fold[m * width + j * group8 + c0 + i];
    }
    float* part = a.parts + blockIdx.x * a.part_pitch;   // part_pitch: cols rounded up to 8
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t c = c0 + j * group8;
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

// Shared memory of a forward (two arrays of 16 bytes a vector) or backward
// (and one of 8) CTA.
template <int V, bool WIDE, bool BACK>
constexpr size_t ring_bytes(uint32_t threads)
{
    return (size_t)(NormLimits<V, WIDE, BACK>::ahead + 1) * V * threads * (BACK ? 40 : 32);
}
template <int V, bool WIDE, bool BACK>
constexpr bool ring_fits()
{
    using L = NormLimits<V, WIDE, BACK>;
    return ring_bytes<V, WIDE, BACK>(L::threads) * L::ctas <= 220 * 1024;
}
static_assert(ring_fits<1, false, false>() && ring_fits<2, false, false>() && ring_fits<4, false, false>() &&
                  ring_fits<4, true, false>() && ring_fits<1, false, true>() && ring_fits<2, false, true>() &&
                  ring_fits<4, false, true>() && ring_fits<4, true, true>(),
              "rings exceed shared memory");

bool norm_full(const NormShape& sh, uint64_t cols) { return (uint64_t)sh.group * sh.vecs * 8 == cols; }

template <int DT, int V, bool WIDE, bool FULL>
cudaError_t launch_forward(const NormFwdArgs& a, const NormShape& sh, uint32_t grid, void* stream)
{
    static std::atomic<uint64_t> allowed{0};
    allow_smem(k_norm_forward<DT, V, WIDE, FULL>, (ring_bytes<V, WIDE, false>(NormLimits<V, WIDE, false>::threads)), allowed);
    return launch_train(k_norm_forward<DT, V, WIDE, FULL>, dim3(grid), sh.threads(),
                        (ring_bytes<V, WIDE, false>(sh.threads())), 1, stream, a);
}

template <int DT>
cudaError_t launch_forward(const NormFwdArgs& a, const NormShape& sh, uint32_t grid, void* stream)
{
    if (sh.vecs == 1)
        return launch_forward<DT, 1, false, false>(a, sh, grid, stream);
    if (sh.vecs == 2)
        return norm_full(sh, a.cols) ? launch_forward<DT, 2, false, true>(a, sh, grid, stream)
                                     : launch_forward<DT, 2, false, false>(a, sh, grid, stream);
    if (sh.group > kNormMidGroup)
        return launch_forward<DT, 4, true, false>(a, sh, grid, stream);
    return norm_full(sh, a.cols) ? launch_forward<DT, 4, false, true>(a, sh, grid, stream)
                                 : launch_forward<DT, 4, false, false>(a, sh, grid, stream);
}

template <int DT, int V, bool WIDE, bool FULL>
cudaError_t launch_backward(const NormBwdArgs& a, const NormShape& sh, uint32_t grid, void* stream)
{
    static std::atomic<uint64_t> allowed{0};
    allow_smem(k_norm_backward<DT, V, WIDE, FULL>, (ring_bytes<V, WIDE, true>(NormLimits<V, WIDE, true>::threads)), allowed);
    return launch_train(k_norm_backward<DT, V, WIDE, FULL>, dim3(grid), sh.threads(),
                        (ring_bytes<V, WIDE, true>(sh.threads())), 1, stream, a);
}

template <int DT>
cudaError_t launch_backward(const NormBwdArgs& a, const NormShape& sh, uint32_t grid, void* stream)
{
    if (sh.vecs == 1)
        return launch_backward<DT, 1, false, false>(a, sh, grid, stream);
    if (sh.vecs == 2)
        return norm_full(sh, a.cols) ? launch_backward<DT, 2, false, true>(a, sh, grid, stream)
                                     : launch_backward<DT, 2, false, false>(a, sh, grid, stream);
    if (sh.group > kNormMidGroup)
        return launch_backward<DT, 4, true, false>(a, sh, grid, stream);
    return norm_full(sh, a.cols) ? launch_backward<DT, 4, false, true>(a, sh, grid, stream)
                                 : launch_backward<DT, 4, false, false>(a, sh, grid, stream);
}

// Resident CTAs an SM that a grid is sized for: NormLimits' threads and ctas.
uint32_t norm_ctas_per_sm(const NormShape& sh, bool backward)
{
    const uint32_t threads =
        sh.vecs == 1 || sh.group > kNormMidGroup ? 1024 : (backward ? 2 : 3) * kNormMidGroup;
    return sh.threads() < threads ? threads / sh.threads() : 1;
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
// 16,384 x 6,400: pack 47 us (6.8 TB/s), unpack 58 us (3.6 TB/s written).
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

    const NormShape sh = norm_shape(x->rows, x->cols, false);
    const uint64_t ctas = (x->rows + sh.rows - 1) / sh.rows;
    const uint64_t room = (uint64_t)sm_count() * norm_ctas_per_sm(sh, false);
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
    a.cols = (uint32_t)x->cols;
    a.inv_cols = (float)(1.0 / (double)x->cols);
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
    return backward_parts(rows, norm_shape(rows, cols, true)) * ((cols + 7) / 8 * 8) * sizeof(float);
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

    const NormShape sh = norm_shape(dy->rows, dy->cols, true);
    const bool f16 = dy->dtype == ZERO_F16;
    const uint64_t pitch = (dy->cols + 7) / 8 * 8;
    cudaError_t e = cudaSuccess;
    uint32_t grid = 0;
    if (dy->rows) {
        const uint64_t room = (uint64_t)sm_count() * norm_ctas_per_sm(sh, true);
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
        a.cols = (uint32_t)dy->cols;
        a.inv_cols = (float)(1.0 / (double)dy->cols);
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
