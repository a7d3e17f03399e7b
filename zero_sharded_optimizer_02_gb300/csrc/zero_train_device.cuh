// Device-side building blocks of the training operators (internal): launches,
// 16-bit vectors with ragged ends, and the 8-bit checkpoint's arithmetic.
#pragma once

#include <atomic>
#include <utility>

#include "zero_device.cuh"
#include "zero_train_internal.h"

namespace zero {
namespace {

// Launches `kern` (which starts with pdl_entry) as a programmatic dependent
// launch unless ZERO_PDL is "0", with a thread-block cluster of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_train(void (*kern)(KArgs...), dim3 grid, unsigned threads, size_t smem,
                         unsigned cluster, void* stream, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (pdl_launches()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// The status of a call whose launches returned `e`; takes the error off the
// runtime's record.
inline zero_status_t train_status(cudaError_t e)
{
    if (e == cudaSuccess)
        return ZERO_OK;
    (void)cudaGetLastError();
    return ZERO_ERR_CUDA;
}

// Streaming multiprocessors of the current device (0 on an error).
inline int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    return n;
}

// Lets `fn` use `bytes` of dynamic shared memory (once per device; `done` has
// a bit per device).
template <typename F>
void allow_smem(F* fn, size_t bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        dev = 64;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit))
        return;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
            cudaSuccess && bit)
        done.fetch_or(bit, std::memory_order_relaxed);
}

// -- 16-bit vectors of 8 elements ---------------------------------------------

template <int DT>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi)
{
    if (DT == ZERO_F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        uint32_t w;
        memcpy(&w, &h, sizeof(w));
        return w;
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        uint32_t w;
        memcpy(&w, &h, sizeof(w));
        return w;
    }
}

template <int DT>
__device__ __forceinline__ uint4 narrow8(const float (&v)[8])
{
    return make_uint4(narrow2<DT>(v[0], v[1]), narrow2<DT>(v[2], v[3]), narrow2<DT>(v[4], v[5]),
                      narrow2<DT>(v[6], v[7]));
}

// A word, a half or a byte, from global memory where `there` says so, else `other`.
// Nothing here looks at it, as a select after the load would: the load stays in
// flight until its value is needed.
__device__ __forceinline__ uint32_t load_word(const void* p, bool there, uint32_t other)
{
    uint32_t w;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, %3;\n\t"
                 "@p ld.global.u32 %0, [%1];\n\t}"
                 : "=&r"(w)
                 : "l"(p), "r"((uint32_t)there), "r"(other));
    return w;
}

__device__ __forceinline__ uint32_t load_half(const void* p, bool there, uint32_t other)
{
    uint32_t w;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, %3;\n\t"
                 "@p ld.global.u16 %0, [%1];\n\t}"
                 : "=&r"(w)
                 : "l"(p), "r"((uint32_t)there), "r"(other));
    return w;
}

__device__ __forceinline__ uint32_t load_byte(const void* p, bool there, uint32_t other)
{
    uint32_t w;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, %3;\n\t"
                 "@p ld.global.nc.u8 %0, [%1];\n\t}"
                 : "=&r"(w)
                 : "l"(p), "r"((uint32_t)there), "r"(other));
    return w;
}

// Up to 8 elements of a row on their way to registers, where nothing looks at
// them before values() does.  The row may start on any element: w[0..3] are the
// aligned words that hold two of them, w[4] the one before those (at an odd
// address) and w[5] the one behind; what is not there is zero.
struct Part8 {
    uint32_t w[6];

    __device__ __forceinline__ void load(const uint16_t* p, uint32_t n)
    {
        const uint32_t odd = reinterpret_cast<uintptr_t>(p) / 2 % 2, head = odd & (n != 0), words = (n - head) / 2;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            w[j] = load_word(p + head + 2 * j, j < words, 0);
        w[4] = load_half(p, head, 0);
        w[5] = load_half(p + n - 1, (n - head) % 2, 0);
    }

    // The elements in order, zeros behind them; p and n as load() had them.
    __device__ __forceinline__ uint4 values(const uint16_t* p, uint32_t n) const
    {
        const uint32_t odd = reinterpret_cast<uintptr_t>(p) / 2 % 2, head = odd & (n != 0), words = (n - head) / 2;
        uint32_t t[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            t[j] = j == words ? w[5] : w[j];
        return make_uint4(__funnelshift_l(w[4] << 16, t[0], 16 * odd), __funnelshift_l(t[0], t[1], 16 * odd),
                          __funnelshift_l(t[1], t[2], 16 * odd), __funnelshift_l(t[2], t[3], 16 * odd));
    }
};

// The elements that [c, c + 8) has of a row of `cols`.
__device__ __forceinline__ uint32_t part_of8(uint64_t c, uint64_t cols)
{
    return c >= cols ? 0 : cols - c < 8 ? (uint32_t)(cols - c) : 8;
}

// Elements [c, c + 8) of a row of `cols` elements; those past its end read as
// zero and are not touched.  VEC: the row's elements c lie on 16-byte
// boundaries (c is a multiple of 8).
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, uint64_t c, uint64_t cols)
{
    if (VEC && c + 8 <= cols)
        return *reinterpret_cast<const uint4*>(row + c);
    Part8 part;
    part.load(row + c, part_of8(c, cols));
    return part.values(row + c, part_of8(c, cols));
}

template <bool VEC>
__device__ __forceinline__ void store8_row(uint16_t* row, uint64_t c, uint64_t cols, uint4 v)
{
    if (VEC && c + 8 <= cols) {
        *reinterpret_cast<uint4*>(row + c) = v;
        return;
    }
    // whole words where the row has them (Part8)
    uint16_t* p = row + c;
    const uint32_t n = part_of8(c, cols), odd = reinterpret_cast<uintptr_t>(p) / 2 % 2, head = odd & (n != 0);
    const uint32_t words = (n - head) / 2;
    const uint32_t t[4] = {__funnelshift_r(v.x, v.y, 16 * odd), __funnelshift_r(v.y, v.z, 16 * odd),
                           __funnelshift_r(v.z, v.w, 16 * odd), v.w >> 16 * odd};
    if (head)
        p[0] = (uint16_t)v.x;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        if (j < words)
            *reinterpret_cast<uint32_t*>(p + head + 2 * j) = t[j];
        if (j == words && (n - head) % 2)
            p[n - 1] = (uint16_t)t[j];
    }
}

// Asynchronous copies of 16 or 8 bytes to shared memory, of which the first
// `bytes` (0: none, src is not touched) come from src and the others are zero.
__device__ __forceinline__ void cp_async16_part(void* dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void cp_async8_part(void* dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}

// 16 bytes from global memory, or zeros.  ONCE: not kept in L1.
template <bool ONCE>
__device__ __forceinline__ uint4 load16(const void* p, bool there)
{
    uint4 r;
    if (ONCE)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
                     "mov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
                     "@p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                     : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
                     : "l"(p), "r"((uint32_t)there));
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\t"
                     "mov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
                     "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                     : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
                     : "l"(p), "r"((uint32_t)there));
    return r;
}

// The n < 8 elements of a row's ragged end, at a 16-byte boundary: four of them
// in x and y, two in z, one in w, as n has them, for tail8() to put in order.
__device__ __forceinline__ uint4 load_tail8(const uint16_t* p, uint32_t n)
{
    uint4 r;
    r.x = load_word(p, n & 4, 0);
    r.y = load_word(p + 2, n & 4, 0);
    r.z = load_word(p + (n & 4), n & 2, 0);
    r.w = load_half(p + (n & 6), n & 1, 0);
    return r;
}

__device__ __forceinline__ uint4 tail8(uint4 r, uint32_t n)
{
    const uint32_t first = n & 2 ? r.z : r.w, second = n & 2 ? r.w : 0;
    return n & 4 ? make_uint4(r.x, r.y, first, second) : make_uint4(first, second, 0, 0);
}

// -- the 8-bit checkpoint -------------------------------------------------------

// Limits of a block's exponent k (zero_act8_t), by the activations' type.
template <int DT>
struct Act8Limits {
    static constexpr int lo = DT == ZERO_F16 ? -24 : -127;
    static constexpr int hi = DT == ZERO_F16 ? 9 : 121;
};

constexpr uint32_t kAct8Bad = 255;

// The scale byte of a block with largest magnitude a (a as fp32; an inf or
// NaN in the block arrives as a value with all exponent bits set).
// a = m * 2^e with 1 <= m < 2: 127 * 2^k >= a first holds for k = e - 6 if
// m <= 127/64 and e - 5 otherwise; adding 0x1FFFF carries into the exponent
// field exactly for the mantissas above 127/64.
template <int DT>
__device__ __forceinline__ uint32_t act8_scale(uint32_t a_bits)
{
    if ((a_bits & 0x7F800000u) == 0x7F800000u)
        return kAct8Bad;
    const int k = (int)((a_bits + 0x1FFFFu) >> 23) - 127 - 6;
    return (uint32_t)(min(max(k, Act8Limits<DT>::lo), Act8Limits<DT>::hi) + 127);
}

// 2^(s - 127) and its inverse; s = 255 gives NaN.  s = 0 is the subnormal 2^-127.
__device__ __forceinline__ float act8_step(uint32_t s)
{
    return __uint_as_float(s == kAct8Bad ? 0x7FC00000u : (s ? s << 23 : 0x00400000u));
}

__device__ __forceinline__ float act8_inverse(uint32_t s)
{
    return s == kAct8Bad ? 0.0f : __uint_as_float((254 - s) << 23);   // s <= 248
}

// x / 2^k to the nearest whole number in [-127, 127] (ties to even), as a byte.
// Both bounds hold for a NaN too, whose block has inverse 0 and bad = true.
__device__ __forceinline__ uint32_t act8_quant(float x, float inverse, bool bad)
{
    const float r = fminf(fmaxf(x * inverse, -127.0f), 127.0f);
    const int q = bad ? 0 : __float2int_rn(r);
    return (uint32_t)q & 0xFFu;
}

// Magnitude bits of a float: integer comparison orders magnitudes, and an inf
// or NaN is above every finite one.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Quantises 8 consecutive values that this thread holds, of a block of 32 that
// the aligned group of 4 lanes holds; every lane of the warp takes part.
// Returns the 8 bytes and the block's scale byte.
template <int DT>
__device__ __forceinline__ uint2 act8_pack8(const float (&x)[8], uint32_t& scale)
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = max(a, mag_bits(x[i]));
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    scale = act8_scale<DT>(a);
    const float inv = act8_inverse(scale);
    const bool bad = scale == kAct8Bad;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i / 4] |= act8_quant(x[i], inv, bad) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

// Adds 1.5 * 2^23 to a value of magnitude at most 2^22: the low byte of the sum
// is that of the nearest whole number (ties to even), two's complement.
constexpr float kRoundBias = 12582912.0f;

// act8_pack8 for finite values whose exponent k is not held down by its upper
// limit: then no x / 2^k passes 127 and one multiply-add rounds it.
__device__ __forceinline__ uint32_t act8_pack4(float a, float b, float c, float d, float inverse)
{
    const uint32_t lo = __byte_perm(__float_as_uint(fmaf(a, inverse, kRoundBias)),
                                    __float_as_uint(fmaf(b, inverse, kRoundBias)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(fmaf(c, inverse, kRoundBias)),
                                    __float_as_uint(fmaf(d, inverse, kRoundBias)), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// The 8 whole numbers of 8 bytes, as floats.
__device__ __forceinline__ void act8_whole8(uint2 q, float (&x)[8])
{
    const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};   // q + 128
#pragma unroll
    for (int i = 0; i < 8; ++i)   // 2^23 + 128 + q, exactly
        x[i] = __uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7540 | (i & 3))) - 8388736.0f;
}

__device__ __forceinline__ uint32_t bf2_add(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The step 2^(s - 127) of a scale byte in both halves of a word, in type DT.
// binary16 holds it for s in [103, 142]; another is kept as the byte itself
// under a mark (0xFFFF, which no step has), for convert4_wide.
template <int DT>
__device__ __forceinline__ uint32_t step2(uint32_t s)
{
    if (DT == ZERO_BF16) {
        const uint32_t h = s == kAct8Bad ? 0x7FC0u : (s ? s << 7 : 0x0040u);
        return h * 0x10001u;
    }
    if (s < 103 || (s > 142 && s != kAct8Bad))
        return 0xFFFF0000u | s;
    const uint32_t h = s == kAct8Bad ? 0x7E00u : s >= 113 ? (s - 112) << 10 : 0x0400u >> (113 - s);
    return h * 0x10001u;
}

// Four signed bytes times the step, as two words of two 16-bit values.
// bfloat16: a byte q is (128 + (q & 127)) - (q < 0 ? 256 : 128): 0x43 above the
// low 7 bits is 128 + them, and the sign bit is the lowest exponent bit that
// makes 0xC300 (-128) 0xC380 (-256).  binary16: 0x64 above the byte with its
// sign bit flipped is 1024 + 128 + q.  Every operation is exact.
template <int DT>
__device__ __forceinline__ void convert4(uint32_t w, uint32_t step, uint32_t& lo, uint32_t& hi)
{
    if (DT == ZERO_BF16) {
        const uint32_t mag = w & 0x7F7F7F7Fu, sign = w & 0x80808080u;
        lo = bf2_mul(bf2_add(__byte_perm(mag, 0x43434343u, 0x4140), __byte_perm(sign, 0xC3C3C3C3u, 0x4140)), step);
        hi = bf2_mul(bf2_add(__byte_perm(mag, 0x43434343u, 0x4342), __byte_perm(sign, 0xC3C3C3C3u, 0x4342)), step);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        lo = h2_mul(h2_sub(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u), step);
        hi = h2_mul(h2_sub(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u), step);
    }
}

// The same in fp32 with one rounding, for steps that binary16 does not hold.
__device__ __noinline__ uint2 convert4_wide(uint32_t w, uint32_t s)
{
    const float step = act8_step(s);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = (float)(int)(int8_t)(w >> (8 * i)) * step;
    return make_uint2(narrow2<ZERO_F16>(v[0], v[1]), narrow2<ZERO_F16>(v[2], v[3]));
}

// The 8 values that 8 bytes of a block with scale byte s stand for, in type DT.
template <int DT>
__device__ __forceinline__ uint4 act8_values8(uint2 q, uint32_t s)
{
    const uint32_t step = step2<DT>(s);
    uint4 r;
    if (DT == ZERO_F16 && step >> 16 == 0xFFFFu) {
        const uint2 a = convert4_wide(q.x, s), b = convert4_wide(q.y, s);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    convert4<DT>(q.x, step, r.x, r.y);
    convert4<DT>(q.y, step, r.z, r.w);
    return r;
}

// Bytes [c, c + 8) of a row of `cols` bytes whose byte c lies on an 8-byte
// boundary; those past its end read as zero and are not touched.
__device__ __forceinline__ uint2 load8_q(const int8_t* row, uint64_t c, uint64_t cols)
{
    if (c + 8 <= cols)
        return *reinterpret_cast<const uint2*>(row + c);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols)
            w[i / 4] |= (uint32_t)(uint8_t)row[c + i] << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store8_q(int8_t* row, uint64_t c, uint64_t cols, uint2 v)
{
    if (c + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + c) = v;
        return;
    }
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols)
            row[c + i] = (int8_t)(w[i / 4] >> (8 * (i & 3)));
}

}  // namespace
}  // namespace zero
