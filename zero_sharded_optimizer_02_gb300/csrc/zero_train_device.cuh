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

// Elements [c, c + 8) of a row of `cols` elements; those past its end read as
// zero and are not touched.  VEC: the row's elements c lie on 16-byte
// boundaries (c is a multiple of 8).
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, uint64_t c, uint64_t cols)
{
    if (VEC && c + 8 <= cols)
        return *reinterpret_cast<const uint4*>(row + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols)
            w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool VEC>
__device__ __forceinline__ void store8_row(uint16_t* row, uint64_t c, uint64_t cols, uint4 v)
{
    if (VEC && c + 8 <= cols) {
        *reinterpret_cast<uint4*>(row + c) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < cols)
            row[c + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
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

// The 8 values that 8 bytes of a block with step `step` stand for (fp32, exact).
__device__ __forceinline__ void act8_unpack8(uint2 q, float step, float (&x)[8])
{
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = (float)(int)(int8_t)(w[i / 4] >> (8 * (i & 3))) * step;
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
