// Weight gradient of a linear layer from an 8-bit checkpoint of its input
// (sm_103a):  dw[o][i] = gain[i] * sum over t of dy[t][o] * xhat[t][i].
//
// A matrix product over the tokens, bound by the tensor cores.  Both operands
// lie with the tokens as rows, so both are "M-major" / "N-major" for
// tcgen05.mma: rows of 64 elements (128 bytes), one per token, in the 128-byte
// swizzle.  Pairs of CTAs (cta_group::2) compute tiles of 256 inputs x 256
// outputs: a CTA holds 128 of the inputs (the rows of its half of the
// accumulator) and 128 of the outputs.
//   - dy goes from global memory to shared memory by TMA;
//   - the checkpoint's bytes go through registers: eight warps load 16
//     elements of a token at a time, turn them into 16-bit values (exact: a
//     whole number of 7 bits and sign times a power of two) and store them
//     where the tensor cores read them.  The 16-bit matrix that a separate
//     unpack would write and read back never exists;
//   - one thread of the pair issues the products; four warps of each CTA drain
//     finished accumulators (two of 256 columns in tensor memory) while the
//     next tile is summed.
// Tiles that would leave pairs idle in the last wave are cut along the tokens
// into `splits` parts each, whose fp32 sums a second launch adds in order.
//
// Every wait is bounded.  One that runs out (it never does in a healthy run)
// ends the kernel's loops and the tiles not finished become NaN, so that the
// optimizer step skips the gradient.
#include <cuda.h>

#include <mutex>

#include "zero_train_device.cuh"

namespace zero {
namespace {

constexpr int kPairs = 76;         // CTA pairs of one wave: 152 SMs
constexpr int kTileI = 256;        // inputs of a pair's tile, 128 a CTA
constexpr int kTileO = 256;        // outputs of a pair's tile
constexpr int kStepT = 64;         // tokens of a stage
constexpr int kStages = 6;
constexpr int kHalf = 128;         // inputs, and outputs, that one CTA loads
constexpr int kOperandBytes = kHalf * kStepT * 2;            // 16 KB
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kGroupBytes = 64 * kStepT * 2;                 // 64 elements of every token
constexpr int kBarriers = 3 * kStages + 4;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kBarriers * 8 + 16;
static_assert(kSmemBytes <= 227 * 1024, "stages exceed shared memory");
constexpr int kTmemCols = 512;     // two accumulators of 256 fp32 columns

constexpr int kConvertWarps = 8;
constexpr int kEpilogueWarps = 4;
// warp 0: copies; warp 1: products; warps 2..9: conversion; warps 10..13: epilogue
constexpr int kFirstEpilogueWarp = 2 + kConvertWarps;
constexpr int kThreads = 32 * (2 + kConvertWarps + kEpilogueWarps);
constexpr int kAhead = 3;          // stages a converting thread loads ahead, in registers

constexpr uint64_t kWaitNs = 4ull * 1000 * 1000 * 1000;

// -- the schedule ---------------------------------------------------------------------

// Tiles 0..full-1 are summed over all tokens by one pair each; each later
// tile is cut along the tokens into `splits` units, whose sums go to the
// workspace.  Unit u is taken by pair u mod kPairs.
struct Plan {
    uint32_t tiles_i, tiles_o;
    uint32_t steps;      // token steps of a whole tile
    uint32_t full;
    uint32_t splits;
    uint32_t units;      // full + (tiles - full) * splits
};

struct Unit {
    uint32_t ti, to;     // tile
    uint32_t k0, k1;     // token steps
    int32_t part;        // index of its fp32 part, or -1
};

// Tiles in the order that keeps concurrent ones close: bands of 8 input tiles,
// output by output, so that a wave reads few distinct rows of either operand.
constexpr uint32_t kBand = 8;
__host__ __device__ inline void tile_at(const Plan& p, uint32_t tile, uint32_t& ti, uint32_t& to)
{
    const uint32_t band = tile / (kBand * p.tiles_o);
    const uint32_t rest = tile - band * kBand * p.tiles_o;
    const uint32_t left = p.tiles_i - band * kBand;
    const uint32_t height = left < kBand ? left : kBand;
    to = rest / height;
    ti = band * kBand + rest % height;
}

__host__ __device__ inline Unit unit_at(const Plan& p, uint32_t u)
{
    Unit r;
    r.k0 = 0;
    r.k1 = p.steps;
    r.part = -1;
    uint32_t tile = u;
    if (u >= p.full) {
        const uint32_t v = u - p.full;
        tile = p.full + v / p.splits;
        if (p.splits > 1) {
            const uint32_t s = v % p.splits;
            r.k0 = (uint32_t)((uint64_t)p.steps * s / p.splits);
            r.k1 = (uint32_t)((uint64_t)p.steps * (s + 1) / p.splits);
            r.part = (int32_t)v;
        }
    }
    tile_at(p, tile, r.ti, r.to);
    return r;
}

// Parts of the last wave's tiles.  In units of one token step of a pair: a
// unit costs its steps and about kUnitCost more to start and drain, and
// cutting adds the second launch, kJoinCost.
constexpr uint32_t kMaxSplits = 32;
constexpr uint32_t kUnitCost = 8;
constexpr uint32_t kJoinCost = 16;

bool make_plan(uint64_t tokens, uint64_t outs, uint64_t ins, Plan* p)
{
    const uint64_t ti = (ins + kTileI - 1) / kTileI, to = (outs + kTileO - 1) / kTileO;
    const uint64_t steps = (tokens + kStepT - 1) / kStepT;
    if (ti > (1u << 20) || to > (1u << 20) || ti * to > (1u << 28) || steps > (1u << 24))
        return false;
    const uint32_t tiles = (uint32_t)(ti * to);
    p->tiles_i = (uint32_t)ti;
    p->tiles_o = (uint32_t)to;
    p->steps = (uint32_t)steps;
    p->full = tiles / kPairs * kPairs;
    const uint32_t rest = tiles - p->full;
    p->splits = 1;
    uint64_t best = UINT64_MAX;
    for (uint32_t s = 1; rest && s <= kMaxSplits && s <= (steps ? steps : 1); ++s) {
        const uint64_t waves = ((uint64_t)rest * s + kPairs - 1) / kPairs;
        const uint64_t cost = waves * ((steps + s - 1) / s + kUnitCost) + (s > 1 ? kJoinCost : 0);
        if (cost < best) {
            best = cost;
            p->splits = s;
        }
    }
    p->units = p->full + rest * p->splits;
    return true;
}

uint64_t plan_workspace(const Plan& p)
{
    return p.splits > 1 ? (uint64_t)(p.units - p.full) * kTileI * kTileO * sizeof(float) : 0;
}

// -- PTX ------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}

// The address, in the cluster's shared window, of `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_shared(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}

// Waits for the phase of parity `parity`; false if that took over kWaitNs or
// another wait of this CTA has run out (`failed`, shared memory).
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile uint32_t* failed)
{
    if (try_wait_cluster(bar, parity))
        return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (try_wait_cluster(bar, parity))
            return true;
        if ((i & 63) == 63 && (*failed || global_ns() - t0 > kWaitNs))
            break;
    }
    *failed = 1;
    return false;
}

// A 64 x 64 box of a 16-bit matrix into this CTA's shared memory at dst; its
// bytes count on barrier `bar` (cluster address) of the pair's first CTA.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// Shared-memory matrix descriptor of an operand whose rows (one per token)
// hold 64 elements in the 128-byte swizzle: 8 rows are 1024 bytes apart
// (stride), the next 64 elements kGroupBytes (leading).
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(kGroupBytes >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// Instruction descriptor: fp32 accumulator, both operands of type DT and
// transposed (tokens as rows), M = 256, N = 256.
template <int DT>
__device__ constexpr uint32_t instr_desc()
{
    constexpr uint32_t t = DT == ZERO_BF16 ? 1 : 0;
    return 1u << 4 | t << 7 | t << 10 | 1u << 15 | 1u << 16 | (kTileO / 8) << 17 | (kTileI / 16) << 24;
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
                 : "memory");
}

// Arrives on barrier `bar` of both CTAs when the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                 ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// -- conversion ---------------------------------------------------------------------

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
// binary16 holds it for s in [103, 142]; others take convert4_wide.
template <int DT>
__device__ __forceinline__ uint32_t step2(uint32_t s)
{
    if (DT == ZERO_BF16) {
        const uint32_t h = s == kAct8Bad ? 0x7FC0u : (s ? s << 7 : 0x0040u);
        return h * 0x10001u;
    }
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

struct WgradArgs {
    const int8_t* q;
    const uint8_t* scale;
    const uint16_t* gain;
    uint16_t* dw;
    float* parts;
    uint64_t q_pitch, scale_pitch, dw_pitch;
    uint64_t tokens, outs, ins;
    uint32_t add;
    Plan plan;
};

// 16 elements of one token on their way through registers.
struct Chunk {
    uint4 q;
    uint32_t s;
};

__device__ __forceinline__ Chunk load_chunk(const WgradArgs& a, uint64_t t, uint64_t c)
{
    Chunk k;
    k.q = make_uint4(0, 0, 0, 0);
    k.s = 127;
    if (t < a.tokens && c < a.ins) {
        const int8_t* p = a.q + t * a.q_pitch + c;
        if (c + 16 <= a.ins) {
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(k.q.x), "=r"(k.q.y), "=r"(k.q.z), "=r"(k.q.w)
                         : "l"(p));
        } else {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c + i < a.ins)
                    w[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
            k.q = make_uint4(w[0], w[1], w[2], w[3]);
        }
        k.s = a.scale[t * a.scale_pitch + c / ZERO_ACT8_BLOCK];
    }
    return k;
}

template <int DT>
__device__ __forceinline__ void convert_chunk(const Chunk& k, uint4& lo, uint4& hi)
{
    if (DT == ZERO_F16 && (k.s < 103 || (k.s > 142 && k.s != kAct8Bad))) {
        const uint2 x = convert4_wide(k.q.x, k.s), y = convert4_wide(k.q.y, k.s);
        const uint2 z = convert4_wide(k.q.z, k.s), w = convert4_wide(k.q.w, k.s);
        lo = make_uint4(x.x, x.y, y.x, y.y);
        hi = make_uint4(z.x, z.y, w.x, w.y);
        return;
    }
    const uint32_t step = step2<DT>(k.s);
    convert4<DT>(k.q.x, step, lo.x, lo.y);
    convert4<DT>(k.q.y, step, lo.z, lo.w);
    convert4<DT>(k.q.z, step, hi.x, hi.y);
    convert4<DT>(k.q.w, step, hi.z, hi.w);
}

__device__ __forceinline__ void store_shared16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// Where a converting thread is in the pair's sequence of token steps.
struct Cursor {
    uint32_t u, k, k1;
    uint64_t c;         // its first input
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    k_weight_grad(const __grid_constant__ CUtensorMap dy, const __grid_constant__ WgradArgs a)
{
    extern __shared__ unsigned char raw[];
    pdl_entry();
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t bars = base + kStages * kStageBytes;
    const uint32_t full_x = bars, full_y = bars + 8 * kStages, empty = bars + 16 * kStages;
    const uint32_t tmem_full = bars + 24 * kStages, tmem_empty = tmem_full + 16;
    uint32_t* words = reinterpret_cast<uint32_t*>(raw + (bars + 8 * kBarriers - smem_u32(raw)));
    volatile uint32_t* failed = words + 1;
    const uint32_t rank = cluster_rank();
    const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        *failed = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_x + 8 * s, 2 * kConvertWarps);
            mbar_init(full_y + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tmem_full + 8 * b, 1);
            mbar_init(tmem_empty + 8 * b, 2 * kEpilogueWarps);
        }
        mbar_fence_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(words)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(words);

    if (warp == 0) {
        if (lane == 0) {   // copies of dy
            uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
            bool ok = true;
            for (uint32_t u = pair; u < a.plan.units && ok; u += pairs) {
                const Unit t = unit_at(a.plan, u);
                const int x = (int)(t.to * kTileO + rank * kHalf);
                for (uint32_t k = t.k0; k < t.k1; ++k) {
                    if (!wait_phase(empty + 8 * stage, phase ^ 1, failed)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0)
                        mbar_arrive_expect_tx(full_y + 8 * stage, 2 * kOperandBytes);
                    const uint32_t bar = map_shared(full_y + 8 * stage, 0);
                    const uint32_t dst = base + stage * kStageBytes + kOperandBytes;
                    tma_box(dst, &dy, x, (int)(k * kStepT), bar);
                    tma_box(dst + kGroupBytes, &dy, x + 64, (int)(k * kStepT), bar);
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | phase << stage;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // The pair does not end under its own copies: both CTAs' bytes count on
            // the first one's barriers, and the other waits for it below.
            if (rank == 0)
                for (uint32_t s = 0; s < kStages; ++s)
                    if (armed >> s & 1)
                        mbar_wait(full_y + 8 * s, armed_phase >> s & 1, kWaitNs);
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {   // products
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            for (uint32_t u = pair; u < a.plan.units && ok; u += pairs) {
                const Unit t = unit_at(a.plan, u);
                ok = wait_phase(tmem_empty + 8 * buf, buf_phase ^ 1, failed);
                if (!ok)
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t acc = tmem + buf * kTileO;
                for (uint32_t k = t.k0; k < t.k1; ++k) {
                    ok = wait_phase(full_y + 8 * stage, phase, failed) &&
                         wait_phase(full_x + 8 * stage, phase, failed);
                    if (!ok)
                        break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint64_t xd = operand_desc(base + stage * kStageBytes);
                    const uint64_t yd = operand_desc(base + stage * kStageBytes + kOperandBytes);
#pragma unroll
                    for (int j = 0; j < kStepT / 16; ++j)   // 16 tokens: 2048 bytes further
                        mma_pair(acc, xd + j * (2048 >> 4), yd + j * (2048 >> 4), instr_desc<DT>(),
                                 k > t.k0 || j > 0);
                    commit_pair(empty + 8 * stage);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (!ok)
                    break;
                commit_pair(tmem_full + 8 * buf);
                buf ^= 1;
                buf_phase ^= buf == 0;
            }
        }
    } else if (warp < kFirstEpilogueWarp) {
        // conversion: this thread's 16 inputs of tokens tok and tok + 32 of every step.
        // Lanes 0..3 and 4..7 store tokens of different parity, whose swizzles
        // keep the eight 16-byte stores of a quarter warp on different banks.
        const uint32_t w = warp - 2, group = w / 4;
        const uint32_t tok = (w % 4) * 8 + lane / 4;
        const uint32_t col = group * 64 + (lane % 4) * 16;
        const uint32_t row = group * kGroupBytes + tok * 128;
        const uint32_t c0 = ((lane % 4) * 2 ^ (tok & 7)) * 16, c1 = ((lane % 4) * 2 + 1 ^ (tok & 7)) * 16;
        uint32_t total = 0;
        for (uint32_t u = pair; u < a.plan.units; u += pairs) {
            const Unit t = unit_at(a.plan, u);
            total += t.k1 - t.k0;
        }
        Cursor at;
        at.u = pair;
        at.k = at.k1 = 0;
        at.c = 0;
        Chunk ahead[kAhead][2];
        auto fetch = [&](Chunk (&k)[2]) {
            if (at.k == at.k1) {
                const Unit t = unit_at(a.plan, at.u);
                at.k = t.k0;
                at.k1 = t.k1;
                at.c = (uint64_t)t.ti * kTileI + rank * kHalf + col;
                at.u += pairs;
            }
            const uint64_t t = (uint64_t)at.k * kStepT + tok;
            k[0] = load_chunk(a, t, at.c);
            k[1] = load_chunk(a, t + 32, at.c);
            ++at.k;
        };
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (j < total)
                fetch(ahead[j]);
        uint32_t stage = 0, phase = 0;
        bool ok = true;   // the same in the whole warp
        for (uint32_t n0 = 0; n0 < total && ok; n0 += kAhead)
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const uint32_t n = n0 + j;
                if (n >= total || !ok)
                    break;
                uint4 v[4];
                convert_chunk<DT>(ahead[j][0], v[0], v[1]);
                convert_chunk<DT>(ahead[j][1], v[2], v[3]);
                if (n + kAhead < total)
                    fetch(ahead[j]);
                ok = __all_sync(0xFFFFFFFFu, wait_phase(empty + 8 * stage, phase ^ 1, failed));
                if (!ok)
                    break;
                const uint32_t dst = base + stage * kStageBytes + row;
                store_shared16(dst + c0, v[0]);
                store_shared16(dst + c1, v[1]);
                store_shared16(dst + 32 * 128 + c0, v[2]);
                store_shared16(dst + 32 * 128 + c1, v[3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    arrive_cluster(map_shared(full_x + 8 * stage, 0));
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
    } else {
        // epilogue: warp w of the CTA may read the tensor memory lanes 32 (w mod 4) .. + 31;
        // a lane is an input, a column an output
        const uint32_t quarter = warp % 4;
        uint32_t buf = 0, buf_phase = 0;
        for (uint32_t u = pair; u < a.plan.units; u += pairs) {
            const Unit t = unit_at(a.plan, u);
            const bool ok = __all_sync(0xFFFFFFFFu, wait_phase(tmem_full + 8 * buf, buf_phase, failed));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t r = rank * kHalf + quarter * 32 + lane;
            const uint64_t i = (uint64_t)t.ti * kTileI + r;
            const uint64_t o0 = (uint64_t)t.to * kTileO;
            const float gain = a.gain && i < a.ins ? widen1<DT>(a.gain[i]) : 1.0f;
            for (uint32_t c = 0; c < kTileO; c += 32) {
                uint32_t v[32];
                tmem_load32(tmem + buf * kTileO + c + (quarter * 32 << 16), v);
                if (!ok)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        v[j] = 0x7FC00000u;
                if (t.part >= 0) {
                    float* p = a.parts + ((uint64_t)t.part * kTileO + c) * kTileI + r;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        p[(uint32_t)j * kTileI] = __uint_as_float(v[j]);
                } else if (i < a.ins) {
                    uint16_t* p = a.dw + (o0 + c) * a.dw_pitch + i;
                    const uint32_t n = o0 + c < a.outs ? (uint32_t)min((uint64_t)32, a.outs - o0 - c) : 0;
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j < n) {
                            float x = __uint_as_float(v[j]) * gain;
                            if (a.add)
                                x += widen1<DT>(p[j * a.dw_pitch]);
                            p[j * a.dw_pitch] = narrow1<DT>(x);
                        }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                arrive_cluster(map_shared(tmem_empty + 8 * buf, 0));
            buf ^= 1;
            buf_phase ^= buf == 0;
        }
    }
    __syncwarp();
    __syncthreads();
    cluster_sync();   // no CTA ends, or frees tensor memory, while its pair may still use it
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

// Adds the parts of the cut tiles in order, 8 inputs a thread.
constexpr int kJoinThreads = 256;
constexpr int kJoinCtas = kTileI * kTileO / 8 / kJoinThreads;   // of one tile
template <int DT, bool VEC>
__global__ void __launch_bounds__(kJoinThreads) k_weight_join(const WgradArgs a)
{
    pdl_entry();
    const uint32_t tile = blockIdx.x / kJoinCtas;
    const uint32_t e = (blockIdx.x % kJoinCtas * kJoinThreads + threadIdx.x) * 8;
    uint32_t ti, to;
    tile_at(a.plan, a.plan.full + tile, ti, to);
    const uint64_t o = (uint64_t)to * kTileO + e / kTileI, i = (uint64_t)ti * kTileI + e % kTileI;
    if (o >= a.outs || i >= a.ins)
        return;
    const float* p = a.parts + (uint64_t)tile * a.plan.splits * (kTileI * kTileO) + e;
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (uint32_t s = 0; s < a.plan.splits; ++s) {
        const float4 lo = *reinterpret_cast<const float4*>(p + (uint64_t)s * (kTileI * kTileO));
        const float4 hi = *reinterpret_cast<const float4*>(p + (uint64_t)s * (kTileI * kTileO) + 4);
        x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
        x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
    }
    if (a.gain)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + k < a.ins)
                x[k] *= widen1<DT>(a.gain[i + k]);
    uint16_t* row = a.dw + o * a.dw_pitch;
    if (a.add)
        add8<DT>(x, load8<VEC>(row, i, a.ins));
    store8_row<VEC>(row, i, a.ins, narrow8<DT>(x));
}

// dw without any token: zero.
__global__ void __launch_bounds__(256) k_weight_zero(const WgradArgs a)
{
    pdl_entry();
    for (uint64_t o = blockIdx.y; o < a.outs; o += gridDim.y)
        for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < a.ins; i += (uint64_t)gridDim.x * 256)
            a.dw[o * a.dw_pitch + i] = 0;
}

// -- host -------------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, found through the runtime (the library
// links no driver library); null if there is none.
EncodeTiled encode_tiled()
{
    static EncodeTiled fn = nullptr;
    static std::once_flag found;
    std::call_once(found, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(f);
        (void)cudaGetLastError();
    });
    return fn;
}

template <int DT>
cudaError_t launch_products(const CUtensorMap& map, const WgradArgs& a, bool vec, void* stream)
{
    static std::atomic<uint64_t> allowed{0};
    allow_smem(k_weight_grad<DT>, kSmemBytes, allowed);
    const uint32_t pairs = a.plan.units < kPairs ? a.plan.units : kPairs;
    cudaError_t e = launch_train(k_weight_grad<DT>, dim3(2 * pairs), kThreads, kSmemBytes, 1, stream, map, a);
    if (e == cudaSuccess && a.plan.splits > 1) {
        const uint32_t cut = a.plan.tiles_i * a.plan.tiles_o - a.plan.full;
        e = launch_train(vec ? k_weight_join<DT, true> : k_weight_join<DT, false>, dim3(cut * kJoinCtas),
                         kJoinThreads, 0, 1, stream, a);
    }
    return e;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" uint64_t zero_act_weight_grad_workspace(uint64_t tokens, uint64_t outs, uint64_t ins)
{
    Plan p;
    if (!make_plan(tokens, outs, ins, &p))
        return UINT64_MAX;
    return plan_workspace(p);
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
    Plan plan;
    if (!make_plan(dy->rows, dy->cols, x->cols, &plan) || dy->pitch >= (1ull << 38))
        return ZERO_ERR_UNSUPPORTED;
    const uint64_t need = plan_workspace(plan);
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

    WgradArgs a = {};
    a.q = x->q;
    a.scale = x->scale;
    a.gain = static_cast<const uint16_t*>(gain);
    a.dw = static_cast<uint16_t*>(dw->base);
    a.parts = static_cast<float*>(workspace);
    a.q_pitch = x->q_pitch;
    a.scale_pitch = x->scale_pitch;
    a.dw_pitch = dw->pitch;
    a.tokens = dy->rows;
    a.outs = dw->rows;
    a.ins = dw->cols;
    a.add = accumulate;
    a.plan = plan;
    if (!some)
        return train_status(launch_train(k_weight_zero, dim3((unsigned)((a.ins + 255) / 256),
                                         (unsigned)(a.outs < 1024 ? a.outs : 1024)), 256, 0, 1, stream, a));
    const EncodeTiled encode = encode_tiled();
    if (!encode)
        return ZERO_ERR_CUDA;
    CUtensorMap map;
    const bool f16 = dy->dtype == ZERO_F16;
    const cuuint64_t dims[2] = {dy->cols, dy->rows};
    const cuuint64_t strides[1] = {2 * dy->pitch};
    const cuuint32_t box[2] = {64, kStepT}, unit[2] = {1, 1};
    if (encode(&map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dy->base,
               dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return ZERO_ERR_CUDA;
    const bool vec = (uintptr_t)dw->base % 16 == 0 && dw->pitch % 8 == 0;
    return train_status(f16 ? launch_products<ZERO_F16>(map, a, vec, stream)
                            : launch_products<ZERO_BF16>(map, a, vec, stream));
}
