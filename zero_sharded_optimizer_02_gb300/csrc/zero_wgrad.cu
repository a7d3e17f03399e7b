// Weight gradient of a linear layer from an 8-bit checkpoint of its input
// (sm_103a):  dw[o][i] = gain[i] * sum over t of dy[t][o] * xhat[t][i].
//
// A matrix product over the tokens, on the tensor cores.  Both operands lie with
// the tokens as rows, so both are "M-major" / "N-major" for tcgen05.mma: rows of
// 64 elements (128 bytes), one per token, in the 128-byte swizzle.  Pairs of CTAs
// (cta_group::2) compute tiles of 256 inputs x 256 outputs: a CTA holds 128 of
// the inputs (the rows of its half of the accumulator) and 128 of the outputs.
//   - dy goes from global memory to shared memory by TMA;
//   - the checkpoint's bytes go to shared memory by TMA too; two pairs of warps
//     load its scale bytes and leave the steps beside them.  Three groups of four
//     warps take the token steps in turn: each turns 16 elements of a token at a
//     time into 16-bit values (exact: a whole number of 7 bits and sign times a
//     power of two) and stores them where the tensor cores read them.  The 16-bit
//     matrix that a separate unpack would write and read back never exists;
//   - one thread of the pair issues the products; four warps of each CTA drain
//     finished accumulators (two of 256 columns in tensor memory) while the
//     next tile is summed.
// Tiles that would leave pairs idle in the last wave are cut along the tokens
// into `splits` parts each, whose fp32 sums a second launch adds in order.
//
// 16,384 tokens, 4,096 -> 16,384: 1.46 to 1.51 ms, 1.48 PFLOP/s (a library product of
// two 16-bit matrices of that shape 1.09 to 1.20 ms, behind an unpack 1.20); bound by the
// shared-memory pipe (92% busy), which carries the operands to the tensor cores,
// the bytes to the converting warps and their values back.
//
// Every wait is bounded.  One that runs out (it never does in a healthy run)
// ends the kernel's loops and the tiles not finished become NaN, so that the
// optimizer step skips the gradient.  A warp that has given up takes no more part
// in the schedule: it no longer knows the barriers' phases, so it neither waits
// for nor announces another tile, and what waits for it gives up in its turn.
#include <cuda.h>

#include <mutex>

#include "zero_train_device.cuh"

namespace zero {
namespace {

constexpr int kPairs = 76;         // CTA pairs of one wave: 152 SMs
constexpr int kTileI = 256;        // inputs of a pair's tile, 128 a CTA
constexpr int kTileO = 256;        // outputs of a pair's tile
constexpr int kStepT = 64;         // tokens of a stage
constexpr int kStages = 5;         // of both operands
constexpr int kRawStages = 6;      // the checkpoint's bytes
constexpr int kHalf = 128;         // inputs, and outputs, that one CTA loads
constexpr int kOperandBytes = kHalf * kStepT * 2;            // 16 KB
constexpr int kGroupBytes = 64 * kStepT * 2;                 // 64 elements of every token
constexpr int kRawBytes = kHalf * kStepT;                    // 8 KB
constexpr int kScaleBytes = kStepT * 16;                     // the steps of 4 blocks of every token
constexpr int kEpilogueWarps = 4;
constexpr int kTurnRows = 16;                                // outputs of a tile that is turned
constexpr int kTurnPitch = 32 * 2 + 16;                      // bytes of an output's 32 inputs there
constexpr int kTurnBytes = 2 * kTurnRows * kTurnPitch;       // two tiles
constexpr int kYAt = kStages * kOperandBytes;
constexpr int kRawAt = kYAt + kStages * kOperandBytes;
constexpr int kScaleAt = kRawAt + kRawStages * kRawBytes;
constexpr int kTurnAt = kScaleAt + kRawStages * kScaleBytes;
constexpr int kBarrierAt = kTurnAt + kEpilogueWarps * kTurnBytes;
constexpr int kBarriers = 2 * kStages + 2 * kRawStages + 5;
constexpr int kSmemBytes = 1024 + kBarrierAt + kBarriers * 8 + 32;
static_assert(kSmemBytes <= 227 * 1024, "stages exceed shared memory");
constexpr int kScalesAhead = 2;    // own steps whose scale bytes are loaded ahead, in registers
constexpr int kTmemCols = 512;     // two accumulators of 256 fp32 columns

constexpr int kGroups = 3;         // converting groups
constexpr int kGroupWarps = 4;
constexpr int kTurns = 2;          // pairs of warps for the scale bytes

// Warps by role.  Warp w runs on the SM's scheduler w mod 4.  Scheduler 1 has
// the thread that issues the products and none of the converting warps: each
// of its waits goes through the scheduler's queue for shared memory, and took
// about 250 clocks of a step's 512 behind their loads and stores.
enum Role { kRoleProducts, kRoleGrads, kRoleRaw, kRoleScales, kRoleConvert, kRoleEpilogue };
struct Seat {
    Role role;
    uint32_t index;   // among the warps of its role
};
constexpr int kConvertWarps = kGroups * kGroupWarps;
static_assert(kConvertWarps == 12 && kTurns == 2, "seats");
__device__ __forceinline__ Seat seat_of(uint32_t warp)
{
    const uint32_t row = warp / 4, col = warp % 4;
    if (col == 1) {
        switch (row) {
        case 0: return {kRoleProducts, 0};
        case 1: return {kRoleGrads, 0};
        case 2: return {kRoleRaw, 0};
        case 3: return {kRoleEpilogue, 1};
        default: return {kRoleScales, row - 4};
        }
    }
    if (row < 4)
        return {kRoleConvert, row * 3 + (col ? col - 1 : 0)};
    if (row == 4)
        return {kRoleEpilogue, col};
    return {kRoleScales, col ? 3u : 2u};
}
constexpr int kThreads = 32 * 23;

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

// Arrives on a barrier of the pair's other (or this) CTA.  Release at CTA
// scope: what the arrival announces is this CTA's shared and tensor memory as
// the tensor cores see it, which the writer's proxy fence (or tcgen05 fence)
// has ordered already.  A release at cluster scope waits for the whole memory
// system and held every token step to about 1,200 clocks.
__device__ __forceinline__ void arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Waits for the phase of parity `parity`; false if that took over limit_ns or
// another wait of this CTA has run out (`failed`, shared memory).  Waits that
// poll slow down each other and every arrival, and two dozen warps wait in this
// kernel: those whose answer is not urgent sleep NS nanoseconds between tries.
template <int NS>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile uint32_t* failed, uint64_t limit_ns)
{
    constexpr uint32_t kLook = NS ? 64 : 1024;   // tries between two looks at the clock and at `failed`
    uint64_t t0 = 0;
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (NS)
            __nanosleep(NS);
        if (i % kLook == kLook - 1) {
            const uint64_t t = global_ns();
            if (!t0)
                t0 = t;
            if (*failed || t - t0 > limit_ns)
                break;
        }
    }
    *failed = 1;
    return false;
}
constexpr int kNow = 0, kSoon = 64, kLater = 500;   // how long a wait sleeps between tries

// Longest wait for what is still under way when a CTA ends.
constexpr uint64_t kDrainNs = 1000 * 1000 * 1000;

// Before a CTA ends: waits until the copies last issued for each of the `armed`
// stages have landed.  After a wait has run out these barriers may never
// complete (they count conversions too), so one limit holds for all of them: a
// copy takes microseconds.
__device__ __forceinline__ void drain_copies(uint32_t bars, uint32_t stages, uint32_t armed, uint32_t phases)
{
    const uint64_t t0 = global_ns();
    for (uint32_t s = 0; s < stages; ++s)
        if (armed >> s & 1)
            for (uint32_t i = 0; i < (1u << 30) && !mbar_try_wait(bars + 8 * s, phases >> s & 1); ++i)
                if (global_ns() - t0 > kDrainNs)
                    return;
}

// A box of a matrix into this CTA's shared memory at dst; its bytes count on
// this CTA's barrier `bar`.
__device__ __forceinline__ void tma_box_own(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
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

// The same, on this CTA's barrier alone.
__device__ __forceinline__ void commit_own(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
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

struct WgradArgs {
    const int8_t* q;
    const uint8_t* scale;
    const uint16_t* gain;
    uint16_t* dw;
    float* parts;
    uint64_t q_pitch, scale_pitch, dw_pitch;
    uint64_t tokens, outs, ins;
    uint32_t add;
    uint32_t dw_vec;     // dw's rows start on 16-byte boundaries
    uint64_t wait_ns;    // longest wait
    Plan plan;
};

// 16 elements of one token and their step: 32 bytes of 16-bit values.
template <int DT>
__device__ __forceinline__ void convert_chunk(uint4 q, uint32_t step, uint4& lo, uint4& hi)
{
    if (DT == ZERO_F16 && step >> 16 == 0xFFFFu) {
        const uint32_t s = step & 0xFF;
        const uint2 x = convert4_wide(q.x, s), y = convert4_wide(q.y, s);
        const uint2 z = convert4_wide(q.z, s), w = convert4_wide(q.w, s);
        lo = make_uint4(x.x, x.y, y.x, y.y);
        hi = make_uint4(z.x, z.y, w.x, w.y);
        return;
    }
    convert4<DT>(q.x, step, lo.x, lo.y);
    convert4<DT>(q.y, step, lo.z, lo.w);
    convert4<DT>(q.z, step, hi.x, hi.y);
    convert4<DT>(q.w, step, hi.z, hi.w);
}

__device__ __forceinline__ void store_shared16(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint4 load_shared16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t load_shared_half(uint32_t addr, bool there)
{
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.u32 %0, 0;\n\t"
                 "@p ld.shared.u16 %0, [%1];\n\t}"
                 : "=&r"(v)
                 : "r"(addr), "r"((uint32_t)there));
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    k_weight_grad(const __grid_constant__ CUtensorMap dy, const __grid_constant__ CUtensorMap q,
                  const __grid_constant__ WgradArgs a)
{
    extern __shared__ unsigned char raw[];
    pdl_entry();
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    const uint32_t bars = base + kBarrierAt;
    const uint32_t full = bars, empty = full + 8 * kStages;
    const uint32_t raw_full = empty + 8 * kStages, raw_empty = raw_full + 8 * kRawStages;
    const uint32_t tmem_full = raw_empty + 8 * kRawStages, tmem_empty = tmem_full + 16, drained = tmem_empty + 16;
    uint32_t* words = reinterpret_cast<uint32_t*>(raw + (bars + 8 * kBarriers - smem_u32(raw)));
    volatile uint32_t* failed = words + 1;
    const uint32_t rank = cluster_rank();
    const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Seat seat = seat_of(warp);

    if (threadIdx.x == 0) {
        *failed = 0;
        for (int g = 0; g < kGroups; ++g)
            words[2 + g] = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + 8 * s, 2 * kGroupWarps + 1);   // both CTAs' conversions, and dy's bytes
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < kRawStages; ++s) {
            mbar_init(raw_full + 8 * s, 3);
            mbar_init(raw_empty + 8 * s, kGroupWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tmem_full + 8 * b, 1);
            mbar_init(tmem_empty + 8 * b, 2 * kEpilogueWarps);
        }
        mbar_init(drained, 1);
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

    uint32_t total = 0;   // token steps of this pair
    for (uint32_t u = pair; u < a.plan.units; u += pairs) {
        const Unit t = unit_at(a.plan, u);
        total += t.k1 - t.k0;
    }

    if (seat.role == kRoleGrads) {
        if (lane == 0) {   // copies of dy
            uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
            bool ok = true;
            for (uint32_t u = pair; u < a.plan.units && ok; u += pairs) {
                const Unit t = unit_at(a.plan, u);
                const int x = (int)(t.to * kTileO + rank * kHalf);
                for (uint32_t k = t.k0; k < t.k1; ++k) {
                    if (!wait_phase<kSoon>(empty + 8 * stage, phase ^ 1, failed, a.wait_ns)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0)
                        mbar_arrive_expect_tx(full + 8 * stage, 2 * kOperandBytes);
                    const uint32_t bar = map_shared(full + 8 * stage, 0);
                    const uint32_t dst = base + kYAt + stage * kOperandBytes;
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
                drain_copies(full, kStages, armed, armed_phase);
        }
    } else if (seat.role == kRoleProducts) {
        if (lane == 0 && rank == 0) {   // products
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            for (uint32_t u = pair; u < a.plan.units && ok; u += pairs) {
                const Unit t = unit_at(a.plan, u);
                ok = wait_phase<kNow>(tmem_empty + 8 * buf, buf_phase ^ 1, failed, a.wait_ns);
                if (!ok)
                    break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t acc = tmem + buf * kTileO;
                for (uint32_t k = t.k0; k < t.k1; ++k) {
                    ok = wait_phase<kNow>(full + 8 * stage, phase, failed, a.wait_ns);
                    if (!ok)
                        break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint64_t xd = operand_desc(base + stage * kOperandBytes);
                    const uint64_t yd = operand_desc(base + kYAt + stage * kOperandBytes);
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
            // The products still under way write the tensor memory that is freed below, and
            // where a wait has run out the epilogue has not waited for them.
            commit_own(drained);
            mbar_wait(drained, 0, kDrainNs);
        }
    } else if (seat.role == kRoleConvert) {
        // conversion: group g takes steps g, g + kGroups, ...  A thread takes 16 inputs of
        // either half at tokens tok and tok + 32.  Lanes 0..3 and 4..7 of a quarter
        // warp take tokens that differ in bits 0 and 2, whose swizzles keep its
        // 16-byte loads, and its stores, on different banks.
        const uint32_t group = seat.index / kGroupWarps;
        const bool leads = seat.index % kGroupWarps == 0;
        // The step at which the leading warp gave up, plus one; written before that step's
        // barrier.  A mere flag could be seen one step early by a warp that is late behind
        // the barrier before: it would leave, and the others wait for it there for ever.
        volatile uint32_t* stopped = words + 2 + group;
        const uint32_t p = lane / 4, j = lane % 4;
        const uint32_t tok = seat.index % kGroupWarps * 8 + (p / 2 ^ (p & 1) * 5);
        const uint32_t sw = tok & 7;
        const uint32_t from0 = tok * 128 + (j ^ sw) * 16, from1 = tok * 128 + (4 + j ^ sw) * 16;
        const uint32_t to0 = tok * 128 + (2 * j ^ sw) * 16, to1 = tok * 128 + (2 * j + 1 ^ sw) * 16;
        uint32_t stage = group, phase = 0, rstage = group, rphase = 0;
        static_assert(kGroups <= kStages && kGroups <= kRawStages, "a group's first stage");
        for (uint32_t n = group; n < total; n += kGroups) {
            // one warp of the group waits, the others for it
            if (leads && !(wait_phase<kNow>(raw_full + 8 * rstage, rphase, failed, a.wait_ns) &&
                           wait_phase<kNow>(empty + 8 * stage, phase ^ 1, failed, a.wait_ns)))
                *stopped = n + 1;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(32 * kGroupWarps) : "memory");
            if (*stopped == n + 1)
                break;
            const uint32_t src = base + kRawAt + rstage * kRawBytes;
            const uint32_t sc = base + kScaleAt + rstage * kScaleBytes + tok * 16 + j / 2 * 8;
            const uint32_t dst = base + stage * kOperandBytes;
            // Rolled: the loop body then stays in the warp scheduler's instruction
            // cache, which 23 warps in six roles otherwise thrash.
#pragma unroll 1
            for (uint32_t h = 0; h < 2; ++h) {   // tokens tok, tok + 32
                uint32_t s0, s1;
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(s0), "=r"(s1) : "r"(sc + h * 32 * 16));
                const uint4 q0 = load_shared16(src + h * 32 * 128 + from0);
                const uint4 q1 = load_shared16(src + h * 32 * 128 + from1);
                uint4 lo, hi;
                convert_chunk<DT>(q0, s0, lo, hi);
                store_shared16(dst + h * 32 * 128 + to0, lo);
                store_shared16(dst + h * 32 * 128 + to1, hi);
                convert_chunk<DT>(q1, s1, lo, hi);
                store_shared16(dst + kGroupBytes + h * 32 * 128 + to0, lo);
                store_shared16(dst + kGroupBytes + h * 32 * 128 + to1, hi);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                arrive_cluster(map_shared(full + 8 * stage, 0));
                mbar_arrive(raw_empty + 8 * rstage);
            }
            if ((stage += kGroups) >= kStages) {
                stage -= kStages;
                phase ^= 1;
            }
            if ((rstage += kGroups) >= kRawStages) {
                rstage -= kRawStages;
                rphase ^= 1;
            }
        }
    } else if (seat.role == kRoleRaw) {
        if (lane == 0) {   // copies of the checkpoint
            uint32_t stage = 0, phase = 0, armed = 0, armed_phase = 0;
            bool ok = true;
            for (uint32_t u = pair; u < a.plan.units && ok; u += pairs) {
                const Unit t = unit_at(a.plan, u);
                const int x = (int)(t.ti * kTileI + rank * kHalf);
                for (uint32_t k = t.k0; k < t.k1; ++k) {
                    ok = wait_phase<kSoon>(raw_empty + 8 * stage, phase ^ 1, failed, a.wait_ns);
                    if (!ok)
                        break;
                    mbar_arrive_expect_tx(raw_full + 8 * stage, kRawBytes);
                    tma_box_own(base + kRawAt + stage * kRawBytes, &q, x, (int)(k * kStepT),
                                raw_full + 8 * stage);
                    armed |= 1u << stage;
                    armed_phase = (armed_phase & ~(1u << stage)) | phase << stage;
                    if (++stage == kRawStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            drain_copies(raw_full, kRawStages, armed, armed_phase);   // as for dy's
        }
    } else if (seat.role == kRoleScales) {
        // scale bytes: pair g of the warps takes steps g, g + kTurns, ...; lane l of
        // its warp w loads those of token 32 w + l and leaves their steps, in the
        // order of blocks 0, 2, 1, 3 (a converting thread takes two 64 inputs apart),
        // beside the bytes.  Rows of scale bytes need no alignment: a word is cut out
        // of the two aligned words around it.  Those lie in this row and its
        // neighbours, except at the array's first and last row, which are read by
        // bytes.  A lane's phase is the same in all its rows (a multiple of 64 tokens
        // apart).  Blocks that do not exist get any step: their inputs are zero and
        // their sums are not stored.
        const uint32_t half = seat.index % 2, turn = seat.index / 2;
        const uint32_t blocks = (uint32_t)((a.ins + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK);
        const uint32_t shift =
            (uint32_t)((uintptr_t)(a.scale + (half * 32 + lane) * a.scale_pitch) & 3) * 8;
        const uint64_t hop = (uint64_t)kTurns * kStepT * a.scale_pitch;
        uint32_t u = pair, k = 0, k1 = 0, skip = turn;   // the step of the next scale bytes
        uint32_t exist = 0;
        const uint8_t* p = nullptr;
        uint32_t w0[kScalesAhead], w1[kScalesAhead];
        auto fetch = [&](uint32_t& lo, uint32_t& hi) {
            k += skip;
            p += hop;
            skip = kTurns;
            if (k >= k1) {
                do {
                    const Unit r = unit_at(a.plan, u);
                    u += pairs;
                    k = r.k0 + (k - k1);
                    k1 = r.k1;
                    const uint32_t b = (r.ti * kTileI + rank * kHalf) / ZERO_ACT8_BLOCK;
                    exist = b < blocks ? min(4u, blocks - b) : 0;
                    p = a.scale + ((uint64_t)k * kStepT + half * 32 + lane) * a.scale_pitch + b;
                } while (k >= k1);
            }
            const uint64_t t0 = (uint64_t)k * kStepT;   // the step's first token
            if (t0 > 0 && t0 + kStepT < a.tokens && a.scale_pitch >= 8) {
                lo = load_word(p - shift / 8, exist, 0x7F7F7F7Fu);
                hi = load_word(p - shift / 8 + 4, exist && shift, 0x7F7F7F7Fu);
                return;
            }
            const uint64_t t = t0 + half * 32 + lane;
            uint32_t w = 0x7F7F7F7Fu;
            if (t < a.tokens)
                for (uint32_t i = 0; i < exist; ++i)
                    w = (w & ~(0xFFu << (8 * i))) | (uint32_t)p[i] << (8 * i);
            lo = w << shift;
            hi = __funnelshift_l(w, 0, shift);
        };
#pragma unroll
        for (int i = 0; i < kScalesAhead; ++i)
            if (turn + i * kTurns < total)
                fetch(w0[i], w1[i]);
        uint32_t stage = turn, phase = 0;
        static_assert(kTurns <= kRawStages, "a pair's first stage");
        bool ok = true;
        for (uint32_t n0 = turn; n0 < total && ok; n0 += kTurns * kScalesAhead)
#pragma unroll
            for (int i = 0; i < kScalesAhead; ++i) {
                const uint32_t n = n0 + i * kTurns;
                if (n >= total || !ok)
                    break;
                ok = __all_sync(0xFFFFFFFFu, wait_phase<kSoon>(raw_empty + 8 * stage, phase ^ 1, failed, a.wait_ns));
                if (!ok)
                    break;
                const uint32_t w = __funnelshift_r(w0[i], w1[i], shift);
                store_shared16(base + kScaleAt + stage * kScaleBytes + (half * 32 + lane) * 16,
                               make_uint4(step2<DT>(w & 0xFF), step2<DT>(w >> 16 & 0xFF),
                                          step2<DT>(w >> 8 & 0xFF), step2<DT>(w >> 24)));
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(raw_full + 8 * stage);
                if (n + kTurns * kScalesAhead < total)
                    fetch(w0[i], w1[i]);
                if ((stage += kTurns) >= kRawStages) {
                    stage -= kRawStages;
                    phase ^= 1;
                }
            }
    } else {
        // epilogue: warp w of the CTA may read the tensor memory lanes 32 (w mod 4) .. + 31;
        // a lane is an input, a column an output
        const uint32_t quarter = warp % 4;
        // A tile of 32 inputs x kTurnRows outputs is turned in shared memory, so that a
        // row of dw is stored 64 bytes at a time by four lanes.  What it is added to is
        // copied there a tile ahead, the first before the products are done: 1,024 tokens,
        // 4,096 -> 4,096 added in 56 us, 69 where it was loaded when needed.
        const uint32_t turn = base + kTurnAt + quarter * kTurnBytes;
        const uint32_t mine = lane * 2, line = lane / 4 * kTurnPitch + lane % 4 * 16;
        constexpr int kOld = 16, kTurnOld = 8;
        uint32_t buf = 0, buf_phase = 0;
        bool ok = true;   // once false, for every later unit: see the top of the file
        for (uint32_t u = pair; u < a.plan.units; u += pairs) {
            const Unit t = unit_at(a.plan, u);
            const uint32_t r = rank * kHalf + quarter * 32 + lane;
            const uint64_t o0 = (uint64_t)t.to * kTileO;
            const uint32_t outs = o0 < a.outs ? (uint32_t)min((uint64_t)kTileO, a.outs - o0) : 0;
            const uint32_t i = t.ti * kTileI + r;
            uint16_t* dw = a.dw + o0 * a.dw_pitch + (i - lane);   // the warp's corner of the tile
            const bool turned = t.part < 0 && a.dw_vec && (uint64_t)i - lane + 32 <= a.ins;
            const auto fetch_old = [&](uint32_t c) {   // of the tile of outputs c ..
                if (turned && a.add && c < kTileO)
#pragma unroll
                    for (int j = 0; j < kTurnRows; j += 8) {
                        const uint32_t to = turn + c / kTurnRows % 2 * (kTurnBytes / 2) + line + j * kTurnPitch;
                        const uint32_t o = c + j + lane / 4;
                        cp_async16_part(reinterpret_cast<void*>(__cvta_shared_to_generic(to)),
                                        dw + o * a.dw_pitch + lane % 4 * 8, o < outs ? 16 : 0);
                    }
                cp_async_commit();
            };
            fetch_old(0);
            ok = ok && __all_sync(0xFFFFFFFFu, wait_phase<kLater>(tmem_full + 8 * buf, buf_phase, failed, a.wait_ns));
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
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
                } else if (turned) {
#pragma unroll
                    for (int h = 0; h < 32; h += kTurnRows) {
                        fetch_old(c + h + kTurnRows);
                        cp_async_wait<1>();
                        __syncwarp();
                        const uint32_t tile = turn + h / kTurnRows % 2 * (kTurnBytes / 2);
#pragma unroll
                        for (int j = 0; j < kTurnRows; j += kTurnOld) {
                            uint32_t old[kTurnOld];
#pragma unroll
                            for (int k = 0; k < kTurnOld; ++k)
                                old[k] = load_shared_half(tile + mine + (j + k) * kTurnPitch, a.add);
#pragma unroll
                            for (int k = 0; k < kTurnOld; ++k)
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(tile + mine + (j + k) * kTurnPitch),
                                             "h"(narrow1<DT>(__uint_as_float(v[h + j + k]) * gain +
                                                             widen1<DT>((uint16_t)old[k])))
                                             : "memory");
                        }
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < kTurnRows; j += 8)
                            if (c + h + j + lane / 4 < outs)
                                *reinterpret_cast<uint4*>(dw + (c + h + j + lane / 4) * a.dw_pitch + lane % 4 * 8) =
                                    load_shared16(tile + line + j * kTurnPitch);
                        __syncwarp();   // the tile has been read
                    }
                } else if (i < a.ins) {
                    uint16_t* p = dw + c * a.dw_pitch + lane;
                    const uint32_t n = outs > c ? min(32u, outs - c) : 0;
                    // rows of dw that start anywhere: kOld old values in flight.  425 tokens,
                    // 3,742 -> 2,688 added in 40 us; with 8 53, with 32, which spill, 79.
#pragma unroll
                    for (int h = 0; h < 32; h += kOld) {
                        uint32_t old[kOld];
#pragma unroll
                        for (int j = 0; j < kOld; ++j)
                            old[j] = load_half(p + (h + j) * a.dw_pitch, a.add && h + j < n, 0);
#pragma unroll
                        for (int j = 0; j < kOld; ++j)
                            if (h + j < n)
                                p[(h + j) * a.dw_pitch] =
                                    narrow1<DT>(__uint_as_float(v[h + j]) * gain + widen1<DT>((uint16_t)old[j]));
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0 && ok)
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

// Map of a matrix for boxes of box_rows x `box` columns (128 bytes wide) in
// the 128-byte swizzle; what lies outside the matrix reads as zero.
bool encode_rows(EncodeTiled encode, CUtensorMap* map, CUtensorMapDataType type, void* base, uint64_t cols,
                 uint64_t rows, uint64_t pitch_bytes, uint32_t box, uint32_t box_rows)
{
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {pitch_bytes};
    const cuuint32_t boxes[2] = {box, box_rows}, unit[2] = {1, 1};
    return encode(map, type, 2, base, dims, strides, boxes, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of dy and of the checkpoint's bytes, for boxes of so many tokens.
bool encode_operands(EncodeTiled encode, CUtensorMap* ymap, CUtensorMap* qmap, const zero_mat_t* dy, const zero_act8_t* x,
                     uint32_t y_tokens = kStepT, uint32_t q_tokens = kStepT)
{
    return encode_rows(encode, ymap,
                       dy->dtype == ZERO_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       dy->base, dy->cols, dy->rows, 2 * dy->pitch, 64, y_tokens) &&
           encode_rows(encode, qmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, x->q, x->cols, x->rows, x->q_pitch, kHalf, q_tokens);
}

WgradArgs make_args(const zero_act8_t* x, const void* gain, uint32_t accumulate, const zero_mat_t* dw, void* workspace,
                    const Plan& plan)
{
    WgradArgs a = {};
    a.q = x->q;
    a.scale = x->scale;
    a.gain = static_cast<const uint16_t*>(gain);
    a.dw = static_cast<uint16_t*>(dw->base);
    a.parts = static_cast<float*>(workspace);
    a.q_pitch = x->q_pitch;
    a.scale_pitch = x->scale_pitch;
    a.dw_pitch = dw->pitch;
    a.tokens = x->rows;
    a.outs = dw->rows;
    a.ins = dw->cols;
    a.add = accumulate;
    a.dw_vec = (uintptr_t)dw->base % 16 == 0 && dw->pitch % 8 == 0;
    a.wait_ns = kWaitNs;
    a.plan = plan;
    return a;
}

template <int DT>
cudaError_t launch_products(const CUtensorMap& dy, const CUtensorMap& q, const WgradArgs& a, void* stream,
                            uint32_t max_pairs = kPairs)
{
    static std::atomic<uint64_t> allowed{0};
    allow_smem(k_weight_grad<DT>, kSmemBytes, allowed);
    const uint32_t pairs = a.plan.units < max_pairs ? a.plan.units : max_pairs;
    cudaError_t e = launch_train(k_weight_grad<DT>, dim3(2 * pairs), kThreads, kSmemBytes, 1, stream, dy, q, a);
    if (e == cudaSuccess && a.plan.splits > 1) {
        const uint32_t cut = a.plan.tiles_i * a.plan.tiles_o - a.plan.full;
        e = launch_train(a.dw_vec ? k_weight_join<DT, true> : k_weight_join<DT, false>, dim3(cut * kJoinCtas),
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
    if (!make_plan(dy->rows, dy->cols, x->cols, &plan) || dy->pitch >= (1ull << 38) ||
        x->q_pitch >= (1ull << 39))
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

    const WgradArgs a = make_args(x, gain, accumulate, dw, workspace, plan);
    if (!some)
        return train_status(launch_train(k_weight_zero, dim3((unsigned)((a.ins + 255) / 256),
                                         (unsigned)(a.outs < 1024 ? a.outs : 1024)), 256, 0, 1, stream, a));
    const EncodeTiled encode = encode_tiled();
    if (!encode)
        return ZERO_ERR_CUDA;
    CUtensorMap ymap, qmap;
    if (!encode_operands(encode, &ymap, &qmap, dy, x))
        return ZERO_ERR_CUDA;
    return train_status(dy->dtype == ZERO_F16 ? launch_products<ZERO_F16>(ymap, qmap, a, stream)
                                              : launch_products<ZERO_BF16>(ymap, qmap, a, stream));
}
