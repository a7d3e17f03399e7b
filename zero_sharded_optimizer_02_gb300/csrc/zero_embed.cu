// Embedding lookup with scaling, and its gradient by sorted tokens (sm_103a).
//
// The gradient's row v is the sum of d_out over the tokens numbered v.  The
// tokens are sorted by number, stably (so equal numbers stay in token order),
// and every row of the table is then one contiguous run of the sorted order.
// Numbers are far from evenly spread: a frequent token takes thousands of rows
// of d_out, so the work is split evenly over the sorted positions, not over the
// table's rows: a thread sums 8 columns of a cell of 16 or 32 positions, run by
// run.
// A run inside one cell is stored at once; one that crosses cells leaves an
// fp32 partial row in each, and a second launch adds those up in their order.
// No atomics: the result does not depend on scheduling.
#include "zero_train_device.cuh"

namespace zero {
namespace {

constexpr int kThreads = 256;
// Vectors of a lookup's thread.  32,768 x 1,600 in 31 us with 2, 34 with 1, 32 with
// 4; of a table whose rows start on any element in 39 with 2, 37 with 1.
template <bool VEC>
constexpr int kLookupUnroll = VEC ? 2 : 1;

__device__ __forceinline__ int64_t load_id(const void* ids, uint32_t bytes, uint64_t i)
{
    return bytes == 8 ? static_cast<const int64_t*>(ids)[i]
                      : (int64_t) static_cast<const int32_t*>(ids)[i];
}

// N token numbers from i on, `stride` apart (-1 past n); the loads are issued
// together, which a branch on their size in between would prevent.
template <int N>
__device__ __forceinline__ void load_ids(const void* ids, uint32_t bytes, uint32_t i, uint32_t stride, uint32_t n,
                                         int64_t (&id)[N])
{
    if (bytes == 8) {
#pragma unroll
        for (int k = 0; k < N; ++k)
            id[k] = i + k * stride < n ? static_cast<const int64_t*>(ids)[i + k * stride] : -1;
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            id[k] = i + k * stride < n ? static_cast<const int32_t*>(ids)[i + k * stride] : -1;
    }
}

// -- lookup ---------------------------------------------------------------------------

struct LookupArgs {
    const uint16_t* table;
    const void* ids;
    uint16_t* out;
    uint32_t* bad;
    uint64_t table_pitch, out_pitch, vocab, dim;
    uint32_t id_bytes;
    uint32_t slots;   // 8-element slots a row
    uint64_t items;   // slots * tokens
    uint64_t token0;
    float scale;
};

// out[t] = scale * table[id]: a thread moves kUnroll vectors of 8 elements,
// a CTA's of neighbouring columns.  Bound by writing: 32,768 x 1,600 in 31 us,
// 105 MB written at 3.4 of the 4.0 TB/s that a memset reaches.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_lookup(const LookupArgs a)
{
    constexpr int kUnroll = kLookupUnroll<VEC>;
    pdl_entry();
    const uint64_t i0 = (uint64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint4 w[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint64_t i = i0 + u * kThreads;
        w[u] = make_uint4(0, 0, 0, 0);
        if (i < a.items) {
            const uint32_t t = (uint32_t)i / a.slots;
            const uint64_t c = (uint64_t)((uint32_t)i - t * a.slots) * 8;
            const int64_t id = load_id(a.ids, a.id_bytes, a.token0 + t);
            if (id >= 0 && (uint64_t)id < a.vocab)
                w[u] = load8<VEC>(a.table + (uint64_t)id * a.table_pitch, c, a.dim);
            else if (id >= 0 && a.bad && c == 0)
                atomicOr(a.bad, 1u);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint64_t i = i0 + u * kThreads;
        if (i < a.items) {
            const uint32_t t = (uint32_t)i / a.slots;
            const uint64_t c = (uint64_t)((uint32_t)i - t * a.slots) * 8;
            float x[8];
            set8<DT>(x, w[u]);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] *= a.scale;
            store8_row<true>(a.out + (a.token0 + t) * a.out_pitch, c, a.dim, narrow8<DT>(x));
        }
    }
}

// -- sort -----------------------------------------------------------------------------

// The lanes whose digit d (of at most BITS bits) equals this lane's, among those
// with `in`.  One ballot a bit: __match_any_sync took ten times as long.
template <int BITS>
__device__ __forceinline__ uint32_t peers_of(uint32_t d, bool in)
{
    uint32_t peers = __ballot_sync(0xFFFFFFFFu, in);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const uint32_t bit = d >> b & 1;
        peers &= __ballot_sync(0xFFFFFFFFu, bit) ^ (bit - 1);
    }
    return peers;
}

// One stable pass of a least-significant-digit radix sort of (number, token)
// pairs is three launches: digit counts of every tile, their exclusive sums
// over (digit, tile), and the move.  Numbers outside the table sort as
// `vocab`, behind every row.
constexpr int kDigitBits = 8;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kTile = 2048;                 // tokens per CTA
constexpr int kWarps = kThreads / 32;
constexpr int kPerWarp = kTile / kWarps;    // consecutive tokens of one warp

struct SortArgs {
    const void* ids;        // first pass: the caller's numbers
    const uint2* in;        // later passes: (number, token) pairs
    uint2* out;
    uint32_t* counts;       // [digit][tile]
    uint32_t* bad;
    uint32_t n, ntiles, shift, id_bytes, vocab;
};

__device__ __forceinline__ uint2 sort_pair(const SortArgs& a, uint32_t i)
{
    if (!a.ids)
        return a.in[i];
    const int64_t id = load_id(a.ids, a.id_bytes, i);
    return make_uint2(id >= 0 && id < (int64_t)a.vocab ? (uint32_t)id : a.vocab, i);
}

__global__ void __launch_bounds__(kThreads) k_sort_count(const SortArgs a)
{
    __shared__ uint32_t h[kDigits];
    pdl_entry();
    for (int d = threadIdx.x; d < kDigits; d += kThreads)
        h[d] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < kTile; j += kThreads) {
        const uint32_t i = blockIdx.x * kTile + j;
        if (i < a.n) {
            atomicAdd(&h[(sort_pair(a, i).x >> a.shift) & (kDigits - 1)], 1u);
            if (a.ids && a.bad && load_id(a.ids, a.id_bytes, i) >= (int64_t)a.vocab)
                atomicOr(a.bad, 1u);
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += kThreads)
        a.counts[(uint64_t)d * a.ntiles + blockIdx.x] = h[d];
}

// Exclusive sums of `n` counts in place, by one CTA, kScanItems a thread at a
// time (the array has room for a multiple of kScanItems).
constexpr int kScanThreads = 1024;
constexpr int kScanItems = 16;
__global__ void __launch_bounds__(kScanThreads) k_sort_scan(uint32_t* counts, uint32_t n)
{
    __shared__ uint32_t warp_sums[32];
    pdl_entry();
    uint32_t carry = 0;
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (uint32_t i0 = 0; i0 < n; i0 += kScanThreads * kScanItems) {
        const uint32_t i = i0 + threadIdx.x * kScanItems;
        uint4 v[kScanItems / 4];
        uint32_t s = 0;
#pragma unroll
        for (int k = 0; k < kScanItems / 4; ++k) {
            v[k] = i + 4 * k < n ? reinterpret_cast<const uint4*>(counts + i)[k] : make_uint4(0, 0, 0, 0);
            s += v[k].x + v[k].y + v[k].z + v[k].w;
        }
        const uint32_t own = s;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= (uint32_t)d)
                s += o;
        }
        if (lane == 31)
            warp_sums[warp] = s;
        __syncthreads();
        uint32_t w = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, w, d);
            if (lane >= (uint32_t)d)
                w += o;
        }
        const uint32_t ahead = __shfl_sync(0xFFFFFFFFu, w, warp ? warp - 1 : 0);
        uint32_t at = carry + (warp ? ahead : 0) + s - own;
        carry += __shfl_sync(0xFFFFFFFFu, w, 31);
#pragma unroll
        for (int k = 0; k < kScanItems / 4; ++k) {
            const uint4 c = v[k];
            v[k] = make_uint4(at, at + c.x, at + c.x + c.y, at + c.x + c.y + c.z);
            at += c.x + c.y + c.z + c.w;
            if (i + 4 * k < n)
                reinterpret_cast<uint4*>(counts + i)[k] = v[k];
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) k_sort_move(const SortArgs a)
{
    __shared__ uint32_t h[kWarps][kDigits];
    pdl_entry();
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int d = lane; d < kDigits; d += 32)
        h[warp][d] = 0;
    __syncwarp();
    constexpr int kRounds = kPerWarp / 32;
    uint2 pair[kRounds];
    uint32_t rank[kRounds];
    const uint32_t i0 = blockIdx.x * kTile + warp * kPerWarp + lane;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t i = i0 + r * 32;
        pair[r] = i < a.n ? sort_pair(a, i) : make_uint2(0, 0);
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool in = i0 + r * 32 < a.n;
        const uint32_t d = (pair[r].x >> a.shift) & (kDigits - 1);
        const uint32_t peers = peers_of<kDigitBits>(d, in);
        const uint32_t before = __popc(peers & ((1u << lane) - 1));
        uint32_t base = 0;
        if (in)
            base = h[warp][d];
        __syncwarp();
        if (in && before == 0)
            h[warp][d] = base + __popc(peers);
        __syncwarp();
        rank[r] = base + before;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += kThreads) {
        uint32_t base = a.counts[(uint64_t)d * a.ntiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = h[w][d];
            h[w][d] = base;
            base += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t i = i0 + r * 32;
        if (i < a.n) {
            a.out[h[warp][(pair[r].x >> a.shift) & (kDigits - 1)] + rank[r]] = pair[r];
        }
    }
}

// Up to kClusterTokens tokens are sorted in one launch, by a cluster of up to 8
// CTAs that keep the pairs in shared memory: CTA r holds positions [r * per, (r + 1)
// * per) of the order so far, a thread I of them.  A pass counts each warp's
// digits, adds the counts up over warps and, through the other CTAs' shared
// memory, over CTAs, and moves every pair to its new place: into the CTA that
// holds it, or in the last pass to global memory.  More tokens take the
// multi-launch passes, and the rows of absent tokens are then written behind the
// sort: 65,537 tokens x 256 added in 40 us (65,536 in 43), stored 59 (43); x 1,600
// added 95 (96), stored 106 (94).
// 65,536 tokens of 50,257 numbers (two passes of 8 bits): 25 us, of which the
// scattered stores to the other CTAs take 5, ranking 8.  Clusters of 16 CTAs, which
// not every part of a GPU can hold, took 5 us less there (1 more up to 16,384
// tokens), and nothing less where the rows of absent tokens are written beside it.
constexpr int kClusterCtas = 8;
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr int kClusterItems = 8;
constexpr uint32_t kClusterTokens = kClusterCtas * kClusterThreads * kClusterItems;
constexpr int kClusterDigitBits = 9;
constexpr int kClusterDigits = 1 << kClusterDigitBits;

struct ClusterSort {
    const void* ids;
    uint2* out;
    uint32_t* bad;
    uint32_t n, id_bytes, vocab, bits, passes;   // bits of a digit
};

constexpr size_t cluster_sort_smem(int items)
{
    return (size_t)kClusterThreads * items * sizeof(uint2) + kClusterWarps * kClusterDigits * sizeof(uint16_t) +
           (2 * kClusterDigits + 32) * sizeof(uint32_t);
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int I>
__global__ void __launch_bounds__(kClusterThreads) k_sort_cluster(const ClusterSort a)
{
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr uint32_t per = kClusterThreads * I;
    uint2* pairs = reinterpret_cast<uint2*>(smem);
    uint16_t* counts = reinterpret_cast<uint16_t*>(smem + per * sizeof(uint2));   // [warp][digit]
    uint32_t* total = reinterpret_cast<uint32_t*>(counts + kClusterWarps * kClusterDigits);
    uint32_t* first = total + kClusterDigits;   // where the CTA's pairs of a digit go
    uint32_t* warp_sums = first + kClusterDigits;
    pdl_entry();
    uint32_t rank_in_cluster, ctas;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_in_cluster));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t at0 = warp * 32 * I + lane;        // this thread's places: at0 + 32 i
    uint2 pair[I];
    bool bad = false;
    int64_t id[I];
    load_ids<I>(a.ids, a.id_bytes, rank_in_cluster * per + at0, 32, a.n, id);
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t t = rank_in_cluster * per + at0 + 32 * i;
        const uint32_t key = id[i] >= 0 && id[i] < (int64_t)a.vocab ? (uint32_t)id[i] : a.vocab;
        pair[i] = make_uint2(t < a.n ? key : 0xFFFFFFFFu, t);
        bad |= id[i] >= (int64_t)a.vocab;
    }
    if (bad && a.bad)
        atomicOr(a.bad, 1u);
    const uint32_t digits = 1u << a.bits, mask = digits - 1;
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t shift = pass * a.bits;
        for (uint32_t d = threadIdx.x; d < kClusterWarps * digits / 2; d += kClusterThreads)
            reinterpret_cast<uint32_t*>(counts)[d] = 0;
        __syncthreads();
        uint16_t* mine = counts + warp * digits;
        uint32_t rank[I];
#pragma unroll
        for (int i = 0; i < I; ++i)   // places past the end have key 0xFFFFFFFF and no count
            rank[i] = peers_of<kClusterDigitBits>(pair[i].x >> shift & mask, pair[i].x != 0xFFFFFFFFu);
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const bool in = pair[i].x != 0xFFFFFFFFu;
            const uint32_t d = pair[i].x >> shift & mask;
            const uint32_t peers = rank[i];
            const uint32_t before = __popc(peers & ((1u << lane) - 1));
            uint32_t base = 0;
            if (in)
                base = mine[d];
            __syncwarp();
            if (in && before == 0)
                mine[d] = (uint16_t)(base + __popc(peers));
            __syncwarp();
            rank[i] = base + before;
        }
        __syncthreads();
        if (threadIdx.x < digits) {   // over the warps
            uint32_t sum = 0;
#pragma unroll
            for (int w = 0; w < kClusterWarps; ++w) {
                const uint32_t c = counts[w * digits + threadIdx.x];
                counts[w * digits + threadIdx.x] = (uint16_t)sum;
                sum += c;
            }
            total[threadIdx.x] = sum;
        }
        cluster_barrier();
        // over the CTAs, then over the digits
        uint32_t lower = 0, all = 0;
        if (threadIdx.x < digits) {
            const uint32_t word = smem_u32(total + threadIdx.x);
#pragma unroll
            for (uint32_t r = 0; r < kClusterCtas; ++r) {
                if (r < ctas) {
                    uint32_t addr, v;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(word), "r"(r));
                    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
                    all += v;
                    lower += r < rank_in_cluster ? v : 0;
                }
            }
        }
        uint32_t sum = all;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= (uint32_t)o)
                sum += v;
        }
        if (lane == 31)
            warp_sums[warp] = sum;
        __syncthreads();
        uint32_t w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, w, o);
            if (lane >= (uint32_t)o)
                w += v;
        }
        const uint32_t ahead = __shfl_sync(0xFFFFFFFFu, w, warp ? warp - 1 : 0);
        if (threadIdx.x < digits)
            first[threadIdx.x] = (warp ? ahead : 0) + sum - all + lower;
        __syncthreads();
        const bool last = pass + 1 == a.passes;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (pair[i].x == 0xFFFFFFFFu)
                continue;
            const uint32_t d = pair[i].x >> shift & mask;
            const uint32_t to = first[d] + mine[d] + rank[i];
            if (last) {
                a.out[to] = pair[i];
            } else {
                uint32_t addr;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(addr)
                             : "r"(smem_u32(pairs + to % per)), "r"(to / per));
                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(pair[i].x), "r"(pair[i].y)
                             : "memory");
            }
        }
        // the pairs are in place, and every CTA has read the others' totals
        cluster_barrier();
        if (!last)
#pragma unroll
            for (int i = 0; i < I; ++i)
                pair[i] = rank_in_cluster * per + at0 + 32 * i < a.n ? pairs[at0 + 32 * i]
                                                                     : make_uint2(0xFFFFFFFFu, 0);
    }
}

template <int I>
cudaError_t launch_cluster_sort(const ClusterSort& a, void* stream)
{
    static std::atomic<uint64_t> allowed{0};
    allow_smem(k_sort_cluster<I>, cluster_sort_smem(I), allowed);
    uint32_t ctas = 1;   // a power of two, as clusters are
    while (ctas < kClusterCtas && ctas * kClusterThreads * I < a.n)
        ctas *= 2;
    return launch_train(k_sort_cluster<I>, dim3(ctas), kClusterThreads, cluster_sort_smem(I), ctas, stream, a);
}

// Up to kCountTokens tokens are sorted by counting: a pair's place is the number
// of pairs before it.  A CTA keeps all numbers in shared memory, a warp counts for
// one token at a time.  Up to there, n^2 comparisons over all SMs take less than
// the radix passes' barriers: 1,021 tokens 3.6 us against 7.0, 2,048 5.0 against
// 9, 4,096 10.3 against 10.5.
constexpr uint32_t kCountTokens = 2048;
constexpr uint32_t kCountCtas = 304;   // two on each of 152 SMs
__global__ void __launch_bounds__(kThreads) k_sort_count_all(const ClusterSort a)
{
    __shared__ __align__(16) uint32_t keys[kCountTokens];
    pdl_entry();
    const uint32_t n4 = (a.n + 3) / 4 * 4;
    bool bad = false;
    for (uint32_t t = threadIdx.x; t < n4; t += kThreads * 4) {
        int64_t id[4];
        load_ids<4>(a.ids, a.id_bytes, t, kThreads, a.n, id);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u = t + k * kThreads;
            if (u < n4)   // past the last token: never before one
                keys[u] = u >= a.n ? 0xFFFFFFFFu
                                   : id[k] >= 0 && id[k] < (int64_t)a.vocab ? (uint32_t)id[k] : a.vocab;
            bad |= id[k] >= (int64_t)a.vocab;
        }
    }
    if (bad && a.bad && blockIdx.x == 0)
        atomicOr(a.bad, 1u);
    __syncthreads();
    const uint32_t lane = threadIdx.x % 32;
    for (uint32_t t = blockIdx.x * kWarps + threadIdx.x / 32; t < a.n; t += gridDim.x * kWarps) {
        const uint32_t key = keys[t];
        uint32_t before = 0;
#pragma unroll 4
        for (uint32_t u = lane * 4; u < n4; u += 128) {   // of equal numbers, earlier tokens come first
            const uint4 k = *reinterpret_cast<const uint4*>(keys + u);
            before += k.x < key + (u < t);
            before += k.y < key + (u + 1 < t);
            before += k.z < key + (u + 2 < t);
            before += k.w < key + (u + 3 < t);
        }
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        if (lane == 0)
            a.out[before] = make_uint2(key, t);
    }
}

// -- rows of absent tokens ------------------------------------------------------------

// Writes zeros to the rows of absent tokens (of a stored gradient) while the sort
// launched before it runs, k_sort_cluster on up to 8 SMs or k_sort_count_all on up
// to 256 CTAs: it starts with it and ends after it (pdl_end), so the sums that
// follow find both done.  It starts only when every CTA of the sort has passed the
// wait for the work before the call (each sort begins with pdl_entry, which waits
// before it lets dependents start), and reads and writes nothing that the sort
// writes.
//
// CTA `me` takes every kZeroCtas-th group of 32 rows, since the rows of absent
// tokens crowd at one end of a vocabulary sorted by frequency and one SM writes
// only about 25 bytes a clock.  It marks its tokens by reading all numbers.
// A thread takes a row (zero_row).  All SMs write at most 4.0 TB/s (a memset of 1 GB), 0.6 of what a copy moves.
constexpr uint32_t kZeroCtas = 128;
constexpr int kZeroThreads = 1024;
constexpr uint32_t kZeroBytes = 8192;
constexpr uint32_t kMarkWords = 8192;   // groups that a CTA marks at a time
static_assert((kZeroCtas & (kZeroCtas - 1)) == 0, "a mask finds a group's CTA");

struct ZeroArgs {
    const void* ids;
    uint16_t* d_table;
    uint64_t table_pitch, dim;
    uint32_t n, id_bytes, vocab;
};

// Zeros for row v, by one thread: what of it is whole 16-byte vectors in memory
// by bulk copies of `zeros` (kZeroBytes of them), the ends by elements.
__device__ void zero_row(uint16_t* d_table, uint64_t pitch, uint64_t dim, uint32_t v, const void* zeros)
{
    uint16_t* row = d_table + (uint64_t)v * pitch;
    const uint64_t head = min((uint64_t)(0 - (reinterpret_cast<uintptr_t>(row) / 2)) % 8, dim);
    const uint64_t body = (dim - head) / 8 * 8;
    for (uint64_t i = 0; i < head; ++i)
        row[i] = 0;
    for (uint64_t i = head + body; i < dim; ++i)
        row[i] = 0;
    char* to = reinterpret_cast<char*>(row + head);
    for (uint64_t b = 0; b < 2 * body; b += kZeroBytes)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to + b),
                     "r"(smem_u32(zeros)), "r"((uint32_t)min((uint64_t)kZeroBytes, 2 * body - b))
                     : "memory");
}

__global__ void __launch_bounds__(kZeroThreads) k_embed_absent(const ZeroArgs a)
{
    __shared__ __align__(16) uint32_t zeros[kZeroBytes / 4];
    __shared__ uint32_t marks[kMarkWords];
    pdl_begin(1);
    const uint32_t me = blockIdx.x;
    for (uint32_t i = threadIdx.x; i < kZeroBytes / 4; i += kZeroThreads)
        zeros[i] = 0;
    fence_proxy_async_smem();
    const uint32_t groups = (a.vocab + 31) / 32;
    const uint32_t mine = me < groups ? (groups - 1 - me) / kZeroCtas + 1 : 0;   // groups of this CTA
    for (uint32_t lo = 0; lo < mine; lo += kMarkWords) {
        const uint32_t n = min(mine - lo, kMarkWords);
        for (uint32_t i = threadIdx.x; i < n; i += kZeroThreads)
            marks[i] = 0;
        __syncthreads();
        constexpr int kBatch = 4;
        for (uint32_t t = threadIdx.x; t < a.n; t += kZeroThreads * kBatch) {
            int64_t id[kBatch];
            load_ids<kBatch>(a.ids, a.id_bytes, t, kZeroThreads, a.n, id);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const uint32_t v = (uint32_t)id[k], word = v / 32 / kZeroCtas - lo;
                if (v / 32 % kZeroCtas == me && id[k] >= 0 && id[k] < (int64_t)a.vocab && word < n)
                    atomicOr(&marks[word], 1u << (v & 31));
            }
        }
        __syncthreads();
        // row 32 ((lo + i) kZeroCtas + me) + bit for word i of the marks
        for (uint32_t r = threadIdx.x; r < n * 32; r += kZeroThreads) {
            const uint32_t v = ((lo + r / 32) * kZeroCtas + me) * 32 + r % 32;
            if (v < a.vocab && !(marks[r / 32] >> (r % 32) & 1))
                zero_row(a.d_table, a.table_pitch, a.dim, v, zeros);
        }
        __syncthreads();
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // the copies read shared memory
    pdl_end(1);
}

// -- sums -----------------------------------------------------------------------------

// How the sums are laid out.
//   kFew   cells of 16 positions, d_out read through L1, two CTAs an SM;
//   kSome  more CTAs of such cells than run at once (kSomeCtas): d_out read past
//          L1, three CTAs an SM;
//   kMany  over kManyTokens tokens: cells of 32 too.
// Smaller cells are more threads and shorter chains of loads, but leave more
// partial rows to write and join.  As few, some and many, us, added:
//   1,021 x 768    11, 12, 16       16,384 x 768    29, 24, 27
//   20,000 x 256   27, 28, 31       20,000 x 1,600  59, 54, 55 (stored)
//   24,000 x 1,600 60, 54, 50       65,536 x 768    76, 68, 61
//   65,536 x 256   47, 46, 43       65,536 x 1,600  134, 112, 101
// Only long batches of narrow rows lose: 24,000 x 256 28, 30, 32.  kSome and kMany
// keep three CTAs an SM by spilling 8 to 48 bytes a thread.
enum Layout { kFew, kSome, kMany };
template <int LAYOUT>
constexpr int kCellOf = LAYOUT == kMany ? 32 : 16;
constexpr int kMaxPairs = 1024;  // positions of one CTA
constexpr uint32_t kSomeCtas = 456;      // three on each of 152 SMs
constexpr uint64_t kManyTokens = 20000;
constexpr int kZeroRows = 128;   // table rows of one CTA that looks for absent tokens
static_assert(kMaxPairs * sizeof(uint2) >= kZeroBytes, "zeros fit where the pairs are");
constexpr int kJoinCells = kThreads / 32;

struct GradArgs {
    const uint16_t* d_out;
    const uint2* pairs;     // (number, token), sorted
    float* parts;           // [cell][2][slots * 8]
    uint16_t* d_table;
    uint64_t d_out_pitch, table_pitch, dim;
    uint32_t n, vocab, slots, cells;
    uint32_t per_cta;       // cells of one CTA
    uint32_t cell_ctas;     // CTAs that take cells; the launch's others take table rows
    float scale;
};

// The first position in [0, n) whose key is >= key (n if none), by one warp:
// 32 probes a step.
__device__ uint32_t lower_bound_warp(const uint2* pairs, uint32_t n, uint32_t key)
{
    const uint32_t lane = threadIdx.x % 32;
    uint32_t lo = 0, hi = n;   // the answer is in [lo, hi]
    while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32;
        const uint64_t p = (uint64_t)lo + (uint64_t)lane * step;
        const bool less = p < hi && pairs[p].x < key;
        const uint32_t count = __popc(__ballot_sync(0xFFFFFFFFu, less));   // a prefix of the lanes
        if (count == 0)
            return lo;
        const uint64_t next = (uint64_t)lo + (uint64_t)count * step;
        lo += (count - 1) * step + 1;
        hi = next < hi ? (uint32_t)next : hi;
    }
    return lo;
}

// Elements [c, c + 8) of the gradient's row, or zeros where not `there`, on their way
// to registers: nothing looks at them before values() (which takes what load()
// did).  VEC: the rows lie on 16-byte boundaries.
template <bool VEC>
struct Row8 {
    Part8 part;

    __device__ __forceinline__ void load(const uint16_t* row, uint64_t c, uint64_t dim, bool there)
    {
        part.load(row + c, there ? part_of8(c, dim) : 0);
    }

    __device__ __forceinline__ uint4 values(const uint16_t* row, uint64_t c, uint64_t dim, bool there) const
    {
        return part.values(row + c, there ? part_of8(c, dim) : 0);
    }
};

template <>
struct Row8<true> {
    uint4 w;

    __device__ __forceinline__ void load(const uint16_t* row, uint64_t c, uint64_t dim, bool there)
    {
        w = make_uint4(0, 0, 0, 0);
        if (there)   // predicated loads would spill: 65,536 x 1,600 added in 106 us, not 101
            w = load8<true>(row, c, dim);
    }

    __device__ __forceinline__ uint4 values(const uint16_t*, uint64_t, uint64_t, bool) const { return w; }
};

// Row v of the gradient at columns [c, c + 8): scale * acc, added onto `old`
// (that row's values) if ADD.
template <int DT, bool VEC, bool ADD>
__device__ __forceinline__ void store_row(const GradArgs& a, uint32_t v, uint64_t c,
                                          const float (&acc)[8], const Row8<VEC>& old)
{
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = acc[i] * a.scale;
    uint16_t* row = a.d_table + (uint64_t)v * a.table_pitch;
    if (ADD)
        add8<DT>(x, old.values(row, c, a.dim, true));
    store8_row<VEC>(row, c, a.dim, narrow8<DT>(x));
}

template <bool VEC, bool ADD>
__device__ __forceinline__ void load_old(const GradArgs& a, uint32_t v, uint64_t c, bool there, Row8<VEC>& old)
{
    if (ADD)
        old.load(a.d_table + (uint64_t)v * a.table_pitch, c, a.dim, there);
}

// Partial rows of a cell: [0] of a run that began before it and ends in it,
// [1] of one that goes on behind it.
__device__ __forceinline__ float* part_of(const GradArgs& a, uint32_t cell, uint32_t which, uint32_t slot)
{
    return a.parts + (((uint64_t)cell * 2 + which) * a.slots + slot) * 8;
}

__device__ __forceinline__ void store_part(float* part, const float (&acc)[8])
{
    reinterpret_cast<float4*>(part)[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4*>(part)[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

__device__ __forceinline__ void add_part(const float* part, float (&acc)[8])
{
    const float4 x = reinterpret_cast<const float4*>(part)[0], y = reinterpret_cast<const float4*>(part)[1];
    acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
    acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
}

// The runs of one cell, at columns [c, c + 8).  pair: the cell's pairs in shared
// memory, with those before and after it around them.  BATCH rows of d_out (and,
// added, the table's rows of the runs that end among them) are loaded ahead.
template <int DT, bool VEC, bool ADD, int LAYOUT>
__device__ __forceinline__ void sum_cell(const GradArgs& a, const uint2* pair, uint32_t cell, uint32_t slot)
{
    constexpr int BATCH = ADD ? 4 : 8, kCell = kCellOf<LAYOUT>;
    const uint64_t c = (uint64_t)slot * 8;
    uint32_t cur = pair[0].x;
    if (cur >= a.vocab)
        return;
    bool before = pair[-1].x == cur;   // the current run began before the cell
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    Row8<VEC> kept;                        // the table's row of the last run
    const bool whole = c + 8 <= a.dim;     // not the ragged end of the rows
    for (int p = 0; p < kCell; p += BATCH) {
        uint4 w[BATCH];
        Row8<VEC> old[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const uint2 at = pair[p + u];
            const uint16_t* from = a.d_out + (uint64_t)at.y * a.d_out_pitch;
            w[u] = load16<LAYOUT != kFew>(from + c, at.x < a.vocab && whole);
            load_old<VEC, ADD>(a, at.x, c, at.x < a.vocab && pair[p + u + 1].x != at.x, old[u]);
        }
        if (!whole) {
            const uint32_t n = part_of8(c, a.dim);
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                w[u] = load_tail8(a.d_out + (uint64_t)pair[p + u].y * a.d_out_pitch + c,
                                  pair[p + u].x < a.vocab ? n : 0);
#pragma unroll
            for (int u = 0; u < BATCH; ++u)
                w[u] = tail8(w[u], n);
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const uint32_t key = pair[p + u].x;
            if (key != cur) {
                if (before)
                    store_part(part_of(a, cell, 0, slot), acc);
                else
                    store_row<DT, VEC, ADD>(a, cur, c, acc, kept);
                before = false;
                cur = key;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = 0.0f;
            }
            if (cur >= a.vocab)
                return;
            add8<DT>(acc, w[u]);
            if (ADD)
                kept = old[u];   // only read if the run ends here
        }
    }
    if (pair[kCell].x == cur)
        store_part(part_of(a, cell, 1, slot), acc);
    else if (before)
        store_part(part_of(a, cell, 0, slot), acc);
    else
        store_row<DT, VEC, ADD>(a, cur, c, acc, kept);
}

// Writes zeros to the rows of absent tokens among kZeroRows rows (a stored
// gradient's, for batches that k_sort_cluster does not sort), as k_embed_absent
// does; here the sorted pairs say which tokens there are.
__device__ void zero_rows(const GradArgs& a, uint32_t v0, void* zeros)
{
    __shared__ uint32_t range[2];
    __shared__ uint32_t present[kZeroRows / 32];
    const uint32_t nv = min((uint32_t)kZeroRows, a.vocab - v0);
    if (threadIdx.x < kZeroRows / 32)
        present[threadIdx.x] = 0;
    for (uint32_t w = threadIdx.x / 32; w < 2; w += blockDim.x / 32) {
        const uint32_t at = lower_bound_warp(a.pairs, a.n, w ? v0 + nv : v0);
        if (threadIdx.x % 32 == 0)
            range[w] = at;
    }
    for (uint32_t i = threadIdx.x; i < kZeroBytes / 16; i += blockDim.x)
        static_cast<uint4*>(zeros)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncthreads();
    for (uint32_t p = range[0] + threadIdx.x; p < range[1]; p += blockDim.x) {
        const uint32_t r = a.pairs[p].x - v0;
        if (p == range[0] || a.pairs[p - 1].x != r + v0)
            atomicOr(&present[r / 32], 1u << (r % 32));
    }
    __syncthreads();
    for (uint32_t r = threadIdx.x; r < nv; r += blockDim.x)
        if (!(present[r / 32] >> (r % 32) & 1))
            zero_row(a.d_table, a.table_pitch, a.dim, v0 + r, zeros);
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // the copies read shared memory
}

// A CTA sums per_cta cells, a thread 8 columns of one (of one after another
// where a row has more columns than the CTA has threads for).  CTAs beyond
// cell_ctas look for absent tokens; the two kinds are dealt alternately, since
// one mostly reads and the other writes.
template <int DT, bool VEC, bool ADD, int LAYOUT>
__global__ void __launch_bounds__(kThreads, LAYOUT == kFew ? 2 : 3) k_embed_cells(const GradArgs a)
{
    constexpr int kCell = kCellOf<LAYOUT>;
    __shared__ __align__(16) uint2 pairs[kMaxPairs + 2];
    pdl_entry();
    const uint32_t total = gridDim.x;
    const uint32_t mine = (uint32_t)((uint64_t)blockIdx.x * a.cell_ctas / total);
    if ((uint32_t)((uint64_t)(blockIdx.x + 1) * a.cell_ctas / total) == mine) {
        zero_rows(a, (blockIdx.x - mine) * kZeroRows, pairs);
        return;
    }
    const uint32_t cell0 = mine * a.per_cta, ncells = min(a.per_cta, a.cells - cell0);
    for (uint32_t i = threadIdx.x; i < ncells * kCell + 2; i += blockDim.x) {
        const int64_t p = (int64_t)cell0 * kCell + i - 1;
        pairs[i] = p >= 0 && p < a.n ? a.pairs[p] : make_uint2(0xFFFFFFFFu, 0);
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < ncells * a.slots; i += blockDim.x) {
        const uint32_t c = i / a.slots;
        sum_cell<DT, VEC, ADD, LAYOUT>(a, pairs + 1 + c * kCell, cell0 + c, i - c * a.slots);
    }
}

// Adds up the runs that cross cells: 15 us at 65,536 tokens x 1,600, bound by the
// latency of its few dependent loads.  A CTA looks at kJoinCells cells and 256
// columns, a warp at one cell: if a run begins in it and goes on behind it, the
// warp adds its partial rows, [1] of every cell but the last and [0] of that.
// A run of over kLongRun cells is left to the whole CTA, an eighth of it a warp.
constexpr uint32_t kLongRun = 8;
template <int DT, bool VEC, bool ADD, int LAYOUT>
__global__ void __launch_bounds__(kThreads) k_embed_join(const GradArgs a)
{
    constexpr int kCell = kCellOf<LAYOUT>;
    __shared__ float sums[kJoinCells][32][9];
    __shared__ uint32_t more[kJoinCells];   // cells behind the first of a long run
    pdl_entry();
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t slot = blockIdx.y * 32 + lane;
    const uint32_t first = blockIdx.x * kJoinCells, cell = first + warp;
    const uint32_t end = (cell + 1) * kCell;   // of the cell
    uint32_t behind = 0;
    if (end < a.n) {
        const uint32_t key = a.pairs[end - 1].x, next = a.pairs[end].x;
        const uint32_t prev = cell ? a.pairs[cell * kCell - 1].x : 0xFFFFFFFFu;
        if (key < a.vocab && next == key && prev != key) {
            behind = 1;
            for (uint32_t c = cell + 1;; c += 32) {   // does the run fill the cell and go on?
                const uint64_t e = ((uint64_t)c + lane + 1) * kCell;
                const uint32_t stops = ~__ballot_sync(0xFFFFFFFFu, e < a.n && a.pairs[e].x == key);
                if (stops) {
                    behind += __ffs(stops) - 1;
                    break;
                }
                behind += 32;
            }
        }
    }
    if (lane == 0)
        more[warp] = behind > kLongRun ? behind : 0;
    if (behind && behind <= kLongRun && slot < a.slots) {
        const uint32_t key = a.pairs[end - 1].x;
        Row8<VEC> old;
        load_old<VEC, ADD>(a, key, (uint64_t)slot * 8, true, old);
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 8
        for (uint32_t k = 0; k < behind; ++k)
            add_part(part_of(a, cell + k, 1, slot), acc);
        add_part(part_of(a, cell + behind, 0, slot), acc);
        store_row<DT, VEC, ADD>(a, key, (uint64_t)slot * 8, acc, old);
    }
    __syncthreads();
    for (uint32_t r = 0; r < kJoinCells; ++r) {
        const uint32_t n = more[r];
        if (n == 0)
            continue;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (slot < a.slots) {
            const uint32_t per = (n + kJoinCells - 1) / kJoinCells;
            const uint32_t k1 = min(n, (warp + 1) * per);
#pragma unroll 8
            for (uint32_t k = warp * per; k < k1; ++k)
                add_part(part_of(a, first + r + k, 1, slot), acc);
            if (warp == kJoinCells - 1)
                add_part(part_of(a, first + r + n, 0, slot), acc);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sums[warp][lane][i] = acc[i];
        __syncthreads();
        if (warp == 0 && slot < a.slots) {
#pragma unroll
            for (int k = 1; k < kJoinCells; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] += sums[k][lane][i];
            const uint32_t key = a.pairs[(first + r + 1) * kCell - 1].x;
            Row8<VEC> old;
            load_old<VEC, ADD>(a, key, (uint64_t)slot * 8, true, old);
            store_row<DT, VEC, ADD>(a, key, (uint64_t)slot * 8, acc, old);
        }
        __syncthreads();
    }
}

// -- host ------------------------------------------------------------------------------

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

bool vec_rows(const zero_mat_t* m) { return aligned16(m->base) && m->pitch % 8 == 0; }

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

// Offsets of the gradient's workspace, in bytes.
struct GradSpace {
    uint64_t pairs[2], counts, parts, total;
    uint32_t tiles, slots;
    Layout layout;
    uint32_t cells;
    uint32_t per_cta;        // cells of one CTA
};

uint32_t cells_per_cta(uint32_t slots, uint32_t cell)
{
    const uint32_t fit = slots && slots < (uint32_t)kThreads ? kThreads / slots : 1;
    return fit < kMaxPairs / cell ? fit : kMaxPairs / cell;
}

GradSpace grad_space(uint64_t tokens, uint64_t dim)
{
    GradSpace g;
    const bool one_launch = tokens <= kClusterTokens;
    g.tiles = one_launch ? 0 : (uint32_t)((tokens + kTile - 1) / kTile);
    g.slots = (uint32_t)((dim + 7) / 8);
    const uint32_t wide = cells_per_cta(g.slots, kCellOf<kSome>) * kCellOf<kSome>;
    g.layout = tokens > kManyTokens ? kMany : (tokens + wide - 1) / wide > kSomeCtas ? kSome : kFew;
    const uint32_t cell = g.layout == kMany ? kCellOf<kMany> : kCellOf<kFew>;
    g.cells = (uint32_t)((tokens + cell - 1) / cell);
    g.per_cta = cells_per_cta(g.slots, cell);
    g.pairs[0] = 0;
    g.pairs[1] = up256(8 * tokens);
    g.counts = g.pairs[1] + (one_launch ? 0 : up256(8 * tokens));
    g.parts = g.counts + up256((uint64_t)kDigits * g.tiles * 4);
    g.total = g.parts + (uint64_t)g.cells * g.slots * 64;
    return g;
}

constexpr uint64_t kMaxIndex = 0x7FFFFFFFull;
// k_embed_join's grid has a row of CTAs per 256 columns.
constexpr uint64_t kMaxGradCols = 65535ull * 256;

template <int DT, bool VEC, bool ADD, int LAYOUT>
cudaError_t launch_sums(const GradArgs& a, uint32_t zero_ctas, void* stream)
{
    const uint32_t work = a.per_cta * a.slots;
    const uint32_t threads = work < kThreads ? (work + 31) / 32 * 32 : kThreads;
    cudaError_t e = cudaSuccess;
    if (a.cell_ctas + zero_ctas)
        e = launch_train(k_embed_cells<DT, VEC, ADD, LAYOUT>, dim3(a.cell_ctas + zero_ctas), threads, 0, 1, stream, a);
    if (e == cudaSuccess && a.cells > 1)
        e = launch_train(k_embed_join<DT, VEC, ADD, LAYOUT>,
                         dim3((a.cells + kJoinCells - 1) / kJoinCells, (a.slots + 31) / 32), kThreads, 0, 1, stream,
                         a);
    return e;
}

template <int DT, bool VEC, bool ADD>
cudaError_t launch_sums(const GradArgs& a, uint32_t zero_ctas, Layout layout, void* stream)
{
    return layout == kFew    ? launch_sums<DT, VEC, ADD, kFew>(a, zero_ctas, stream)
           : layout == kSome ? launch_sums<DT, VEC, ADD, kSome>(a, zero_ctas, stream)
                             : launch_sums<DT, VEC, ADD, kMany>(a, zero_ctas, stream);
}

template <int DT>
cudaError_t launch_sums(const GradArgs& a, uint32_t zero_ctas, bool vec, bool add, Layout layout, void* stream)
{
    if (add)
        return vec ? launch_sums<DT, true, true>(a, zero_ctas, layout, stream)
                   : launch_sums<DT, false, true>(a, zero_ctas, layout, stream);
    return vec ? launch_sums<DT, true, false>(a, zero_ctas, layout, stream)
               : launch_sums<DT, false, false>(a, zero_ctas, layout, stream);
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status_t zero_embed_lookup(const zero_mat_t* table, const zero_ids_t* ids,
                                           float scale, const zero_mat_t* out, uint32_t* d_bad,
                                           void* stream)
{
    zero_status_t st = check_mat(table, false);
    if (st == ZERO_OK)
        st = check_mat(out, true);
    if (st == ZERO_OK)
        st = check_ids(ids);
    if (st != ZERO_OK)
        return st;
    if (out->rows != ids->count || out->cols != table->cols || out->dtype != table->dtype ||
        nonfinite_host(scale))
        return ZERO_ERR_INVALID_ARG;
    if ((uintptr_t)d_bad % 4 != 0)
        return ZERO_ERR_ALIGNMENT;
    if (table->rows > kMaxIndex || table->cols > kMaxIndex)
        return ZERO_ERR_UNSUPPORTED;
    if (ids->count == 0 || table->cols == 0)
        return ZERO_OK;
    const Span outs[2] = {span_of(out), span_of(d_bad, 4)};
    const Span ins[2] = {span_of(table), span_of(ids->ids, ids->count * ids->bytes)};
    if (any_overlap(outs, 2, ins, 2))
        return ZERO_ERR_INVALID_ARG;
    const void* p[4];
    int n = 0;
    const void* all[4] = {table->base, ids->ids, out->base, d_bad};
    for (const void* q : all)
        if (q)
            p[n++] = q;
    st = require_device(p, n);
    if (st != ZERO_OK)
        return st;

    LookupArgs a = {};
    a.table = static_cast<const uint16_t*>(table->base);
    a.ids = ids->ids;
    a.out = static_cast<uint16_t*>(out->base);
    a.bad = d_bad;
    a.table_pitch = table->pitch;
    a.out_pitch = out->pitch;
    a.vocab = table->rows;
    a.dim = table->cols;
    a.id_bytes = ids->bytes;
    a.slots = (uint32_t)((table->cols + 7) / 8);
    a.scale = scale;
    // launches of at most 2^30 slots (or one token), so item numbers fit 32 bits
    const uint64_t step = a.slots > (1u << 30) ? 1 : (1u << 30) / a.slots;
    const bool vec = vec_rows(table), f16 = table->dtype == ZERO_F16;
    cudaError_t e = cudaSuccess;
    for (uint64_t t = 0; t < ids->count && e == cudaSuccess; t += step) {
        a.token0 = t;
        a.items = (ids->count - t < step ? ids->count - t : step) * a.slots;
        const uint32_t per_cta = kThreads * (vec ? kLookupUnroll<true> : kLookupUnroll<false>);
        const dim3 grid((unsigned)((a.items + per_cta - 1) / per_cta));
        if (vec)
            e = launch_train(f16 ? k_embed_lookup<ZERO_F16, true> : k_embed_lookup<ZERO_BF16, true>,
                             grid, kThreads, 0, 1, stream, a);
        else
            e = launch_train(f16 ? k_embed_lookup<ZERO_F16, false> : k_embed_lookup<ZERO_BF16, false>,
                             grid, kThreads, 0, 1, stream, a);
    }
    return train_status(e);
}

extern "C" uint64_t zero_embed_grad_workspace(uint64_t tokens, uint64_t vocab, uint64_t dim)
{
    if (tokens > kMaxIndex || vocab > kMaxIndex || dim > kMaxGradCols)
        return UINT64_MAX;
    return grad_space(tokens, dim).total;
}

extern "C" zero_status_t zero_embed_grad(const zero_mat_t* d_out, const zero_ids_t* ids,
                                         float scale, uint32_t accumulate,
                                         const zero_mat_t* d_table, void* workspace,
                                         uint64_t workspace_bytes, uint32_t* d_bad, void* stream)
{
    zero_status_t st = check_mat(d_out, true);
    if (st == ZERO_OK)
        st = check_mat(d_table, false);
    if (st == ZERO_OK)
        st = check_ids(ids);
    if (st != ZERO_OK)
        return st;
    if (d_out->rows != ids->count || d_out->cols != d_table->cols ||
        d_out->dtype != d_table->dtype || accumulate > 1 || nonfinite_host(scale))
        return ZERO_ERR_INVALID_ARG;
    if ((uintptr_t)d_bad % 4 != 0)
        return ZERO_ERR_ALIGNMENT;
    if (d_table->rows > kMaxIndex || d_table->cols > kMaxGradCols)
        return ZERO_ERR_UNSUPPORTED;
    if (d_table->rows == 0 || d_table->cols == 0)
        return ZERO_OK;
    const uint32_t n = (uint32_t)ids->count;
    const GradSpace g = grad_space(n, d_table->cols);
    if ((uint64_t)g.cells * g.slots / kThreads + d_table->rows / kZeroRows + 2 > kMaxIndex)
        return ZERO_ERR_UNSUPPORTED;   // the grid of k_embed_cells
    if (g.total && (!workspace || workspace_bytes < g.total))
        return ZERO_ERR_INVALID_ARG;
    if (!aligned16(workspace))
        return ZERO_ERR_ALIGNMENT;
    const Span outs[3] = {span_of(d_table), span_of(workspace, g.total), span_of(d_bad, 4)};
    const Span ins[2] = {span_of(d_out), span_of(ids->ids, ids->count * ids->bytes)};
    if (any_overlap(outs, 3, ins, 2))
        return ZERO_ERR_INVALID_ARG;
    const void* p[5];
    int np = 0;
    const void* all[5] = {n ? d_out->base : nullptr, n ? ids->ids : nullptr, d_table->base,
                          g.total ? workspace : nullptr, d_bad};
    for (const void* q : all)
        if (q)
            p[np++] = q;
    st = require_device(p, np);
    if (st != ZERO_OK)
        return st;
    if (n == 0 && accumulate)
        return ZERO_OK;

    char* ws = static_cast<char*>(workspace);
    uint2* pairs[2] = {reinterpret_cast<uint2*>(ws + g.pairs[0]), reinterpret_cast<uint2*>(ws + g.pairs[1])};
    uint32_t* counts = reinterpret_cast<uint32_t*>(ws + g.counts);
    const uint32_t vocab = (uint32_t)d_table->rows;
    const bool vec = vec_rows(d_table);
    cudaError_t e = cudaSuccess;
    int cur = 0;
    if (n && n <= kClusterTokens) {
        uint32_t bits = 1;
        while (bits < 32 && vocab >> bits)
            ++bits;
        ClusterSort c = {};
        c.ids = ids->ids;
        c.out = pairs[0];
        c.bad = d_bad;
        c.n = n;
        c.id_bytes = ids->bytes;
        c.vocab = vocab;
        c.passes = (bits + kClusterDigitBits - 1) / kClusterDigitBits;
        c.bits = (bits + c.passes - 1) / c.passes;
        const uint32_t items = (n + kClusterCtas * kClusterThreads - 1) / (kClusterCtas * kClusterThreads);
        const uint32_t count_ctas = (n + kWarps - 1) / kWarps < kCountCtas ? (n + kWarps - 1) / kWarps : kCountCtas;
        e = n <= kCountTokens
                ? launch_train(k_sort_count_all, dim3(count_ctas), kThreads, 0, 1, stream, c)
            : items <= 1 ? launch_cluster_sort<1>(c, stream)
            : items <= 2 ? launch_cluster_sort<2>(c, stream)
            : items <= 4 ? launch_cluster_sort<4>(c, stream)
                         : launch_cluster_sort<8>(c, stream);
        if (e == cudaSuccess && !accumulate) {
            ZeroArgs z = {};
            z.ids = ids->ids;
            z.d_table = static_cast<uint16_t*>(d_table->base);
            z.table_pitch = d_table->pitch;
            z.dim = d_table->cols;
            z.n = n;
            z.id_bytes = ids->bytes;
            z.vocab = vocab;
            e = launch_train(k_embed_absent, dim3(kZeroCtas), kZeroThreads, 0, 1, stream, z);
        }
    }
    for (uint32_t shift = 0; n > kClusterTokens && e == cudaSuccess && shift < 32 && (shift == 0 || vocab >> shift);
         shift += kDigitBits) {
        SortArgs s = {};
        s.ids = shift ? nullptr : ids->ids;
        s.in = pairs[cur];
        if (shift)
            cur ^= 1;
        s.out = pairs[cur];
        s.counts = counts;
        s.bad = d_bad;
        s.n = n;
        s.ntiles = g.tiles;
        s.shift = shift;
        s.id_bytes = ids->bytes;
        s.vocab = vocab;
        e = launch_train(k_sort_count, dim3(g.tiles), kThreads, 0, 1, stream, s);
        if (e == cudaSuccess)
            e = launch_train(k_sort_scan, dim3(1), kScanThreads, 0, 1, stream, counts,
                             (uint32_t)(kDigits * g.tiles));
        if (e == cudaSuccess)
            e = launch_train(k_sort_move, dim3(g.tiles), kThreads, 0, 1, stream, s);
    }
    if (e != cudaSuccess)
        return train_status(e);
    GradArgs a = {};
    a.d_out = static_cast<const uint16_t*>(d_out->base);
    a.pairs = pairs[cur];
    a.parts = reinterpret_cast<float*>(ws + g.parts);
    a.d_table = static_cast<uint16_t*>(d_table->base);
    a.d_out_pitch = d_out->pitch;
    a.table_pitch = d_table->pitch;
    a.dim = d_table->cols;
    a.n = n;
    a.vocab = vocab;
    a.slots = g.slots;
    a.cells = g.cells;
    a.per_cta = g.per_cta;
    a.cell_ctas = (a.cells + a.per_cta - 1) / a.per_cta;
    a.scale = scale;
    const uint32_t zero_ctas =
        accumulate || (n && n <= kClusterTokens) ? 0 : (uint32_t)(((uint64_t)vocab + kZeroRows - 1) / kZeroRows);
    const bool add = accumulate != 0;
    e = d_table->dtype == ZERO_F16 ? launch_sums<ZERO_F16>(a, zero_ctas, vec, add, g.layout, stream)
                                   : launch_sums<ZERO_BF16>(a, zero_ctas, vec, add, g.layout, stream);
    return train_status(e);
}
