// Embedding lookup with scaling, and its gradient by sorted tokens (sm_103a).
//
// The gradient's row v is the sum of d_out over the tokens numbered v.  The
// tokens are sorted by number, stably (so equal numbers stay in token order),
// and every row of the table is then one contiguous run of the sorted order,
// summed by one CTA's threads with no atomics.  Numbers are far from evenly
// spread: a frequent token takes thousands of rows.  A run is therefore cut
// at the multiples of kRun positions: pieces that fill a whole such cell are
// summed first, each on its own, into fp32 partial rows, and a second launch
// adds the partial rows of a long run, and its two ends, in their order.
#include "zero_train_device.cuh"

namespace zero {
namespace {

constexpr int kThreads = 256;
constexpr int kLookupUnroll = 4;

__device__ __forceinline__ int64_t load_id(const void* ids, uint32_t bytes, uint64_t i)
{
    return bytes == 8 ? static_cast<const int64_t*>(ids)[i]
                      : (int64_t) static_cast<const int32_t*>(ids)[i];
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

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_lookup(const LookupArgs a)
{
    pdl_entry();
    const uint64_t i0 = (uint64_t)blockIdx.x * (kThreads * kLookupUnroll) + threadIdx.x;
    uint4 w[kLookupUnroll];
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
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
    for (int u = 0; u < kLookupUnroll; ++u) {
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
    const uint32_t* keys;   // later passes
    const uint32_t* toks;
    uint32_t* keys_out;
    uint32_t* toks_out;
    uint32_t* counts;       // [digit][tile]
    uint32_t* bad;
    uint32_t n, ntiles, shift, id_bytes, vocab;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i)
{
    if (!a.ids)
        return a.keys[i];
    const int64_t id = load_id(a.ids, a.id_bytes, i);
    return id >= 0 && id < (int64_t)a.vocab ? (uint32_t)id : a.vocab;
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
            atomicAdd(&h[(sort_key(a, i) >> a.shift) & (kDigits - 1)], 1u);
            if (a.ids && a.bad && load_id(a.ids, a.id_bytes, i) >= (int64_t)a.vocab)
                atomicOr(a.bad, 1u);
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kDigits; d += kThreads)
        a.counts[(uint64_t)d * a.ntiles + blockIdx.x] = h[d];
}

// Exclusive sums of `n` counts in place, by one CTA.
constexpr int kScanThreads = 1024;
__global__ void __launch_bounds__(kScanThreads) k_sort_scan(uint32_t* counts, uint32_t n)
{
    __shared__ uint32_t warp_sums[32];
    pdl_entry();
    uint32_t carry = 0;
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (uint32_t i0 = 0; i0 < n; i0 += kScanThreads) {
        const uint32_t i = i0 + threadIdx.x;
        const uint32_t v = i < n ? counts[i] : 0;
        uint32_t s = v;
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
        const uint32_t before = warp ? __shfl_sync(0xFFFFFFFFu, w, warp - 1) : 0;
        const uint32_t total = __shfl_sync(0xFFFFFFFFu, w, 31);
        if (i < n)
            counts[i] = carry + before + s - v;
        carry += total;
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
    uint32_t key[kRounds], rank[kRounds];
    const uint32_t i0 = blockIdx.x * kTile + warp * kPerWarp + lane;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const uint32_t i = i0 + r * 32;
        key[r] = i < a.n ? sort_key(a, i) : 0;
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool in = i0 + r * 32 < a.n;
        const uint32_t d = in ? (key[r] >> a.shift) & (kDigits - 1) : kDigits;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, d);
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
            const uint32_t at = h[warp][(key[r] >> a.shift) & (kDigits - 1)] + rank[r];
            a.keys_out[at] = key[r];
            a.toks_out[at] = a.ids ? i : a.toks[i];
        }
    }
}

// -- sums -----------------------------------------------------------------------------

constexpr int kRun = 32;        // positions of a cell
constexpr int kRowsPerCta = 32; // table rows of one CTA
constexpr int kJoinSlices = kThreads / 32;

struct GradArgs {
    const uint16_t* d_out;
    const uint32_t* keys;   // sorted
    const uint32_t* toks;
    float* parts;           // [cell][slots * 8]
    uint16_t* d_table;
    uint64_t d_out_pitch, table_pitch, dim;
    uint32_t n, vocab, slots, cells;
    uint32_t row_ctas;      // the CTAs before these take cells
    uint32_t add;
    float scale;
};

// The first position in [0, n) whose key is >= key (n if none), by one warp:
// 32 probes a step.
__device__ uint32_t lower_bound_warp(const uint32_t* keys, uint32_t n, uint32_t key)
{
    const uint32_t lane = threadIdx.x % 32;
    uint32_t lo = 0, hi = n;   // the answer is in [lo, hi]
    while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32;
        const uint64_t p = (uint64_t)lo + (uint64_t)lane * step;
        const bool less = p < hi && keys[p] < key;
        const uint32_t count = __popc(__ballot_sync(0xFFFFFFFFu, less));   // a prefix of the lanes
        if (count == 0)
            return lo;
        const uint64_t next = (uint64_t)lo + (uint64_t)count * step;
        lo += (count - 1) * step + 1;
        hi = next < hi ? (uint32_t)next : hi;
    }
    return lo;
}

// Adds the d_out rows of positions [p0, p1) at columns [c, c + 8) onto acc, in
// order; loads run four rows ahead of the additions.
template <int DT>
__device__ __forceinline__ void add_rows(const GradArgs& a, uint32_t p0, uint32_t p1, uint64_t c,
                                         float (&acc)[8])
{
    for (uint32_t p = p0; p < p1; p += 4) {
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (p + u < p1)
                w[u] = load8<true>(a.d_out + (uint64_t)a.toks[p + u] * a.d_out_pitch, c, a.dim);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (p + u < p1)
                add8<DT>(acc, w[u]);
    }
}

template <int DT, bool VEC>
__device__ __forceinline__ void store_row(const GradArgs& a, uint32_t v, uint64_t c,
                                          const float (&acc)[8])
{
    uint16_t* row = a.d_table + (uint64_t)v * a.table_pitch;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = acc[i] * a.scale;
    if (a.add)
        add8<DT>(x, load8<VEC>(row, c, a.dim));
    store8_row<VEC>(row, c, a.dim, narrow8<DT>(x));
}

// The first CTAs sum whole cells of one number into partial rows; the others
// take kRowsPerCta table rows each and finish those whose run holds no whole
// cell.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_rows(const GradArgs a)
{
    __shared__ uint32_t start[kRowsPerCta + 1];
    pdl_entry();
    if (blockIdx.x < a.cells) {
        const uint32_t p = blockIdx.x * kRun;
        if (p + kRun > a.n || a.keys[p] != a.keys[p + kRun - 1] || a.keys[p] >= a.vocab)
            return;
        for (uint32_t s = threadIdx.x; s < a.slots; s += kThreads) {
            float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            add_rows<DT>(a, p, p + kRun, (uint64_t)s * 8, acc);
            float4* part = reinterpret_cast<float4*>(a.parts + ((uint64_t)blockIdx.x * a.slots + s) * 8);
            part[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            part[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        }
        return;
    }
    const uint32_t v0 = (blockIdx.x - a.cells) * kRowsPerCta;
    const uint32_t nv = min((uint32_t)kRowsPerCta, a.vocab - v0);
    if (threadIdx.x < 64) {
        const uint32_t w = threadIdx.x / 32;
        const uint32_t at = lower_bound_warp(a.keys, a.n, w ? v0 + nv : v0);
        if (threadIdx.x % 32 == 0)
            start[w ? nv : 0] = at;
    }
    __syncthreads();
    const uint32_t lo = start[0], hi = start[nv];
    __syncthreads();
    // position p opens the rows after its predecessor's number up to its own
    for (uint32_t p = lo + threadIdx.x; p <= hi; p += kThreads) {
        const uint32_t from = p == lo ? 0 : a.keys[p - 1] - v0 + 1;
        const uint32_t to = p == hi ? nv : a.keys[p] - v0;
        for (uint32_t v = from; v <= to; ++v)
            start[v] = p;
    }
    __syncthreads();
    const uint32_t items = nv * a.slots;
    for (uint32_t i = threadIdx.x; i < items; i += kThreads) {
        const uint32_t v = i / a.slots;
        const uint64_t c = (uint64_t)(i - v * a.slots) * 8;
        const uint32_t s = start[v], e = start[v + 1];
        if (a.add && s == e)
            continue;
        const uint32_t cell = (s + kRun - 1) / kRun * kRun;
        if (cell + kRun <= e)
            continue;   // k_embed_join's
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        add_rows<DT>(a, s, e, c, acc);
        store_row<DT, VEC>(a, v0 + v, c, acc);
    }
}

__device__ __forceinline__ bool whole_cell(const GradArgs& a, uint32_t cell, uint32_t key)
{
    const uint64_t p = (uint64_t)cell * kRun;
    return p + kRun <= a.n && a.keys[p] == key && a.keys[p + kRun - 1] == key;
}

// One CTA per cell and 256 columns; the one whose cell is the first whole one
// of a run joins the run: its head, its whole cells (in 8 slices of
// consecutive cells) and its tail.
template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) k_embed_join(const GradArgs a)
{
    __shared__ float sums[kJoinSlices][32][9];
    __shared__ uint32_t run[2];
    pdl_entry();
    const uint32_t cell = blockIdx.x;
    const uint32_t p = cell * kRun;
    if (p + kRun > a.n)
        return;
    const uint32_t key = a.keys[p];
    if (key >= a.vocab || !whole_cell(a, cell, key) || (cell > 0 && whole_cell(a, cell - 1, key)))
        return;
    if (threadIdx.x < 64) {
        const uint32_t w = threadIdx.x / 32;
        const uint32_t at = lower_bound_warp(a.keys, a.n, key + w);
        if (threadIdx.x % 32 == 0)
            run[w] = at;
    }
    __syncthreads();
    const uint32_t s = run[0], e = run[1];
    const uint32_t ncells = e / kRun - cell;
    const uint32_t lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const uint32_t slot = blockIdx.y * 32 + lane;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot < a.slots) {
        if (slice == 0)
            add_rows<DT>(a, s, p, (uint64_t)slot * 8, acc);
        const uint32_t per = (ncells + kJoinSlices - 1) / kJoinSlices;
        const uint32_t c1 = min(ncells, (slice + 1) * per);
#pragma unroll 4
        for (uint32_t k = slice * per; k < c1; ++k) {
            const float4* part = reinterpret_cast<const float4*>(
                a.parts + ((uint64_t)(cell + k) * a.slots + slot) * 8);
            const float4 x = part[0], y = part[1];
            acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
            acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
        }
        if (slice == kJoinSlices - 1)
            add_rows<DT>(a, (cell + ncells) * kRun, e, (uint64_t)slot * 8, acc);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sums[slice][lane][i] = acc[i];
    __syncthreads();
    if (slice != 0 || slot >= a.slots)
        return;
#pragma unroll
    for (int k = 1; k < kJoinSlices; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc[i] += sums[k][lane][i];
    store_row<DT, VEC>(a, key, (uint64_t)slot * 8, acc);
}

// -- host ------------------------------------------------------------------------------

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

bool vec_rows(const zero_mat_t* m) { return aligned16(m->base) && m->pitch % 8 == 0; }

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

// Offsets of the gradient's workspace, in bytes.
struct GradSpace {
    uint64_t keys[2], toks[2], counts, parts, total;
    uint32_t tiles, cells, slots;
};

GradSpace grad_space(uint64_t tokens, uint64_t dim)
{
    GradSpace g;
    g.tiles = (uint32_t)((tokens + kTile - 1) / kTile);
    g.cells = (uint32_t)(tokens / kRun);
    g.slots = (uint32_t)((dim + 7) / 8);
    uint64_t at = 0;
    for (int i = 0; i < 2; ++i) {
        g.keys[i] = at;
        at += up256(4 * tokens);
        g.toks[i] = at;
        at += up256(4 * tokens);
    }
    g.counts = at;
    at += up256((uint64_t)kDigits * g.tiles * 4);
    g.parts = at;
    at += (uint64_t)g.cells * g.slots * 32;
    g.total = at;
    return g;
}

constexpr uint64_t kMaxIndex = 0x7FFFFFFFull;
// k_embed_join's grid has a row of CTAs per 256 columns.
constexpr uint64_t kMaxGradCols = 65535ull * 256;

template <int DT, bool VEC>
cudaError_t launch_sums(const GradArgs& a, void* stream)
{
    cudaError_t e = launch_train(k_embed_rows<DT, VEC>, dim3(a.cells + a.row_ctas), kThreads, 0, 1,
                                 stream, a);
    if (e == cudaSuccess && a.cells)
        e = launch_train(k_embed_join<DT, VEC>, dim3(a.cells, (a.slots + 31) / 32), kThreads, 0, 1,
                         stream, a);
    return e;
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
        const dim3 grid((unsigned)((a.items + kThreads * kLookupUnroll - 1) / (kThreads * kLookupUnroll)));
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
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + g.keys[0]),
                         reinterpret_cast<uint32_t*>(ws + g.keys[1])};
    uint32_t* toks[2] = {reinterpret_cast<uint32_t*>(ws + g.toks[0]),
                         reinterpret_cast<uint32_t*>(ws + g.toks[1])};
    uint32_t* counts = reinterpret_cast<uint32_t*>(ws + g.counts);
    const uint32_t vocab = (uint32_t)d_table->rows;
    cudaError_t e = cudaSuccess;
    int cur = 0;
    for (uint32_t shift = 0; n && shift < 32 && (shift == 0 || vocab >> shift); shift += kDigitBits) {
        SortArgs s = {};
        s.ids = shift ? nullptr : ids->ids;
        s.keys = keys[cur];
        s.toks = toks[cur];
        if (shift)
            cur ^= 1;
        s.keys_out = keys[cur];
        s.toks_out = toks[cur];
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
        if (e != cudaSuccess)
            return train_status(e);
    }
    GradArgs a = {};
    a.d_out = static_cast<const uint16_t*>(d_out->base);
    a.keys = keys[cur];
    a.toks = toks[cur];
    a.parts = reinterpret_cast<float*>(ws + g.parts);
    a.d_table = static_cast<uint16_t*>(d_table->base);
    a.d_out_pitch = d_out->pitch;
    a.table_pitch = d_table->pitch;
    a.dim = d_table->cols;
    a.n = n;
    a.vocab = vocab;
    a.slots = g.slots;
    a.cells = g.cells;
    a.row_ctas = (uint32_t)(((uint64_t)vocab + kRowsPerCta - 1) / kRowsPerCta);
    a.add = accumulate;
    a.scale = scale;
    const bool vec = vec_rows(d_table);
    if (d_table->dtype == ZERO_F16)
        e = vec ? launch_sums<ZERO_F16, true>(a, stream) : launch_sums<ZERO_F16, false>(a, stream);
    else
        e = vec ? launch_sums<ZERO_BF16, true>(a, stream) : launch_sums<ZERO_BF16, false>(a, stream);
    return train_status(e);
}
