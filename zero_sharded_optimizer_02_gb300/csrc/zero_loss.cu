// Losses behind the output layer: token log-probabilities, distillation with
// cross-entropy, policy and preference losses (zero_train.h).
//
// Every one of them is the softmax of a row of logits, a few numbers of the row
// that turn the target's log-probability into a loss and a slope, and the row's
// gradient a (p_j - [j is the target]), from which distillation takes a q_j more.
//
// Exponentials are taken to base 2 at x k - c, with k = log2(e) / T and c the row's
// largest x k: one fused multiply-add an element.  Every sum uses the same k and
// names the c that it is relative to, so what k and c were rounded by cancels but
// for a factor 1 + 2^-24 on the distance to the largest logit.  With R the sum over
// all elements but the target, and e the target's own: p = e / (R + e), 1 - p =
// R / (R + e) and log p = -log1p(R / e), which all keep their relative precision
// however near to 1 p is.
#include "zero_train_device.cuh"

namespace zero {
namespace {

constexpr uint32_t kThreads = 512;
constexpr uint32_t kWarps = kThreads / 32;
constexpr uint32_t kNone = 0xFFFFFFFFu;   // no target in the vocabulary
constexpr float kLn2 = 0.69314718f;
constexpr float kLowest = -1e30f;         // c of a sum without finite elements: x k - c is -inf or NaN there too

enum LossOp { kLogp, kSlope, kDistill, kPolicy, kPairs };

struct LossArgs {
    const uint16_t* logits;
    uint16_t* grad;
    uint64_t pitch, grad_pitch;
    uint32_t rows, vocab;
    const void* ids;          // NULL: every row is there, without a target
    const void* starts;       // kLogp: rows outside starts[0], starts[2 pairs] are left out
    const void* top_ids;
    uint32_t id_bytes, start_bytes, top_id_bytes;
    uint32_t pairs;
    float k, k1;              // log2(e) / T, log2(e)
    float temperature;
    float scale;              // of the gradient, 1 / T in it
    // inputs and outputs, one a row
    const float *slope, *old_logp, *ref, *advantage, *weight;
    float *logp, *lse, *loss;
    uint32_t* bad;
    // policy
    float low, high, kl;      // 1 - clip_low, 1 + clip_high
    // distillation
    const uint16_t* top;
    uint64_t top_pitch;
    uint32_t top_n;
    float soft, hard;         // of the loss
    // preference: of which sequence a row is, the slope of each, and the flag
    int32_t* seq;
    float* seq_slope;
    uint32_t* seq_bad;
    float beta, smoothing;
    float* reward;
};

__device__ __forceinline__ int64_t load_id(const void* ids, uint32_t bytes, uint64_t i)
{
    return bytes == 8 ? static_cast<const int64_t*>(ids)[i]
                      : (int64_t) static_cast<const int32_t*>(ids)[i];
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// -- sums of exponentials ---------------------------------------------------------

// r = sum of 2^(x k - c); relative to another c by a factor 2^(c - other).
struct Sum {
    float c, r;
};

__device__ __forceinline__ Sum join(Sum a, Sum b)
{
    const float c = fmaxf(a.c, b.c);
    return Sum{c, a.r * ex2(a.c - c) + b.r * ex2(b.c - c)};
}

// What a row's sums come to: over its elements but the target at k and, where the
// cross-entropy needs another temperature, at k1; and over the teacher's entries,
// w = sum of 2^(t k - c) and wd = the same times (t - x).
struct RowSums {
    Sum s, s1, w;
    float wd;
};

template <bool DUAL, bool TOP>
__device__ __forceinline__ RowSums join(const RowSums& a, const RowSums& b)
{
    RowSums o;
    o.s = join(a.s, b.s);
    if (DUAL)
        o.s1 = join(a.s1, b.s1);
    if (TOP) {
        o.w = join(a.w, b.w);
        // an entry of weight 0 counts as absent; inf * 0 must not come in here
        const float fa = ex2(a.w.c - o.w.c), fb = ex2(b.w.c - o.w.c);
        o.wd = (fa != 0.0f ? a.wd * fa : 0.0f) + (fb != 0.0f ? b.wd * fb : 0.0f);
    }
    return o;
}

template <bool DUAL, bool TOP>
__device__ __forceinline__ RowSums from_lane(const RowSums& a, int xor_lane)
{
    RowSums o;
    o.s.c = __shfl_xor_sync(0xFFFFFFFFu, a.s.c, xor_lane);
    o.s.r = __shfl_xor_sync(0xFFFFFFFFu, a.s.r, xor_lane);
    if (DUAL) {
        o.s1.c = __shfl_xor_sync(0xFFFFFFFFu, a.s1.c, xor_lane);
        o.s1.r = __shfl_xor_sync(0xFFFFFFFFu, a.s1.r, xor_lane);
    }
    if (TOP) {
        o.w.c = __shfl_xor_sync(0xFFFFFFFFu, a.w.c, xor_lane);
        o.w.r = __shfl_xor_sync(0xFFFFFFFFu, a.w.r, xor_lane);
        o.wd = __shfl_xor_sync(0xFFFFFFFFu, a.wd, xor_lane);
    }
    return o;
}

__device__ __forceinline__ RowSums no_sums()
{
    return RowSums{{kLowest, 0.0f}, {kLowest, 0.0f}, {kLowest, 0.0f}, 0.0f};
}

// -- a row's numbers ----------------------------------------------------------------

// What a row has besides its logits.
struct RowIn {
    bool there;       // false: padding, left out
    uint32_t target;  // kNone: none
    float a, b, c, d; // kSlope, kPairs: slope; kPolicy: old, ref, advantage, weight; kDistill: weight
};

template <int OP>
__device__ __forceinline__ RowIn load_row(const LossArgs& a, uint32_t row, bool flags)
{
    RowIn in = {true, kNone, 0.0f, 0.0f, 0.0f, 0.0f};
    if (OP == kLogp && a.starts) {
        in.there = (int64_t)row >= load_id(a.starts, a.start_bytes, 0) &&
                   (int64_t)row < load_id(a.starts, a.start_bytes, 2ull * a.pairs);
        if (!in.there)
            return in;
    }
    if (OP == kPairs) {
        const int32_t s = a.seq[row];
        in.there = s >= 0;
        if (!in.there)
            return in;
        in.a = *a.seq_bad ? __uint_as_float(0x7FC00000u) : a.seq_slope[s];
    }
    if (a.ids) {
        const int64_t id = load_id(a.ids, a.id_bytes, row);
        in.there = id >= 0 && id < (int64_t)a.vocab;
        if (flags && a.bad && id >= (int64_t)a.vocab)
            atomicOr(a.bad, 1u);
        if (!in.there)
            return in;
        in.target = (uint32_t)id;
    }
    if (OP == kSlope)
        in.a = a.slope[row];
    if (OP == kPolicy) {
        in.a = a.old_logp[row];
        in.b = a.ref ? a.ref[row] : 0.0f;
        in.c = a.advantage[row];
        in.d = a.weight ? a.weight[row] : 1.0f;
    }
    if (OP == kDistill)
        in.a = a.weight ? a.weight[row] : 1.0f;
    return in;
}

// The gradient of an element is g 2^(x k - c) + g1 2^(x k1 - c1), of the target
// `at`; entry q of the teacher takes gq 2^(t k - cw) from its own.
struct RowOut {
    float g, c, g1, c1, at, gq, cw;
};

__device__ __forceinline__ float log_prob(float x2, float e, float r)
{
    return r < e ? -log1pf(r / e) : kLn2 * (x2 - log2f(r + e));
}

// exp(d) - d - 1, from its series where the difference would cancel.
__device__ __forceinline__ float exp_minus_line(float d)
{
    if (fabsf(d) < 0.3f)
        return 0.5f * d * d * (1.0f + d / 3 * (1.0f + d / 4 * (1.0f + d / 5 * (1.0f + d / 6 * (1.0f + d / 7)))));
    return expm1f(d) - d;
}

// The row's results from its sums and its target's logit (-inf if it has none);
// writes: this thread stores them.
template <int OP, bool DUAL, bool TOP>
__device__ __forceinline__ RowOut finish(const LossArgs& a, uint32_t row, const RowIn& in, const RowSums& t, float x,
                                         bool writes)
{
    RowOut o = {};
    const float x2 = fmaf(x, a.k, -t.s.c), e = ex2(x2), s = t.s.r + e;
    o.c = t.s.c;
    if (OP == kDistill) {
        const float w = in.a;
        // at T: of the teacher; at 1: of the target.  One sum serves both where T is 1.
        const float soft = TOP && t.w.r != 0.0f ? a.soft : 0.0f;   // NaN counts as present
        const float at_t = soft * a.temperature * (w * a.scale), at_1 = a.hard * (w * a.scale);
        o.cw = t.w.c;
        o.gq = TOP && t.w.r != 0.0f ? at_t / t.w.r : 0.0f;
        float e1 = e, x1 = x2, r1 = t.s.r;
        if (DUAL) {
            x1 = fmaf(x, a.k1, -t.s1.c);
            e1 = ex2(x1);
            r1 = t.s1.r;
            o.c1 = t.s1.c;
            o.g = at_t / s;
            o.g1 = at_1 / (r1 + e1);
        } else {
            o.g = (at_t + at_1) / s;
        }
        o.at = at_t * (e / s) - at_1 * (r1 / (r1 + e1));
        if (writes && a.loss) {
            float loss = 0.0f;
            if (TOP && soft != 0.0f)
                loss = soft * a.temperature * a.temperature *
                       (t.wd / t.w.r / a.temperature + kLn2 * ((t.s.c - t.w.c) + (log2f(s) - log2f(t.w.r))));
            if (a.hard != 0.0f)
                loss -= a.hard * log_prob(x1, e1, r1);
            a.loss[row] = w * loss;
        }
        return o;
    }
    float slope = in.a;
    if (OP == kLogp || OP == kPolicy) {
        const float lp = log_prob(x2, e, t.s.r);
        if (writes && a.logp)
            a.logp[row] = lp;
        if (OP == kLogp && writes && a.lse)
            a.lse[row] = fmaf(t.s.c, kLn2, logf(s));
        if (OP == kPolicy) {
            const float r = expf(lp - in.a), kept = r * in.c, cut = fminf(fmaxf(r, a.low), a.high) * in.c;
            const bool inside = !(kept > cut);   // of a NaN too, which then reaches loss and gradient
            float loss = inside ? -kept : -cut;
            slope = inside ? -kept : 0.0f;
            if (a.kl != 0.0f) {
                const float d = in.b - lp;
                loss = fmaf(a.kl, exp_minus_line(d), loss);
                slope = fmaf(-a.kl, expm1f(d), slope);
            }
            slope *= in.d;
            if (writes && a.loss)
                a.loss[row] = in.d * loss;
        }
    }
    const float g = -(slope * a.scale);
    o.g = g / s;
    o.at = -g * (t.s.r / s);
    return o;
}

// A row that is left out.
template <int OP>
__device__ __forceinline__ void finish_absent(const LossArgs& a, uint32_t row)
{
    if ((OP == kLogp || OP == kPolicy) && a.logp)
        a.logp[row] = 0.0f;
    if (OP == kLogp && a.lse)
        a.lse[row] = 0.0f;
    if ((OP == kDistill || OP == kPolicy) && a.loss)
        a.loss[row] = 0.0f;
}

// -- vectors of logits ----------------------------------------------------------------

template <int DT>
__device__ __forceinline__ float wide1(uint16_t h)
{
    if (DT == ZERO_F16)
        return __half2float(__ushort_as_half(h));
    return __uint_as_float((uint32_t)h << 16);
}

template <int DT>
__device__ __forceinline__ void wide8(uint4 v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (DT == ZERO_F16) {
            __half2 h;
            memcpy(&h, &w[i], sizeof(h));
            const float2 f = __half22float2(h);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// -- a CTA a row ------------------------------------------------------------------------

template <int DT, int OP, bool GRAD, bool DUAL>
__global__ void __launch_bounds__(kThreads) k_loss_rows(const LossArgs a)
{
    constexpr bool TOP = OP == kDistill;
    __shared__ RowSums part[kWarps];
    __shared__ int64_t top_id[ZERO_DISTILL_MAX_TOP];
    __shared__ float top_w[ZERO_DISTILL_MAX_TOP];
    pdl_entry();
    const uint32_t tid = threadIdx.x, vecs = (a.vocab + 7) / 8;
    if (OP == kLogp && a.seq_bad && blockIdx.x == 0 && tid == 0)
        *a.seq_bad = 0;
    for (uint32_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const RowIn in = load_row<OP>(a, row, tid == 0);
        const uint16_t* z = a.logits + row * a.pitch;
        uint16_t* d = GRAD ? a.grad + row * a.grad_pitch : nullptr;
        if (!in.there) {
            if (tid == 0)
                finish_absent<OP>(a, row);
            if (GRAD)
                for (uint32_t v = tid; v < vecs; v += kThreads)
                    store8_row<true>(d, 8ull * v, a.vocab, make_uint4(0, 0, 0, 0));
            continue;
        }
        const uint32_t target = OP == kDistill && a.hard == 0.0f ? kNone : in.target;
        const float x = target != kNone ? wide1<DT>(z[target]) : -INFINITY;
        RowSums t = no_sums();
        uint32_t entry = kNone;
        float entry_x = 0.0f;
        if (TOP && tid < a.top_n) {
            const int64_t id = load_id(a.top_ids, a.top_id_bytes, (uint64_t)row * a.top_n + tid);
            const float q = wide1<DT>(a.top[row * a.top_pitch + tid]);
            if (a.bad && id >= (int64_t)a.vocab)
                atomicOr(a.bad, 1u);
            if (id >= 0 && id < (int64_t)a.vocab && q != -INFINITY) {
                entry = (uint32_t)id;
                entry_x = wide1<DT>(z[id]);
                t.w.c = q * a.k;
                t.w.r = ex2(fmaf(q, a.k, -t.w.c));
                t.wd = t.w.r * (q - entry_x);
            }
            top_id[tid] = entry == kNone ? -1 : id;
            top_w[tid] = q * a.k;
        }
        for (uint32_t v = tid; v < vecs; v += kThreads) {
            float y[8];
            wide8<DT>(load8<true>(z, 8ull * v, a.vocab), y);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (8 * v + i >= a.vocab || 8 * v + i == target)
                    y[i] = -INFINITY;
            float top = y[0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                top = fmaxf(top, y[i]);
            Sum s = {fmaxf(top * a.k, kLowest), 0.0f}, s1 = {fmaxf(top * a.k1, kLowest), 0.0f};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s.r += ex2(fmaf(y[i], a.k, -s.c));
                if (DUAL)
                    s1.r += ex2(fmaf(y[i], a.k1, -s1.c));
            }
            t.s = join(t.s, s);
            if (DUAL)
                t.s1 = join(t.s1, s1);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1)
            t = join<DUAL, TOP>(t, from_lane<DUAL, TOP>(t, m));
        __syncthreads();   // the last row's sums have been read
        if (tid % 32 == 0)
            part[tid / 32] = t;
        __syncthreads();
        t = part[0];
        for (uint32_t w = 1; w < kWarps; ++w)
            t = join<DUAL, TOP>(t, part[w]);
        if (target != kNone) {   // the target's own exponential must not overflow either
            t.s = join(t.s, Sum{fmaxf(x * a.k, kLowest), 0.0f});
            if (DUAL)
                t.s1 = join(t.s1, Sum{fmaxf(x * a.k1, kLowest), 0.0f});
        }
        const RowOut o = finish<OP, DUAL, TOP>(a, row, in, t, x, tid == 0);
        for (uint32_t v = tid; GRAD && v < vecs; v += kThreads) {
            float y[8];
            wide8<DT>(load8<true>(z, 8ull * v, a.vocab), y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float g = o.g * ex2(fmaf(y[i], a.k, -o.c));
                if (DUAL)
                    g = fmaf(o.g1, ex2(fmaf(y[i], a.k1, -o.c1)), g);
                y[i] = 8 * v + i == target ? o.at : g;
            }
            store8_row<true>(d, 8ull * v, a.vocab, narrow8<DT>(y));
        }
        if (GRAD && TOP && a.top_n) {
            __syncthreads();   // the row is written; its teacher's entries go over it
            if (entry != kNone) {
                float q = 0.0f;   // of all entries of this number, in order
                for (uint32_t k = 0; k < a.top_n; ++k)
                    q += top_id[k] == (int64_t)entry ? ex2(top_w[k] - o.cw) : 0.0f;
                float g = o.g * ex2(fmaf(entry_x, a.k, -o.c));
                if (DUAL)
                    g = fmaf(o.g1, ex2(fmaf(entry_x, a.k1, -o.c1)), g);
                if (entry == target)
                    g = o.at;
                d[entry] = (uint16_t)narrow2<DT>(fmaf(-o.gq, q, g), 0.0f);
            }
        }
    }
}

// -- pairs of sequences -------------------------------------------------------------------

constexpr uint32_t kPairThreads = 256;

// A CTA a pair: the sums of its two sequences in 64 bits, its loss and the slope of
// each sequence's log-probabilities.  The CTAs behind them write of which sequence
// each row is.
__global__ void __launch_bounds__(kPairThreads) k_pairs(const LossArgs a)
{
    pdl_entry();
    const uint32_t tid = threadIdx.x;
    if (blockIdx.x >= a.pairs) {
        const uint64_t row = (uint64_t)(blockIdx.x - a.pairs) * kPairThreads + tid;
        if (row >= a.rows)
            return;
        uint32_t lo = 0, hi = 2 * a.pairs + 1;   // the first start behind the row
        while (lo < hi) {
            const uint32_t mid = (lo + hi) / 2;
            if (load_id(a.starts, a.start_bytes, mid) <= (int64_t)row)
                lo = mid + 1;
            else
                hi = mid;
        }
        a.seq[row] = lo == 0 || lo == 2 * a.pairs + 1 ? -1 : (int32_t)(lo - 1);
        return;
    }
    const uint32_t pair = blockIdx.x;
    int64_t at[3];
    for (int i = 0; i < 3; ++i)
        at[i] = load_id(a.starts, a.start_bytes, 2ull * pair + i);
    const bool ok = at[0] >= 0 && at[0] <= at[1] && at[1] <= at[2] && at[2] <= (int64_t)a.rows;
    double sum[2] = {0.0, 0.0};
    if (ok)
        for (int i = 0; i < 2; ++i)
            for (int64_t row = at[i] + tid; row < at[i + 1]; row += kPairThreads) {
                const int64_t id = load_id(a.ids, a.id_bytes, row);
                if (id >= 0 && id < (int64_t)a.vocab)
                    sum[i] += (double)a.logp[row] - (a.ref ? (double)a.ref[row] : 0.0);
            }
    __shared__ double part[2][kPairThreads / 32];
    for (int i = 0; i < 2; ++i) {
        for (int m = 16; m; m >>= 1)
            sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], m);
        if (tid % 32 == 0)
            part[i][tid / 32] = sum[i];
    }
    __syncthreads();
    if (tid != 0)
        return;
    for (int i = 0; i < 2; ++i) {
        sum[i] = 0.0;
        for (uint32_t w = 0; w < kPairThreads / 32; ++w)
            sum[i] += part[i][w];
        if (!ok)
            sum[i] = (double)__uint_as_float(0x7FC00000u);
        if (a.reward)
            a.reward[2 * pair + i] = (float)(a.beta * sum[i]);
    }
    const float m = (float)(a.beta * (sum[0] - sum[1]));
    const float small = log1pf(expf(-fabsf(m)));   // -log sigmoid(|m|)
    const float lose = m < 0.0f ? small - m : small, win = m > 0.0f ? small + m : small;
    a.loss[pair] = (1.0f - a.smoothing) * lose + a.smoothing * (m != m ? m : win);
    // d loss / d m = smoothing sigmoid(m) - (1 - smoothing) sigmoid(-m)
    const float e = expf(-fabsf(m)), high = 1.0f / (1.0f + e), low = e / (1.0f + e);
    const float up = m < 0.0f ? low : high, down = m < 0.0f ? high : low;
    const float slope = (a.smoothing * up - (1.0f - a.smoothing) * down) * a.beta;
    a.seq_slope[2 * pair] = slope;
    a.seq_slope[2 * pair + 1] = -slope;
    if (!ok) {
        atomicOr(a.seq_bad, 1u);
        if (a.bad)
            atomicOr(a.bad, 1u);
    }
}

// -- launches -------------------------------------------------------------------------------

template <int OP, bool GRAD, bool DUAL>
cudaError_t launch_rows(const LossArgs& a, int dtype, void* stream)
{
    const int sms = sm_count();
    if (!sms)
        return cudaErrorInvalidDevice;
    const uint32_t room = 4u * (uint32_t)sms, grid = a.rows == 0 ? 1 : a.rows < room ? a.rows : room;
    if (dtype == ZERO_F16)
        return launch_train(k_loss_rows<ZERO_F16, OP, GRAD, DUAL>, dim3(grid), kThreads, 0, 1, stream, a);
    return launch_train(k_loss_rows<ZERO_BF16, OP, GRAD, DUAL>, dim3(grid), kThreads, 0, 1, stream, a);
}

constexpr float kLeastTemperature = 1.0f / 1048576, kMostTemperature = 1048576;

// Checks of what the entry points have in common, and the launch arguments it gives.
zero_status_t check_rows(const zero_mat_t* logits, const zero_ids_t* targets, const zero_mat_t* d_logits,
                         float temperature, float scale, LossArgs& a)
{
    zero_status_t st = check_mat(logits, true);
    if (st == ZERO_OK && d_logits)
        st = check_mat(d_logits, true);
    if (st == ZERO_OK && targets)
        st = check_ids(targets);
    if (st != ZERO_OK)
        return st;
    if (logits->cols == 0 || (d_logits && !same_shape(logits, d_logits)) ||
        (targets && targets->count != logits->rows) || nonfinite_host(scale) ||
        !(temperature >= kLeastTemperature && temperature <= kMostTemperature))
        return ZERO_ERR_INVALID_ARG;
    if (logits->cols > ZERO_LOSS_MAX_VOCAB || logits->rows > 0x7FFFFFFFull)
        return ZERO_ERR_UNSUPPORTED;
    a = LossArgs{};
    a.logits = static_cast<const uint16_t*>(logits->base);
    a.pitch = logits->pitch;
    if (d_logits) {
        a.grad = static_cast<uint16_t*>(d_logits->base);
        a.grad_pitch = d_logits->pitch;
    }
    a.rows = (uint32_t)logits->rows;
    a.vocab = (uint32_t)logits->cols;
    if (targets) {
        a.ids = targets->ids;
        a.id_bytes = targets->bytes;
    }
    constexpr double log2e = 1.4426950408889634;
    a.k = (float)(log2e / (double)temperature);
    a.k1 = (float)log2e;
    a.temperature = temperature;
    a.scale = scale;
    return ZERO_OK;
}

// Vectors and workspaces that a call reads or writes.
struct Vec {
    const void* p;
    uint64_t bytes;
    bool out;
};

// Alignment and overlap of everything that a call touches, and that it is device
// memory.  d_logits may take the logits' place.
zero_status_t check_memory(const zero_mat_t* logits, const zero_mat_t* d_logits, const zero_mat_t* top,
                           const Vec* vecs, int n)
{
    constexpr int kMost = 16;
    Span outs[kMost], ins[kMost];
    const void* p[kMost];
    int n_outs = 0, n_ins = 0, np = 0;
    const bool in_place = d_logits && same_place(logits, d_logits);
    if (d_logits)
        outs[n_outs++] = span_of(d_logits);
    if (!in_place)
        ins[n_ins++] = span_of(logits);
    if (top)
        ins[n_ins++] = span_of(top);
    const void* mats[3] = {logits->base, d_logits ? d_logits->base : nullptr, top ? top->base : nullptr};
    for (const void* m : mats)
        if (m)
            p[np++] = m;
    for (int i = 0; i < n; ++i) {
        if (!vecs[i].p)
            continue;
        if (vecs[i].bytes)
            (vecs[i].out ? outs[n_outs++] : ins[n_ins++]) = span_of(vecs[i].p, vecs[i].bytes);
        p[np++] = vecs[i].p;
    }
    return any_overlap(outs, n_outs, ins, n_ins) ? ZERO_ERR_INVALID_ARG : require_device(p, np);
}

bool aligned4(const void* p) { return (uintptr_t)p % 4 == 0; }

Vec ids_vec(const zero_ids_t* ids)
{
    return ids ? Vec{ids->ids, ids->count * ids->bytes, false} : Vec{nullptr, 0, false};
}

// Where the preference loss keeps its parts: the rows' log-probabilities (if the
// caller has no use for them) and sequences, the sequences' slopes and a flag.
struct PairSpace {
    uint64_t logp, seq, slope, flag, total;
};

PairSpace pair_space(uint64_t tokens, uint64_t pairs)
{
    const auto up = [](uint64_t n) { return (n + 15) / 16 * 16; };
    PairSpace s;
    s.logp = 0;
    s.seq = up(4 * tokens);
    s.slope = s.seq + up(4 * tokens);
    s.flag = s.slope + up(8 * pairs);
    s.total = s.flag + 16;
    return s;
}

constexpr uint64_t kMaxRows = 0x7FFFFFFFull;

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" zero_status_t zero_token_logprob(const zero_mat_t* logits, const zero_ids_t* targets,
                                            float temperature, float* logp, float* lse, uint32_t* d_bad,
                                            void* stream)
{
    LossArgs a;
    if (!targets || (!logp && !lse))
        return ZERO_ERR_INVALID_ARG;
    zero_status_t st = check_rows(logits, targets, nullptr, temperature, 1.0f, a);
    if (st != ZERO_OK)
        return st;
    if (!aligned4(logp) || !aligned4(lse) || !aligned4(d_bad))
        return ZERO_ERR_ALIGNMENT;
    if (a.rows == 0)
        return ZERO_OK;
    const uint64_t n = 4 * logits->rows;
    const Vec vecs[4] = {ids_vec(targets), {logp, n, true}, {lse, n, true}, {d_bad, 4, true}};
    st = check_memory(logits, nullptr, nullptr, vecs, 4);
    if (st != ZERO_OK)
        return st;
    a.logp = logp;
    a.lse = lse;
    a.bad = d_bad;
    return train_status(launch_rows<kLogp, false, false>(a, logits->dtype, stream));
}

extern "C" zero_status_t zero_token_logprob_backward(const zero_mat_t* logits, const zero_ids_t* targets,
                                                     float temperature, const float* d_logp,
                                                     const zero_mat_t* d_logits, uint32_t* d_bad, void* stream)
{
    LossArgs a;
    if (!targets || !d_logits)
        return ZERO_ERR_INVALID_ARG;
    zero_status_t st = check_rows(logits, targets, d_logits, temperature, 1.0f, a);
    if (st != ZERO_OK)
        return st;
    if (!d_logp && a.rows)
        return ZERO_ERR_INVALID_ARG;
    if (!aligned4(d_logp) || !aligned4(d_bad))
        return ZERO_ERR_ALIGNMENT;
    if (a.rows == 0)
        return ZERO_OK;
    const Vec vecs[3] = {ids_vec(targets), {d_logp, 4 * logits->rows, false}, {d_bad, 4, true}};
    st = check_memory(logits, d_logits, nullptr, vecs, 3);
    if (st != ZERO_OK)
        return st;
    a.slope = d_logp;
    a.scale = (float)(1.0 / (double)temperature);
    a.bad = d_bad;
    return train_status(launch_rows<kSlope, true, false>(a, logits->dtype, stream));
}

extern "C" zero_status_t zero_distill_loss(const zero_mat_t* logits, const zero_mat_t* top,
                                           const zero_ids_t* top_ids, float temperature, float soft,
                                           const zero_ids_t* targets, float hard, const float* weight,
                                           float scale, float* loss, const zero_mat_t* d_logits,
                                           uint32_t* d_bad, void* stream)
{
    LossArgs a;
    zero_status_t st = check_rows(logits, targets, d_logits, temperature, scale, a);
    if (st != ZERO_OK)
        return st;
    if ((!top) != (!top_ids) || nonfinite_host(soft) || nonfinite_host(hard) || (!targets && hard != 0.0f) ||
        (!loss && !d_logits))
        return ZERO_ERR_INVALID_ARG;
    if (top) {
        st = check_mat(top, true);
        if (st == ZERO_OK)
            st = check_ids(top_ids);
        if (st != ZERO_OK)
            return st;
        if (top->rows != logits->rows || top->dtype != logits->dtype)
            return ZERO_ERR_INVALID_ARG;
        if (top->cols > ZERO_DISTILL_MAX_TOP)
            return ZERO_ERR_UNSUPPORTED;
        if (top_ids->count != top->rows * top->cols)
            return ZERO_ERR_INVALID_ARG;
        if (top->cols == 0)
            top = nullptr;
    }
    if (!aligned4(weight) || !aligned4(loss) || !aligned4(d_bad))
        return ZERO_ERR_ALIGNMENT;
    if (a.rows == 0)
        return ZERO_OK;
    const uint64_t n = 4 * logits->rows;
    const Vec vecs[5] = {ids_vec(targets), ids_vec(top ? top_ids : nullptr), {weight, n, false}, {loss, n, true},
                         {d_bad, 4, true}};
    st = check_memory(logits, d_logits, top, vecs, 5);
    if (st != ZERO_OK)
        return st;
    a.weight = weight;
    a.loss = loss;
    a.bad = d_bad;
    a.soft = soft;
    a.hard = hard;
    if (top) {
        a.top = static_cast<const uint16_t*>(top->base);
        a.top_pitch = top->pitch;
        a.top_n = (uint32_t)top->cols;
        a.top_ids = top_ids->ids;
        a.top_id_bytes = top_ids->bytes;
    } else {
        a.k = a.k1;   // the cross-entropy alone
    }
    const bool dual = top && hard != 0.0f && temperature != 1.0f;
    cudaError_t e;
    if (d_logits)
        e = dual ? launch_rows<kDistill, true, true>(a, logits->dtype, stream)
                 : launch_rows<kDistill, true, false>(a, logits->dtype, stream);
    else
        e = dual ? launch_rows<kDistill, false, true>(a, logits->dtype, stream)
                 : launch_rows<kDistill, false, false>(a, logits->dtype, stream);
    return train_status(e);
}

extern "C" zero_status_t zero_policy_loss(const zero_mat_t* logits, const zero_ids_t* targets, float temperature,
                                          const float* old_logp, const float* ref_logp, const float* advantage,
                                          const float* weight, float clip_low, float clip_high, float kl,
                                          float scale, float* loss, float* logp, const zero_mat_t* d_logits,
                                          uint32_t* d_bad, void* stream)
{
    LossArgs a;
    if (!targets || (!loss && !logp && !d_logits))
        return ZERO_ERR_INVALID_ARG;
    zero_status_t st = check_rows(logits, targets, d_logits, temperature, scale, a);
    if (st != ZERO_OK)
        return st;
    if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f) || nonfinite_host(clip_high) ||
        nonfinite_host(kl) || (a.rows && (!old_logp || !advantage || (!ref_logp && kl != 0.0f))))
        return ZERO_ERR_INVALID_ARG;
    const void* fp32[7] = {old_logp, ref_logp, advantage, weight, loss, logp, d_bad};
    for (const void* v : fp32)
        if (!aligned4(v))
            return ZERO_ERR_ALIGNMENT;
    if (a.rows == 0)
        return ZERO_OK;
    if (kl == 0.0f)
        ref_logp = nullptr;
    const uint64_t n = 4 * logits->rows;
    const Vec vecs[8] = {ids_vec(targets), {old_logp, n, false}, {ref_logp, n, false}, {advantage, n, false},
                         {weight, n, false}, {loss, n, true}, {logp, n, true}, {d_bad, 4, true}};
    st = check_memory(logits, d_logits, nullptr, vecs, 8);
    if (st != ZERO_OK)
        return st;
    a.old_logp = old_logp;
    a.ref = ref_logp;
    a.advantage = advantage;
    a.weight = weight;
    a.low = (float)(1.0 - (double)clip_low);
    a.high = (float)(1.0 + (double)clip_high);
    a.kl = kl;
    a.scale = (float)((double)scale / (double)temperature);
    a.loss = loss;
    a.logp = logp;
    a.bad = d_bad;
    return train_status(d_logits ? launch_rows<kPolicy, true, false>(a, logits->dtype, stream)
                                 : launch_rows<kPolicy, false, false>(a, logits->dtype, stream));
}

extern "C" uint64_t zero_preference_loss_workspace(uint64_t tokens, uint64_t pairs)
{
    return tokens > kMaxRows || pairs > kMaxRows ? UINT64_MAX : pair_space(tokens, pairs).total;
}

extern "C" zero_status_t zero_preference_loss(const zero_mat_t* logits, const zero_ids_t* targets,
                                              const zero_ids_t* starts, const float* ref_logp, float beta,
                                              float smoothing, float scale, float* loss, float* reward,
                                              float* logp, const zero_mat_t* d_logits, void* workspace,
                                              uint64_t workspace_bytes, uint32_t* d_bad, void* stream)
{
    LossArgs a;
    if (!targets)
        return ZERO_ERR_INVALID_ARG;
    zero_status_t st = check_rows(logits, targets, d_logits, 1.0f, scale, a);
    if (st == ZERO_OK)
        st = check_ids(starts);
    if (st != ZERO_OK)
        return st;
    if (starts->count % 2 == 0 || nonfinite_host(beta) || !(smoothing >= 0.0f && smoothing <= 1.0f))
        return ZERO_ERR_INVALID_ARG;
    const uint64_t pairs = starts->count / 2;
    if (!loss && pairs)
        return ZERO_ERR_INVALID_ARG;
    const void* fp32[5] = {ref_logp, loss, reward, logp, d_bad};
    for (const void* v : fp32)
        if (!aligned4(v))
            return ZERO_ERR_ALIGNMENT;
    const PairSpace space = pair_space(logits->rows, pairs);
    if (!workspace || workspace_bytes < space.total)
        return ZERO_ERR_INVALID_ARG;
    if ((uintptr_t)workspace % 16 != 0)
        return ZERO_ERR_ALIGNMENT;
    if (a.rows == 0 && pairs == 0)
        return ZERO_OK;
    const uint64_t n = 4 * logits->rows;
    const Vec vecs[8] = {ids_vec(targets), ids_vec(starts), {ref_logp, n, false}, {loss, 4 * pairs, true},
                         {reward, 8 * pairs, true}, {logp, n, true}, {workspace, space.total, true},
                         {d_bad, 4, true}};
    st = check_memory(logits, d_logits, nullptr, vecs, 8);
    if (st != ZERO_OK)
        return st;
    char* ws = static_cast<char*>(workspace);
    a.starts = starts->ids;
    a.start_bytes = starts->bytes;
    a.pairs = (uint32_t)pairs;
    a.logp = logp ? logp : reinterpret_cast<float*>(ws + space.logp);
    a.seq = reinterpret_cast<int32_t*>(ws + space.seq);
    a.seq_slope = reinterpret_cast<float*>(ws + space.slope);
    a.seq_bad = reinterpret_cast<uint32_t*>(ws + space.flag);
    a.ref = ref_logp;
    a.beta = beta;
    a.smoothing = smoothing;
    a.loss = loss;
    a.reward = reward;
    a.bad = d_bad;
    LossArgs first = a;
    first.grad = nullptr;
    cudaError_t e = launch_rows<kLogp, false, false>(first, logits->dtype, stream);
    if (e == cudaSuccess)
        e = launch_train(k_pairs, dim3((unsigned)(pairs + (logits->rows + kPairThreads - 1) / kPairThreads)),
                         kPairThreads, 0, 1, stream, a);
    if (e == cudaSuccess && d_logits && a.rows)
        e = launch_rows<kPairs, true, false>(a, logits->dtype, stream);
    return train_status(e);
}
