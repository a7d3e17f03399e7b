// Host-side argument checks of the training operators (zero_train.h).
#include "zero_train_internal.h"

namespace zero {

namespace {

// Keeps every byte offset the kernels form far inside 64 bits.
constexpr uint64_t kMaxElems = 1ull << 56;

bool shape_ok(uint64_t rows, uint64_t cols, uint64_t pitch)
{
    return pitch >= cols && cols < kMaxElems && pitch < kMaxElems && rows < kMaxElems &&
           (pitch == 0 || rows <= kMaxElems / pitch);
}

}  // namespace

Span span_of(const zero_mat_t* m)
{
    return Span{(uintptr_t)m->base, m->cols ? m->rows : 0, 2 * m->cols, 2 * m->pitch};
}

Span span_of_q(const zero_act8_t* a)
{
    return Span{(uintptr_t)a->q, a->cols ? a->rows : 0, a->cols, a->q_pitch};
}

Span span_of_scale(const zero_act8_t* a)
{
    return Span{(uintptr_t)a->scale, a->cols ? a->rows : 0,
                (a->cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK, a->scale_pitch};
}

Span span_of(const void* p, uint64_t bytes) { return Span{(uintptr_t)p, bytes ? 1u : 0u, bytes, bytes}; }

bool spans_overlap(const Span& a, const Span& b)
{
    if (!a.base || !b.base || !a.rows || !b.rows || !a.row_bytes || !b.row_bytes)
        return false;
    const uintptr_t a1 = a.base + (a.rows - 1) * a.pitch_bytes + a.row_bytes;
    const uintptr_t b1 = b.base + (b.rows - 1) * b.pitch_bytes + b.row_bytes;
    if (a1 <= b.base || b1 <= a.base)
        return false;
    if (a.pitch_bytes == b.pitch_bytes && a.pitch_bytes) {
        const uint64_t pitch = a.pitch_bytes;
        // b's rows start d bytes past one of a's (modulo the pitch)
        const uint64_t d = b.base >= a.base ? (b.base - a.base) % pitch
                                            : (pitch - (a.base - b.base) % pitch) % pitch;
        if (d >= a.row_bytes && d + b.row_bytes <= pitch)
            return false;
    }
    return true;
}

bool any_overlap(const Span* outs, int n_outs, const Span* ins, int n_ins)
{
    for (int i = 0; i < n_outs; ++i) {
        for (int j = i + 1; j < n_outs; ++j)
            if (spans_overlap(outs[i], outs[j]))
                return true;
        for (int j = 0; j < n_ins; ++j)
            if (spans_overlap(outs[i], ins[j]))
                return true;
    }
    return false;
}

zero_status_t check_mat(const zero_mat_t* m, bool act)
{
    if (!m || (m->dtype != ZERO_F16 && m->dtype != ZERO_BF16) ||
        !shape_ok(m->rows, m->cols, m->pitch))
        return ZERO_ERR_INVALID_ARG;
    if (!m->base)
        return m->rows && m->cols ? ZERO_ERR_INVALID_ARG : ZERO_OK;
    const uintptr_t b = (uintptr_t)m->base;
    if (act ? (b % 16 != 0 || m->pitch % 8 != 0) : b % 2 != 0)
        return ZERO_ERR_ALIGNMENT;
    const uint64_t bytes = 2 * m->rows * m->pitch;
    return b + bytes < b ? ZERO_ERR_INVALID_ARG : ZERO_OK;
}

zero_status_t check_act8(const zero_act8_t* a)
{
    if (!a || !shape_ok(a->rows, a->cols, a->q_pitch) || a->scale_pitch >= kMaxElems ||
        a->scale_pitch < (a->cols + ZERO_ACT8_BLOCK - 1) / ZERO_ACT8_BLOCK ||
        (a->scale_pitch && a->rows > kMaxElems / a->scale_pitch))
        return ZERO_ERR_INVALID_ARG;
    if (!a->q || !a->scale)
        return a->rows && a->cols ? ZERO_ERR_INVALID_ARG : ZERO_OK;
    if ((uintptr_t)a->q % 16 != 0 || a->q_pitch % 16 != 0)
        return ZERO_ERR_ALIGNMENT;
    const uintptr_t q = (uintptr_t)a->q, s = (uintptr_t)a->scale;
    if (q + a->rows * a->q_pitch < q || s + a->rows * a->scale_pitch < s)
        return ZERO_ERR_INVALID_ARG;
    return ZERO_OK;
}

zero_status_t check_ids(const zero_ids_t* ids)
{
    if (!ids || (ids->bytes != 4 && ids->bytes != 8) || (!ids->ids && ids->count))
        return ZERO_ERR_INVALID_ARG;
    if (ids->count > 0x7FFFFFFFull)
        return ZERO_ERR_UNSUPPORTED;
    if ((uintptr_t)ids->ids % ids->bytes != 0)
        return ZERO_ERR_ALIGNMENT;
    const uintptr_t p = (uintptr_t)ids->ids;
    return p + ids->count * ids->bytes < p ? ZERO_ERR_INVALID_ARG : ZERO_OK;
}

}  // namespace zero
