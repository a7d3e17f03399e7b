// Host-side argument checks shared by the training operators (zero_train.h).
// Not part of the public ABI.
#pragma once

#include <stdint.h>

#include "zero_internal.h"
#include "zero_train.h"

namespace zero {

// A strided range of device memory, for overlap checks: `rows` rows of
// `row_bytes` bytes, `pitch_bytes` apart.
struct Span {
    uintptr_t base;
    uint64_t rows;
    uint64_t row_bytes;
    uint64_t pitch_bytes;
};

// The memory of a matrix, a checkpoint's two arrays, or `bytes` in a row.
Span span_of(const zero_mat_t* m);
Span span_of_q(const zero_act8_t* a);
Span span_of_scale(const zero_act8_t* a);
Span span_of(const void* p, uint64_t bytes);

// True if the two ranges share a byte.  Ranges of the same pitch that
// interleave (column slices of one buffer) do not overlap if their columns
// do not.
bool spans_overlap(const Span& a, const Span& b);

// True if any of outs[0..n_outs) overlaps another of them or one of ins.
bool any_overlap(const Span* outs, int n_outs, const Span* ins, int n_ins);

// Shape, size and alignment of an activation matrix (act = true: 16-byte rows)
// or a parameter matrix (2-byte aligned, any pitch).  A NULL base is accepted
// only for a matrix without elements.
zero_status_t check_mat(const zero_mat_t* m, bool act);

// The same for a checkpoint descriptor.
zero_status_t check_act8(const zero_act8_t* a);

// The same for token numbers (at most 2^31 - 1 of them).
zero_status_t check_ids(const zero_ids_t* ids);

inline bool same_shape(const zero_mat_t* a, const zero_mat_t* b)
{
    return a->rows == b->rows && a->cols == b->cols && a->dtype == b->dtype;
}

// True for an inf or NaN.
inline bool nonfinite_host(float x) { return !(x - x == 0.0f); }

// The same matrix in memory: an operator may then work in place.
inline bool same_place(const zero_mat_t* a, const zero_mat_t* b)
{
    return a->base == b->base && a->pitch == b->pitch;
}

}  // namespace zero
