// tern_mat.h -- strided matrices of the C ABI, as its checks of arguments see
// them (host only).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "tern_plan.h"

namespace tern {

// A strided [rows, cols] buffer (a column slice of a wider one).
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    size_t es;
    size_t bytes() const { return rows && cols ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0; }
};

// Do two strided buffers share an element?  Slices of one matrix (equal row
// strides) interleave: there only the columns count.
inline bool mats_overlap(const Mat &a, const Mat &b) {
    if (!ranges_overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
    if (a.ld * (int64_t)a.es != b.ld * (int64_t)b.es || a.ld == 0) return true;
    const uint64_t ldb = (uint64_t)a.ld * a.es;
    const uint64_t x = (uint64_t)(uintptr_t)a.p, y = (uint64_t)(uintptr_t)b.p;
    const uint64_t d = y >= x ? (y - x) % ldb : (ldb - (x - y) % ldb) % ldb;   // columns b lies behind a
    return d < (uint64_t)a.cols * a.es || ldb - d < (uint64_t)b.cols * b.es;
}

inline bool any_overlap(const Mat *outs, int nout, const Mat *ins, int nin) {
    for (int i = 0; i < nout; i++) {
        for (int j = i + 1; j < nout; j++)
            if (mats_overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < nin; j++)
            if (mats_overlap(outs[i], ins[j])) return true;
    }
    return false;
}

}  // namespace tern
