// tern_softmax.h -- rows of logits held in registers, shared by the log
// probabilities (tern_logprob.hip) and the distillation loss (tern_distill.hip).
//
// A row, or a segment of one, is read once: W waves take it in strides of W * 512
// elements, eight neighbours a lane, and NV such eights stay in a lane's
// registers as they came.  Its largest element is then known before the first
// exponential, so a sum needs no rescaling, and what comes after the sums (the
// top alternatives, the gradient) reads registers again and not memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/tern.h"
#include "tern_mat.h"
#include "tern_plan.h"
#include "tern_rows.h"

namespace tern {
namespace rows {

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.4426950408889634074;
constexpr float kLn2 = 0.693147180559945309f;

__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// (v_max3: fmaxf of loaded bits makes two instructions, one to quiet NaNs)
__device__ inline float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// The lanes of a row meet: those of a workgroup, or of the one wave that has it.
template <int W>
__device__ inline void meet() {
    if constexpr (W > 1) {
        __syncthreads();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Eight elements that are not there.
template <int DT>
__device__ inline Raw8<DT> none8() {
    constexpr uint32_t w = DT == TERN_BF16 ? 0xFF80FF80u : 0xFF800000u;
    Raw8<DT> r;
#pragma unroll
    for (int i = 0; i < Raw8<DT>::N; i++) r.v[i] = u32x4{w, w, w, w};
    return r;
}

// A lane's number that the compiler takes for new: it would compute what depends
// on it for all rows ahead of the loop over them, and spill that.
__device__ inline int fresh(int tid) {
    asm volatile("" : "+v"(tid));
    return tid;
}

// The n elements from z on into registers, -inf behind them.
template <int DT, int W, int NV>
__device__ inline void load_row(const char *z, int n, int tid, Raw8<DT> (&x)[NV]) {
    constexpr int ST = W * 512, ES = esize<DT>();
    tid = fresh(tid);
    const int full = n & ~7;
    const uint32_t lane = (uint32_t)tid * (8 * ES);
    if (n == NV * ST) {   // every lane has all its eights
#pragma unroll
        for (int i = 0; i < NV; i++) x[i] = load8<DT>(z + i * ST * ES + lane);
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; i++) {
        x[i] = none8<DT>();
        if (tid * 8 < full - i * ST) x[i] = load8<DT>(z + i * ST * ES + lane);
    }
    if (n & 7 && tid == full % ST / 8) {   // the lane that has the last, partial eight
        const char *p = z + (int64_t)full * ES;
        Raw8<DT> t = none8<DT>();
#pragma unroll
        for (int j = 0; j < 7; j++) {
            if (full + j >= n) continue;
            if constexpr (DT == TERN_BF16) {
                const uint32_t e = ((const uint16_t *)p)[j], keep = j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                t.v[0][j >> 1] = (t.v[0][j >> 1] & keep) | e << (j & 1 ? 16 : 0);
            } else {
                t.v[j >> 2][j & 3] = ((const uint32_t *)p)[j];
            }
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (i == full / ST) x[i] = t;
    }
}

__device__ inline float max8(const float *f) {
    return max3(max3(f[0], f[1], f[2]), max3(f[3], f[4], f[5]), fmaxf(f[6], f[7]));
}

// unpack8 that the compiler does not see through: it would keep the unpacked
// elements, or the exponentials, of one pass over the registers for the next, at
// twice the registers.  (The registers themselves are not made opaque: passes under
// a condition would then leave two versions of them.)
template <int DT>
__device__ inline void unpack8_again(const Raw8<DT> &r, float *f) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if constexpr (DT == TERN_BF16) {
            const uint32_t w = r.v[0][i >> 1];
            if (i & 1) asm volatile("v_and_b32 %0, 0xffff0000, %1" : "=v"(f[i]) : "v"(w));
            else asm volatile("v_lshlrev_b32 %0, 16, %1" : "=v"(f[i]) : "v"(w));
        } else {
            const uint32_t w = r.v[i >> 2][i & 3];
            asm volatile("v_mov_b32 %0, %1" : "=v"(f[i]) : "v"(w));
        }
    }
}

// A pass over the registers: f(i, eight elements) of each stride that the row
// reaches; nothing moves across turns, or all would be unpacked first.
template <int DT, int W, int NV, class F>
__device__ inline void each8(const Raw8<DT> (&x)[NV], int n, F f) {
#pragma unroll
    for (int i = 0; i < NV; i++) {
        if (i * W * 512 < n) {
            float e[8];
            unpack8_again<DT>(x[i], e);
            f(i, e);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// A lane's largest element (NaN loses against a number).
template <int DT, int W, int NV>
__device__ inline float lane_max(const Raw8<DT> (&x)[NV], int n) {
    float m = -kInf;
    each8<DT, W, NV>(x, n, [&](int, const float *f) {
        m = max3(max3(m, f[0], f[1]), max3(f[2], f[3], f[4]), max3(f[5], f[6], f[7]));
    });
    return m;
}

// Reductions over the W waves of a row; sh holds W floats, which are free
// again after the next meeting.
template <class Op, int W>
__device__ inline float row_all(float x, float *sh, int tid) {
    x = wave_all<Op>(x);
    if constexpr (W > 1) {
        if ((tid & 63) == 0) sh[tid >> 6] = x;
        __syncthreads();
        x = sh[0];
#pragma unroll
        for (int i = 1; i < W; i++) x = Op::of(x, sh[i]);
    }
    return x;
}
template <int W>
__device__ inline void row_sums(float &a, float &b, float (*sh)[W], int tid) {
    a = wave_all<Add>(a);
    b = wave_all<Add>(b);
    if constexpr (W > 1) {
        if ((tid & 63) == 0) sh[0][tid >> 6] = a, sh[1][tid >> 6] = b;
        __syncthreads();
        a = sh[0][0], b = sh[1][0];
#pragma unroll
        for (int i = 1; i < W; i++) a += sh[0][i], b += sh[1][i];
    }
}

// Bits that order as the values do, -0 as +0, NaN outermost.
__device__ inline uint32_t ordered(float f) {
    const uint32_t b = as_u(f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float from_ordered(uint32_t o) { return as_f(o & 0x80000000u ? o ^ 0x80000000u : ~o); }
// The value, then the lower index: no two elements of a row have one key.
__device__ inline uint64_t key_of(float f, uint32_t i) { return (uint64_t)ordered(f) << 32 | (0xFFFFFFFFu - i); }
__device__ inline int index_of(uint64_t key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }
__device__ inline float value_of(uint64_t key) { return from_ordered((uint32_t)(key >> 32)); }

// The exponents of a row, in units of log 2: (z - m0) c by one fused multiply-add,
// from m0 c as rounded, which is `off` less than it should be.  Where m0 c is so large
// that this would matter, or overflow, `far` says that the row takes its differences
// first, element by element.
struct Exponent {
    float c, mc, off;
    bool far;
    __device__ Exponent(float m0, float factor) : c(factor), mc(m0 * factor), off(fmaf(m0, factor, -mc)) {
        far = !(fabsf(mc) < 1048576.0f);
    }
    __device__ float of(float z) const { return fmaf(z, c, -mc); }
};

// z - m by halves (half of it), and its product with a factor: the difference of any two numbers fits.
__device__ inline float half_apart(float z, float m) { return fmaf(z, 0.5f, -0.5f * m); }
__device__ inline float apart(float z, float m, float f) { return 2.0f * (half_apart(z, m) * f); }

// A row's sum of exponentials, to which its largest element gives 1 (nothing allowed:
// 0): a rounding below that would make a probability above 1.
__device__ inline float at_least_one(float s) { return s > 0.0f && s < 1.0f ? 1.0f : s; }

template <int DT>
__device__ inline float at(const char *z, int64_t v) { return load1<DT>(z + v * esize<DT>()); }

}  // namespace rows

// ---------------------------------------------------------------------------
// How the rows are dealt out (host).
// ---------------------------------------------------------------------------

// Eights a lane holds at most: 64 registers.
constexpr int held(int32_t dt) { return dt == TERN_BF16 ? 16 : 8; }
constexpr int kMaxSegments = 64;
// workgroups of a launch; they go on to further rows
constexpr int64_t kMaxGroups = 1 << 16;

struct RowPlan {
    int S, W, NV;        // parts of a row, a workgroup (or wave) each; its waves, and eights of a lane
    int64_t part, seg;   // elements of a part, and of the segments that it takes in turn
};

inline int64_t cdiv_(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whole rows where there are enough of them; few long rows are cut, so that up to 512
// workgroups share them.  `most`: waves of a workgroup; in_turn: a part may take
// several segments, else it is one.  Rounded down, since a second turn of few
// workgroups costs more than it gives (127 rows of 131072 fp32 with gradient: 47 us
// in 5 parts, 40 in 4).  A gradient reads cut rows again, so that more rows than that
// stay whole (300 rows of 50021: 25 us whole, 27 cut); in turn, they are cut while
// the 1024 workgroups that run at once get 24576 elements each (20 alternatives, 200
// rows: of 131072 36 us whole, 28 in 3 parts, 24 in 5; of 32768 11 us whole, 15 in 3).
inline RowPlan plan_rows(int32_t dt, int64_t T, int64_t V, int most, bool in_turn) {
    const int nv = held(dt);
    RowPlan p{};
    const int64_t fits = (int64_t)most * 512 * nv;
    int64_t S = in_turn ? 1 : cdiv_(V, fits);
    if (S > 1) S = cdiv_(V, fits / 2);   // cut anyway: halves, two of which share a compute unit
    const int64_t rows = std::max<int64_t>(T, 1);
    if (T < 128) S = std::max(S, std::min(512 / rows, cdiv_(V, 4096)));
    if (in_turn && T < 512) S = std::max(S, std::min(1024 / rows, V / 24576));
    S = std::min<int64_t>(S, kMaxSegments);
    p.part = cdiv_(cdiv_(V, S), 8) * 8;
    p.S = (int)cdiv_(V, p.part);
    p.seg = cdiv_(cdiv_(p.part, cdiv_(p.part, fits)), 8) * 8;
    // waves: what the registers take, and four where single ones leave the chip empty
    // (16 waves where 4 do cost more than they give: 300 rows of 50021, 20 alternatives,
    // 29 us with 16 and 20 with 4)
    p.W = 1;
    for (int w : {4, 8, 16})
        if ((int64_t)p.W * 512 * nv < p.seg) p.W = w;
    if (p.W == 1 && T * p.S < 2048 && p.seg > 512) p.W = 4;
    p.NV = nv;
    for (int v : {4, 1})
        if ((int64_t)p.W * 512 * v >= p.seg) p.NV = v;
    return p;
}

// f<W, NV>() of the kernel that a plan of LEAST to MOST waves asks for.
template <int32_t DT, int LEAST, int MOST, class F>
void with_plan(const RowPlan &p, F f) {
    constexpr int H = held(DT);
    const bool big = p.NV > 4;
    if constexpr (LEAST <= 1) {
        if (p.W == 1) {
            if (big) f.template operator()<1, H>();
            else if (p.NV > 1) f.template operator()<1, 4>();
            else f.template operator()<1, 1>();
        }
    }
    if (p.W == 4) {
        if (big) f.template operator()<4, H>();
        else f.template operator()<4, 4>();
    }
    if constexpr (MOST >= 8)
        if (p.W == 8) f.template operator()<8, H>();
    if constexpr (MOST >= 16)
        if (p.W == 16) f.template operator()<16, H>();
}

inline bool row_sizes_ok(int64_t T, int64_t V) { return T >= 0 && T <= kMaxT && V >= 1 && V <= kMaxInOut; }
inline bool row_stride_ok(int64_t ld, int64_t V) { return ld >= V && ld % 8 == 0 && ld <= kMaxInOut * 8; }
// a factor of the logits and its product with log2 e, above 0 and finite
inline bool factor_ok(double x) { return x > 0.0 && x * rows::kLog2e <= 3.4e38; }
inline bool off_by(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) != 0; }
inline Mat vec(const void *p, int64_t n, size_t es) { return {p, 1, n, n, es}; }

}  // namespace tern
