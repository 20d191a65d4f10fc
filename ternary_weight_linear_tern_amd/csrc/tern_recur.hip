// tern_recur.hip -- the gated linear recurrence between the receptance, key
// and value projections and the output projection (C ABI in include/tern.h).
//
//   w_t = sigmoid(k_t)          h_t = h_{t-1} + w_t (v_t - h_{t-1})
//   s_t = sigmoid(r_t)          y_t = s_t h_t
//
// per channel, over packed sequences.  The update is written with w and not
// with the kept share 1 - w: a gate near 0 (a long memory) keeps its relative
// accuracy.  All states, gradients and sums are fp32.
//
// A step is an affine map of the state, h -> (1 - w) h + w v, and affine maps
// compose to affine maps (A, B): h -> A h + B.  So the T tokens (the packed
// sequences laid end to end) are cut into chunks of `L` rows:
//   recur_agg    the pair (A, B) of every chunk, from K and V;
//   recur_carry  the state that enters every chunk, by composing the pairs;
//   recur_fwd    the tokens again from the entering state, writing Y.
// A sequence's first token drops what came before: the composition restarts
// there with A = 0 and B = h0, and a pair with A = 0 returns B without
// multiplying, so nothing of one sequence (a NaN, an infinity) reaches the
// next.
//
// Backward, with u_t = dy_t s_t and g_t the gradient that reaches h_t:
//   g_t = u_t + (1 - w_{t+1}) g_{t+1}   (+ dhT behind the last token)
//   dv = g w,  dk = g (v - h_{t-1}) w (1 - w),  dr = dy h s (1 - s)
// p_t = (1 - w_t) g_t, the gradient of h_{t-1}, is again an affine chain, run
// from the last token to the first, and cut into the same chunks.  The states
// h_{t-1} come from the forward's checkpoints (one row every 16 tokens).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tern.h"
#include "tern_cursor.h"
#include "tern_plan.h"

namespace tern {
namespace rdev {

constexpr int kBlk = TERN_RECUR_BLOCK;   // rows between two checkpoints of the state

struct RecurArgs {
    const void *K, *V, *R;     // [T, C], row stride ld
    int64_t ld;
    const float *h0;           // [S, C] or null (zeros)
    const int64_t *off;        // [S + 1] or null (one sequence of T tokens)
    int64_t S, T;
    int C, ncb;                // channels; column blocks of a wave
    int L, nch;                // rows of a chunk; chunks
    void *Y;                   // [T, C], row stride ldy
    int64_t ldy;
    float *hT;                 // [S, C] or null
    float *states;             // [ceil(T / 16), C]: the state before each 16-row block
    float *agg;                // [nch][2][C]
    float *carry;              // [nch][C], or null with one chunk
    const void *dY;            // [T, C], row stride lddy
    int64_t lddy;
    const float *dhT;          // [S, C] or null (zeros)
    void *dK, *dV, *dR;        // [T, C], row stride ldd
    int64_t ldd;
    float *dh0;                // [S, C] or null
};

// One lane's channels: 4 bytes of a row (256 consecutive bytes a wave).
struct Bf {
    static constexpr int N = 2;
    using Raw = uint32_t;
    __device__ static void unpack(Raw x, float *f) {
        f[0] = __builtin_bit_cast(float, x << 16);
        f[1] = __builtin_bit_cast(float, x & 0xFFFF0000u);
    }
    // round to nearest even (NaN stays NaN)
    __device__ static Raw pack(const float *f) {
        Raw r = 0;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const __bf16 b = (__bf16)f[i];
            r |= (Raw)__builtin_bit_cast(unsigned short, b) << (16 * i);
        }
        return r;
    }
};
struct Fp {
    static constexpr int N = 1;
    using Raw = float;
    __device__ static void unpack(Raw x, float *f) { f[0] = x; }
    __device__ static Raw pack(const float *f) { return f[0]; }
};

template <int N>
__device__ inline void load_f(const float *p, float *f) {
#pragma unroll
    for (int i = 0; i < N; i++) f[i] = p[i];
}
template <int N>
__device__ inline void store_f(float *p, const float *f) {
#pragma unroll
    for (int i = 0; i < N; i++) p[i] = f[i];
}

__device__ inline float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * -1.44269504088896340736f); }
__device__ inline float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_neg(x)); }

// sigmoid(x) and its derivative sigmoid(x) sigmoid(-x), neither by a
// difference that would cancel where the gate saturates
__device__ inline float sigmoid_d(float x, float &d) {
    const float e = exp_neg(fabsf(x));
    const float i = __builtin_amdgcn_rcpf(1.0f + e);
    d = e * i * i;
    return x < 0.0f ? e * i : i;
}

// wave-uniform position of the wave: column block and chunk (or, beyond the
// chunks, a group of 64 sequences)
__device__ inline void wave_pos(const RecurArgs &a, int &c, int64_t &y) {
    const int64_t b = blockIdx.x;
    y = b / a.ncb;
    c = (int)(b - y * a.ncb);
}

// The rows of one checkpoint block (rows beyond the chunk's end repeat its
// last one), all loads issued together.
template <class E>
__device__ inline void load_rows(typename E::Raw *x, const void *p, int64_t ld, int64_t tb, int64_t t1, int col) {
    constexpr int es = 4 / E::N;
    const char *base = (const char *)p + (tb * ld + col) * es;
#pragma unroll
    for (int j = 0; j < kBlk; j++) {
        const int64_t r = tb + j < t1 ? j : t1 - 1 - tb;
        x[j] = *(const typename E::Raw *)(base + r * ld * es);
    }
}

// Keeps loads that were issued before it from sinking to their uses.
__device__ inline void issued() { __builtin_amdgcn_sched_barrier(0); }

// Sequences without tokens pass their state through: dst[s] = src[s].
template <int N>
__device__ inline void copy_empty(const RecurArgs &a, int64_t group, int col, const float *src, float *dst) {
    const int64_t s = group * 64 + threadIdx.x;
    bool e = false;
    if (s < a.S) e = a.off ? a.off[s + 1] <= a.off[s] : a.T == 0;
    uint64_t m = __ballot(e);
    while (m) {
        const int64_t i = group * 64 + __builtin_ctzll(m);
        m &= m - 1;
        if (col < a.C) {
            float f[N] = {};
            if (src) load_f<N>(src + i * a.C + col, f);
            store_f<N>(dst + i * a.C + col, f);
        }
    }
}

// (A, B) of a chunk in token order
template <class E>
__global__ __launch_bounds__(64) void recur_agg_kernel(RecurArgs a) {
    constexpr int N = E::N;
    using Raw = typename E::Raw;
    int cb;
    int64_t ch;
    wave_pos(a, cb, ch);
    const int col = (cb * 64 + (int)threadIdx.x) * N;
    if (col >= a.C) return;
    const int64_t t0 = ch * a.L, t1 = t0 + a.L < a.T ? t0 + a.L : a.T;
    Cursor cu{a.off, a.S, a.T, 0};
    cu.seek(t0);
    int64_t nb = cu.end();
    bool first = cu.live() && cu.begin() == t0;
    float A[N], B[N];
#pragma unroll
    for (int i = 0; i < N; i++) A[i] = 1.0f, B[i] = 0.0f;
    auto row = [&](Raw kr, Raw vr) {
        float kf[N], vf[N];
        E::unpack(kr, kf);
        E::unpack(vr, vf);
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float w = sigmoid(kf[i]);
            A[i] = fmaf(-w, A[i], A[i]);
            B[i] = fmaf(w, vf[i] - B[i], B[i]);
        }
    };
    Raw k[kBlk], v[kBlk];
    load_rows<E>(k, a.K, a.ld, t0, t1, col);
    load_rows<E>(v, a.V, a.ld, t0, t1, col);
    for (int64_t tb = t0; tb < t1; tb += kBlk) {
        // the next block's loads fly while this one is worked on
        const int64_t tn = tb + kBlk < t1 ? tb + kBlk : tb;
        Raw k2[kBlk], v2[kBlk];
        load_rows<E>(k2, a.K, a.ld, tn, t1, col);
        load_rows<E>(v2, a.V, a.ld, tn, t1, col);
        issued();
        if (!first && cu.live() && nb >= tb + kBlk && tb + kBlk <= t1) {
#pragma unroll
            for (int j = 0; j < kBlk; j++) row(k[j], v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kBlk; j++) {
                const int64_t t = tb + j;
                if (t >= t1) continue;
                if (t >= nb) {
                    cu.forth(t);
                    nb = cu.end();
                    first = cu.live();
                }
                if (first) {
                    first = false;
#pragma unroll
                    for (int i = 0; i < N; i++) A[i] = 0.0f, B[i] = 0.0f;
                    if (a.h0) load_f<N>(a.h0 + cu.cur * a.C + col, B);
                }
                if (cu.live()) row(k[j], v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kBlk; j++) k[j] = k2[j], v[j] = v2[j];
    }
    float *g = a.agg + ch * 2 * a.C + col;
    store_f<N>(g, A);
    store_f<N>(g + a.C, B);
}

// (A, B) applied to h, and the A of (A1, B1) after (A0, B0).  A = 0 forgets
// what came before, whatever it holds.
__device__ inline float apply(float A, float B, float h) { return A == 0.0f ? B : fmaf(A, h, B); }
__device__ inline float compose(float A1, float A0) { return A1 == 0.0f ? 0.0f : A1 * A0; }

// carry[ch] = the state entering chunk ch (REV: chunks in descending order).
// 16 columns x 64 segments of chunks: every thread composes its segment's
// pairs, the segments are scanned by doubling in shared memory, and every
// thread walks its segment again from the state that enters it.
template <bool REV>
__global__ __launch_bounds__(1024) void recur_carry_kernel(RecurArgs a) {
    __shared__ float sA[64][17], sB[64][17];
    const int x = threadIdx.x & 15, y = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + x;
    const bool in = col < a.C;
    const int per = (a.nch + 63) / 64;
    const int i0 = y * per, i1 = i0 + per < a.nch ? i0 + per : a.nch;
    auto ch = [&](int i) { return (int64_t)(REV ? a.nch - 1 - i : i); };
    float A = 1.0f, B = 0.0f;
    if (in)
        for (int i = i0; i < i1; i++) {
            const float *g = a.agg + ch(i) * 2 * a.C + col;
            const float A1 = g[0], B1 = g[a.C];
            B = apply(A1, B1, B);
            A = compose(A1, A);
        }
    sA[y][x] = A;
    sB[y][x] = B;
    __syncthreads();
    for (int d = 1; d < 64; d <<= 1) {
        float A0 = 1.0f, B0 = 0.0f;
        if (y >= d) A0 = sA[y - d][x], B0 = sB[y - d][x];
        __syncthreads();
        if (y >= d) {
            sB[y][x] = apply(sA[y][x], sB[y][x], B0);
            sA[y][x] = compose(sA[y][x], A0);
        }
        __syncthreads();
    }
    float h = y ? sB[y - 1][x] : 0.0f;   // the state before the first chunk is zero
    if (in)
        for (int i = i0; i < i1; i++) {
            const float *g = a.agg + ch(i) * 2 * a.C + col;
            a.carry[ch(i) * a.C + col] = h;
            h = apply(g[0], g[a.C], h);
        }
}

// Y, hT and the checkpoints of a chunk from the state that enters it
template <class E>
__global__ __launch_bounds__(64) void recur_fwd_kernel(RecurArgs a) {
    constexpr int N = E::N;
    using Raw = typename E::Raw;
    int cb;
    int64_t ch;
    wave_pos(a, cb, ch);
    const int col = (cb * 64 + (int)threadIdx.x) * N;
    if (ch >= a.nch) {
        if (a.hT) copy_empty<N>(a, ch - a.nch, col, a.h0, a.hT);
        return;
    }
    if (col >= a.C) return;
    const int64_t t0 = ch * a.L, t1 = t0 + a.L < a.T ? t0 + a.L : a.T;
    Cursor cu{a.off, a.S, a.T, 0};
    cu.seek(t0);
    int64_t nb = cu.end();
    bool first = cu.live() && cu.begin() == t0;
    float h[N] = {};
    if (a.carry) load_f<N>(a.carry + ch * a.C + col, h);
    auto row = [&](Raw kr, Raw vr, Raw rr, int64_t t) {
        float kf[N], vf[N], rf[N], y[N];
        E::unpack(kr, kf);
        E::unpack(vr, vf);
        E::unpack(rr, rf);
#pragma unroll
        for (int i = 0; i < N; i++) {
            h[i] = fmaf(sigmoid(kf[i]), vf[i] - h[i], h[i]);
            y[i] = sigmoid(rf[i]) * h[i];
        }
        *(Raw *)((char *)a.Y + (t * a.ldy + col) * (4 / N)) = E::pack(y);
    };
    Raw k[kBlk], v[kBlk], r[kBlk];
    load_rows<E>(k, a.K, a.ld, t0, t1, col);
    load_rows<E>(v, a.V, a.ld, t0, t1, col);
    load_rows<E>(r, a.R, a.ld, t0, t1, col);
    for (int64_t tb = t0; tb < t1; tb += kBlk) {
        const int64_t tn = tb + kBlk < t1 ? tb + kBlk : tb;
        Raw k2[kBlk], v2[kBlk], r2[kBlk];
        load_rows<E>(k2, a.K, a.ld, tn, t1, col);
        load_rows<E>(v2, a.V, a.ld, tn, t1, col);
        load_rows<E>(r2, a.R, a.ld, tn, t1, col);
        issued();
        if (a.states) store_f<N>(a.states + tb / kBlk * a.C + col, h);
        if (!first && cu.live() && nb > tb + kBlk && tb + kBlk <= t1) {
#pragma unroll
            for (int j = 0; j < kBlk; j++) row(k[j], v[j], r[j], tb + j);
        } else {
#pragma unroll
            for (int j = 0; j < kBlk; j++) {
                const int64_t t = tb + j;
                if (t >= t1) continue;
                if (t >= nb) {
                    cu.forth(t);
                    nb = cu.end();
                    first = cu.live();
                }
                if (first) {
                    first = false;
#pragma unroll
                    for (int i = 0; i < N; i++) h[i] = 0.0f;
                    if (a.h0) load_f<N>(a.h0 + cu.cur * a.C + col, h);
                }
                if (!cu.live()) continue;
                row(k[j], v[j], r[j], t);
                if (a.hT && t + 1 == nb) store_f<N>(a.hT + cu.cur * a.C + col, h);
            }
        }
#pragma unroll
        for (int j = 0; j < kBlk; j++) k[j] = k2[j], v[j] = v2[j], r[j] = r2[j];
    }
}

// dY of one token, in the activations' type or in fp32
template <class E, class D>
__device__ inline void load_dy(const RecurArgs &a, int64_t t, int col, float *f) {
    if constexpr (D::N == E::N) {
        D::unpack(*(const typename D::Raw *)((const char *)a.dY + (t * a.lddy + col) * (4 / D::N)), f);
    } else {
        load_f<E::N>((const float *)a.dY + t * a.lddy + col, f);
    }
}

// (A, B) of a chunk for p_t, in descending token order
template <class E, class D>
__global__ __launch_bounds__(64) void recur_bagg_kernel(RecurArgs a) {
    constexpr int N = E::N;
    int cb;
    int64_t ch;
    wave_pos(a, cb, ch);
    const int col = (cb * 64 + (int)threadIdx.x) * N;
    if (col >= a.C) return;
    const int64_t t0 = ch * a.L, t1 = t0 + a.L < a.T ? t0 + a.L : a.T;
    Cursor cu{a.off, a.S, a.T, 0};
    cu.seek(t1 - 1);
    float A[N], B[N];
#pragma unroll
    for (int i = 0; i < N; i++) A[i] = 1.0f, B[i] = 0.0f;
    bool last = cu.live() && cu.end() == t1;
    int64_t st = cu.begin();
    const int nblk = (int)((t1 - t0 + kBlk - 1) / kBlk);
    for (int b = nblk - 1; b >= 0; b--) {
        const int64_t tb = t0 + (int64_t)b * kBlk;
        const int n = (int)(t1 - tb < kBlk ? t1 - tb : kBlk);
        typename E::Raw k[kBlk], r[kBlk];
        float dy[kBlk][N];
#pragma unroll
        for (int j = 0; j < kBlk; j++) {
            const int64_t t = tb + (j < n ? j : n - 1);
            k[j] = *(const typename E::Raw *)((const char *)a.K + (t * a.ld + col) * (4 / N));
            r[j] = *(const typename E::Raw *)((const char *)a.R + (t * a.ld + col) * (4 / N));
            load_dy<E, D>(a, t, col, dy[j]);
        }
#pragma unroll
        for (int j = kBlk - 1; j >= 0; j--) {
            if (j >= n) continue;
            const int64_t t = tb + j;
            if (t < st) {
                cu.back(t);
                st = cu.begin();
                last = cu.live();
            }
            if (last) {
                last = false;
#pragma unroll
                for (int i = 0; i < N; i++) A[i] = 0.0f, B[i] = 0.0f;
                if (a.dhT) load_f<N>(a.dhT + cu.cur * a.C + col, B);
            }
            if (!cu.live()) continue;
            float kf[N], rf[N];
            E::unpack(k[j], kf);
            E::unpack(r[j], rf);
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float w = sigmoid(kf[i]);
                const float g = fmaf(dy[j][i], sigmoid(rf[i]), B[i]);
                A[i] = fmaf(-w, A[i], A[i]);
                B[i] = fmaf(-w, g, g);
            }
        }
    }
    float *g = a.agg + ch * 2 * a.C + col;
    store_f<N>(g, A);
    store_f<N>(g + a.C, B);
}

// dK, dV, dR and dh0 of a chunk from the gradient that enters it at its end;
// h of each 16-row block is run forward from its checkpoint first
template <class E, class D>
__global__ __launch_bounds__(64) void recur_bwd_kernel(RecurArgs a) {
    constexpr int N = E::N;
    int cb;
    int64_t ch;
    wave_pos(a, cb, ch);
    const int col = (cb * 64 + (int)threadIdx.x) * N;
    if (ch >= a.nch) {
        if (a.dh0) copy_empty<N>(a, ch - a.nch, col, a.dhT, a.dh0);
        return;
    }
    if (col >= a.C) return;
    const int64_t t0 = ch * a.L, t1 = t0 + a.L < a.T ? t0 + a.L : a.T;
    Cursor cu{a.off, a.S, a.T, 0};
    cu.seek(t1 - 1);
    float p[N] = {};
    if (a.carry) load_f<N>(a.carry + ch * a.C + col, p);
    bool last = cu.live() && cu.end() == t1;
    int64_t st = cu.begin();
    const int nblk = (int)((t1 - t0 + kBlk - 1) / kBlk);
    for (int b = nblk - 1; b >= 0; b--) {
        const int64_t tb = t0 + (int64_t)b * kBlk;
        const int n = (int)(t1 - tb < kBlk ? t1 - tb : kBlk);
        typename E::Raw k[kBlk], v[kBlk], r[kBlk];
        float dy[kBlk][N], h[kBlk + 1][N];   // h[j]: the state before row j
        load_f<N>(a.states + tb / kBlk * a.C + col, h[0]);
#pragma unroll
        for (int j = 0; j < kBlk; j++) {
            const int64_t t = tb + (j < n ? j : n - 1);
            const int64_t o = (t * a.ld + col) * (4 / N);
            k[j] = *(const typename E::Raw *)((const char *)a.K + o);
            v[j] = *(const typename E::Raw *)((const char *)a.V + o);
            r[j] = *(const typename E::Raw *)((const char *)a.R + o);
            load_dy<E, D>(a, t, col, dy[j]);
        }
        // forward through the block: the state before every row
        {
            Cursor f = cu;
            f.back(tb);
            int64_t nb = f.end();
            bool first = f.live() && f.begin() == tb;
#pragma unroll
            for (int j = 0; j < kBlk; j++) {
                if (j < n) {
                    if (tb + j >= nb) {
                        f.forth(tb + j);
                        nb = f.end();
                        first = f.live();
                    }
                    if (first) {
                        first = false;
#pragma unroll
                        for (int i = 0; i < N; i++) h[j][i] = 0.0f;
                        if (a.h0) load_f<N>(a.h0 + f.cur * a.C + col, h[j]);
                    }
                }
                float kf[N], vf[N];
                E::unpack(k[j], kf);
                E::unpack(v[j], vf);
#pragma unroll
                for (int i = 0; i < N; i++) h[j + 1][i] = fmaf(sigmoid(kf[i]), vf[i] - h[j][i], h[j][i]);
            }
        }
#pragma unroll
        for (int j = kBlk - 1; j >= 0; j--) {
            if (j >= n) continue;
            const int64_t t = tb + j;
            if (t < st) {
                cu.back(t);
                st = cu.begin();
                last = cu.live();
            }
            if (last) {
                last = false;
#pragma unroll
                for (int i = 0; i < N; i++) p[i] = 0.0f;
                if (a.dhT) load_f<N>(a.dhT + cu.cur * a.C + col, p);
            }
            if (!cu.live()) continue;
            float kf[N], vf[N], rf[N], dk[N], dv[N], dr[N];
            E::unpack(k[j], kf);
            E::unpack(v[j], vf);
            E::unpack(r[j], rf);
#pragma unroll
            for (int i = 0; i < N; i++) {
                float wd, sd;
                const float w = sigmoid_d(kf[i], wd), s = sigmoid_d(rf[i], sd);
                const float g = fmaf(dy[j][i], s, p[i]);
                // the state behind the row from the one before it (a sequence's
                // first row starts from h0, not from the checkpoint's chain)
                const float hb = h[j][i], hn = fmaf(w, vf[i] - hb, hb);
                dr[i] = dy[j][i] * hn * sd;
                dv[i] = g * w;
                dk[i] = g * (vf[i] - hb) * wd;
                p[i] = fmaf(-w, g, g);
            }
            const int64_t o = (t * a.ldd + col) * (4 / N);
            *(typename E::Raw *)((char *)a.dK + o) = E::pack(dk);
            *(typename E::Raw *)((char *)a.dV + o) = E::pack(dv);
            *(typename E::Raw *)((char *)a.dR + o) = E::pack(dr);
            if (a.dh0 && t == st) store_f<N>(a.dh0 + cu.cur * a.C + col, p);
        }
    }
}

// One token of every sequence: a row each, elementwise.
template <class E>
__global__ __launch_bounds__(256) void recur_step_kernel(const void *K, const void *V, const void *R, int64_t ld,
                                                         int64_t rows, int C, const float *h_in, float *h_out, void *Y,
                                                         int64_t ldy) {
    constexpr int N = E::N;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per = C / N;
    const int64_t row = i / per;
    if (row >= rows) return;
    const int col = (int)(i - row * per) * N;
    const int64_t o = (row * ld + col) * (4 / N);
    float k[N], v[N], r[N], h[N], y[N];
    E::unpack(*(const typename E::Raw *)((const char *)K + o), k);
    E::unpack(*(const typename E::Raw *)((const char *)V + o), v);
    E::unpack(*(const typename E::Raw *)((const char *)R + o), r);
    load_f<N>(h_in + row * C + col, h);
#pragma unroll
    for (int j = 0; j < N; j++) {
        h[j] = fmaf(sigmoid(k[j]), v[j] - h[j], h[j]);
        y[j] = sigmoid(r[j]) * h[j];
    }
    store_f<N>(h_out + row * C + col, h);
    *(typename E::Raw *)((char *)Y + (row * ldy + col) * (4 / N)) = E::pack(y);
}

}  // namespace rdev

namespace {

using rdev::RecurArgs;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Chunks: enough waves to fill the chip (16 a compute unit), no shorter than
// a checkpoint block.
struct RecurPlan {
    int64_t ncb, L, nch;
};
RecurPlan plan_recur(int64_t T, int64_t C, int32_t act) {
    RecurPlan p;
    p.ncb = cdiv(C, act == TERN_BF16 ? 128 : 64);
    const int64_t waves = 4096;
    p.L = cdiv(cdiv(T * p.ncb, waves), TERN_RECUR_BLOCK) * TERN_RECUR_BLOCK;
    if (p.L < TERN_RECUR_BLOCK) p.L = TERN_RECUR_BLOCK;
    if (p.L > (1 << 30)) p.L = 1 << 30;
    p.nch = cdiv(T, p.L);
    return p;
}

size_t plan_ws(const RecurPlan &p, int64_t C) { return p.nch <= 1 ? 0 : (size_t)p.nch * (size_t)C * 3 * 4; }

// A strided [rows, cols] buffer (a column slice of a wider one).
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
    size_t es;
    size_t bytes() const { return rows && cols ? ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es : 0; }
};

// Do two strided buffers share an element?  Slices of one matrix (equal row
// strides) interleave: there only the columns count.
bool mats_overlap(const Mat &a, const Mat &b) {
    if (!ranges_overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
    if (a.ld * (int64_t)a.es != b.ld * (int64_t)b.es || a.ld == 0) return true;
    const uint64_t ldb = (uint64_t)a.ld * a.es;
    const uint64_t x = (uint64_t)(uintptr_t)a.p, y = (uint64_t)(uintptr_t)b.p;
    const uint64_t d = y >= x ? (y - x) % ldb : (ldb - (x - y) % ldb) % ldb;   // columns b lies behind a
    return d < (uint64_t)a.cols * a.es || ldb - d < (uint64_t)b.cols * b.es;
}

bool any_overlap(const Mat *outs, int nout, const Mat *ins, int nin) {
    for (int i = 0; i < nout; i++) {
        for (int j = i + 1; j < nout; j++)
            if (mats_overlap(outs[i], outs[j])) return true;
        for (int j = 0; j < nin; j++)
            if (mats_overlap(outs[i], ins[j])) return true;
    }
    return false;
}

bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }
bool act_ok(int32_t dt) { return dt == TERN_F32 || dt == TERN_BF16; }
size_t esize(int32_t dt) { return dt == TERN_BF16 ? 2 : 4; }
int launched() { return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

// sizes, strides and sequence arguments common to forward and backward
int check_sizes(int64_t T, int64_t C, int64_t n_seq, const int64_t *offsets, const int64_t *lds, int nld) {
    if (T < 0 || T > kMaxT || C < 0 || C > kMaxInOut || C % 8 != 0 || n_seq < 0 || n_seq > kMaxT) return TERN_ERR_SHAPE;
    if (!offsets && n_seq != 1) return TERN_ERR_SHAPE;
    for (int i = 0; i < nld; i++)
        if (lds[i] < C || lds[i] % 8 != 0 || lds[i] > kMaxInOut * 8) return TERN_ERR_SHAPE;
    return TERN_OK;
}

dim3 grid_of(int64_t n) { return dim3((unsigned)n); }
// a launch counts its threads in 32 bits
bool grid_fits(int64_t blocks, int64_t threads) { return blocks <= INT64_C(0xFFFFFFFF) / threads; }

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

size_t tern_recur_states_bytes(int64_t T, int64_t C) {
    if (T < 0 || T > kMaxT || C < 0 || C > kMaxInOut || C % 8 != 0) return 0;
    return (size_t)cdiv(T, TERN_RECUR_BLOCK) * (size_t)C * 4;
}

size_t tern_recur_workspace_bytes(int64_t T, int64_t C) {
    if (T < 0 || T > kMaxT || C < 0 || C > kMaxInOut || C % 8 != 0) return 0;
    const size_t a = plan_ws(plan_recur(T, C, TERN_BF16), C), b = plan_ws(plan_recur(T, C, TERN_F32), C);
    return ((a > b ? a : b) + 255) & ~size_t(255);
}

int tern_recur_fwd(const void *K, const void *V, const void *R, int64_t ld, int32_t act_dtype, const float *h0,
                   const int64_t *offsets, int64_t n_seq, int64_t T, int64_t C, void *Y, int64_t ldy, float *hT,
                   float *states, void *workspace, size_t workspace_bytes, void *stream) {
    const int64_t lds[] = {ld, ldy};
    int rc = check_sizes(T, C, n_seq, offsets, lds, 2);
    if (rc) return rc;
    if (!act_ok(act_dtype)) return TERN_ERR_DTYPE;
    const bool tok = T > 0 && C > 0;
    if (tok && (!K || !V || !R || !Y)) return TERN_ERR_NULL;
    const RecurPlan p = plan_recur(T, C, act_dtype);
    const size_t wsb = plan_ws(p, C);
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (misaligned(K) || misaligned(V) || misaligned(R) || misaligned(Y) || misaligned(h0) || misaligned(hT) ||
        misaligned(states) || misaligned(workspace) || ((uintptr_t)offsets & 7u))
        return TERN_ERR_ALIGN;
    const size_t es = esize(act_dtype);
    const Mat outs[] = {{Y, T, C, ldy, es},
                        {hT, n_seq, C, C, 4},
                        {states, cdiv(T, TERN_RECUR_BLOCK), C, C, 4},
                        {workspace, 1, (int64_t)wsb, (int64_t)wsb, 1}};
    const Mat ins[] = {{K, T, C, ld, es}, {V, T, C, ld, es}, {R, T, C, ld, es}, {h0, n_seq, C, C, 4},
                       {offsets, 1, n_seq + 1, n_seq + 1, 8}};
    if (any_overlap(outs, 4, ins, 5)) return TERN_ERR_ALIAS;
    const int64_t empties = hT ? cdiv(n_seq, 64) : 0;
    if (C == 0 || (p.nch + empties) == 0) return TERN_OK;
    if (!grid_fits(p.ncb * (p.nch + empties), 64)) return TERN_ERR_SHAPE;
    RecurArgs a{};
    a.K = K; a.V = V; a.R = R; a.ld = ld; a.h0 = h0; a.off = offsets; a.S = n_seq; a.T = T;
    a.C = (int)C; a.ncb = (int)p.ncb; a.L = (int)p.L; a.nch = (int)p.nch;
    a.Y = Y; a.ldy = ldy; a.hT = hT; a.states = states;
    a.agg = (float *)workspace;
    a.carry = wsb ? (float *)workspace + (size_t)p.nch * 2 * C : nullptr;
    hipStream_t st = (hipStream_t)stream;
    const bool bf = act_dtype == TERN_BF16;
    const dim3 g1 = grid_of(p.ncb * p.nch), g3 = grid_of(p.ncb * (p.nch + empties));
    if (a.carry) {
        if (bf) hipLaunchKernelGGL(rdev::recur_agg_kernel<rdev::Bf>, g1, dim3(64), 0, st, a);
        else hipLaunchKernelGGL(rdev::recur_agg_kernel<rdev::Fp>, g1, dim3(64), 0, st, a);
        hipLaunchKernelGGL(rdev::recur_carry_kernel<false>, grid_of(cdiv(C, 16)), dim3(1024), 0, st, a);
    }
    if (bf) hipLaunchKernelGGL(rdev::recur_fwd_kernel<rdev::Bf>, g3, dim3(64), 0, st, a);
    else hipLaunchKernelGGL(rdev::recur_fwd_kernel<rdev::Fp>, g3, dim3(64), 0, st, a);
    return launched();
}

int tern_recur_bwd(const void *K, const void *V, const void *R, int64_t ld, int32_t act_dtype, const float *h0,
                   const int64_t *offsets, int64_t n_seq, int64_t T, int64_t C, const float *states, const void *dY,
                   int64_t lddy, int32_t dy_dtype, const float *dhT, void *dK, void *dV, void *dR, int64_t ldd,
                   float *dh0, void *workspace, size_t workspace_bytes, void *stream) {
    const int64_t lds[] = {ld, lddy, ldd};
    int rc = check_sizes(T, C, n_seq, offsets, lds, 3);
    if (rc) return rc;
    if (!act_ok(act_dtype) || !(dy_dtype == TERN_F32 || dy_dtype == act_dtype)) return TERN_ERR_DTYPE;
    const bool tok = T > 0 && C > 0;
    if (tok && (!K || !V || !R || !states || !dY || !dK || !dV || !dR)) return TERN_ERR_NULL;
    const RecurPlan p = plan_recur(T, C, act_dtype);
    const size_t wsb = plan_ws(p, C);
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (misaligned(K) || misaligned(V) || misaligned(R) || misaligned(h0) || misaligned(states) || misaligned(dY) ||
        misaligned(dhT) || misaligned(dK) || misaligned(dV) || misaligned(dR) || misaligned(dh0) ||
        misaligned(workspace) || ((uintptr_t)offsets & 7u))
        return TERN_ERR_ALIGN;
    const size_t es = esize(act_dtype);
    const Mat outs[] = {{dK, T, C, ldd, es}, {dV, T, C, ldd, es}, {dR, T, C, ldd, es}, {dh0, n_seq, C, C, 4},
                        {workspace, 1, (int64_t)wsb, (int64_t)wsb, 1}};
    const Mat ins[] = {{K, T, C, ld, es}, {V, T, C, ld, es}, {R, T, C, ld, es}, {h0, n_seq, C, C, 4},
                       {offsets, 1, n_seq + 1, n_seq + 1, 8}, {states, cdiv(T, TERN_RECUR_BLOCK), C, C, 4},
                       {dY, T, C, lddy, esize(dy_dtype)}, {dhT, n_seq, C, C, 4}};
    if (any_overlap(outs, 5, ins, 8)) return TERN_ERR_ALIAS;
    const int64_t empties = dh0 ? cdiv(n_seq, 64) : 0;
    if (C == 0 || (p.nch + empties) == 0) return TERN_OK;
    if (!grid_fits(p.ncb * (p.nch + empties), 64)) return TERN_ERR_SHAPE;
    RecurArgs a{};
    a.K = K; a.V = V; a.R = R; a.ld = ld; a.h0 = h0; a.off = offsets; a.S = n_seq; a.T = T;
    a.C = (int)C; a.ncb = (int)p.ncb; a.L = (int)p.L; a.nch = (int)p.nch;
    a.states = const_cast<float *>(states);
    a.dY = dY; a.lddy = lddy; a.dhT = dhT; a.dK = dK; a.dV = dV; a.dR = dR; a.ldd = ldd; a.dh0 = dh0;
    a.agg = (float *)workspace;
    a.carry = wsb ? (float *)workspace + (size_t)p.nch * 2 * C : nullptr;
    hipStream_t st = (hipStream_t)stream;
    const dim3 g1 = grid_of(p.ncb * p.nch), g3 = grid_of(p.ncb * (p.nch + empties)), b(64);
    const int form = act_dtype == TERN_F32 ? 2 : dy_dtype == TERN_F32 ? 1 : 0;
    if (a.carry) {
        if (form == 0) hipLaunchKernelGGL((rdev::recur_bagg_kernel<rdev::Bf, rdev::Bf>), g1, b, 0, st, a);
        else if (form == 1) hipLaunchKernelGGL((rdev::recur_bagg_kernel<rdev::Bf, rdev::Fp>), g1, b, 0, st, a);
        else hipLaunchKernelGGL((rdev::recur_bagg_kernel<rdev::Fp, rdev::Fp>), g1, b, 0, st, a);
        hipLaunchKernelGGL(rdev::recur_carry_kernel<true>, grid_of(cdiv(C, 16)), dim3(1024), 0, st, a);
    }
    if (form == 0) hipLaunchKernelGGL((rdev::recur_bwd_kernel<rdev::Bf, rdev::Bf>), g3, b, 0, st, a);
    else if (form == 1) hipLaunchKernelGGL((rdev::recur_bwd_kernel<rdev::Bf, rdev::Fp>), g3, b, 0, st, a);
    else hipLaunchKernelGGL((rdev::recur_bwd_kernel<rdev::Fp, rdev::Fp>), g3, b, 0, st, a);
    return launched();
}

int tern_recur_step(const void *K, const void *V, const void *R, int64_t ld, int32_t act_dtype, int64_t rows,
                    int64_t C, const float *h, float *h_out, void *Y, int64_t ldy, void *stream) {
    if (rows < 0 || rows > kMaxT || C < 0 || C > kMaxInOut || C % 8 != 0) return TERN_ERR_SHAPE;
    if (ld < C || ld % 8 != 0 || ld > kMaxInOut * 8 || ldy < C || ldy % 8 != 0 || ldy > kMaxInOut * 8)
        return TERN_ERR_SHAPE;
    if (!act_ok(act_dtype)) return TERN_ERR_DTYPE;
    if (rows == 0 || C == 0) return TERN_OK;
    if (!K || !V || !R || !h || !h_out || !Y) return TERN_ERR_NULL;
    if (misaligned(K) || misaligned(V) || misaligned(R) || misaligned(h) || misaligned(h_out) || misaligned(Y))
        return TERN_ERR_ALIGN;
    const size_t es = esize(act_dtype);
    const Mat outs[] = {{Y, rows, C, ldy, es}, {h_out, rows, C, C, 4}};
    // every lane reads its state before it writes it, so h_out may be h itself
    const Mat ins[] = {{K, rows, C, ld, es}, {V, rows, C, ld, es}, {R, rows, C, ld, es},
                       {h == h_out ? nullptr : h, rows, C, C, 4}};
    if (any_overlap(outs, 2, ins, 4)) return TERN_ERR_ALIAS;
    const bool bf = act_dtype == TERN_BF16;
    const int64_t n = cdiv(rows * (C / (bf ? 2 : 1)), 256);
    if (!grid_fits(n, 256)) return TERN_ERR_SHAPE;
    hipStream_t st = (hipStream_t)stream;
    if (bf)
        hipLaunchKernelGGL(rdev::recur_step_kernel<rdev::Bf>, grid_of(n), dim3(256), 0, st, K, V, R, ld, rows, (int)C,
                           h, h_out, Y, ldy);
    else
        hipLaunchKernelGGL(rdev::recur_step_kernel<rdev::Fp>, grid_of(n), dim3(256), 0, st, K, V, R, ld, rows, (int)C,
                           h, h_out, Y, ldy);
    return launched();
}

}  // extern "C"
