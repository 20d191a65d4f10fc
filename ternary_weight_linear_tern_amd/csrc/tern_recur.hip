// tern_recur.hip -- the gated linear recurrence between the receptance, key
// and value projections and the output projection (C ABI in include/tern.h).
//
//   w_t = sigmoid(k_t)          h_t = h_{t-1} + w_t (v_t - h_{t-1})
//   s_t = sigmoid(r_t)          y_t = s_t h_t
//
// per channel, over packed sequences.  A step multiplies by the smaller of the
// two gates, w and the kept share 1 - w = sigmoid(-k), from whichever end it is:
// h + w (v - h) or v + (1 - w) (h - v).  So a gate near 0 (a long memory) keeps its
// relative accuracy, and of a gate near 1 neither the little that is kept nor a
// value much smaller than the state it replaces is lost.  All states, gradients
// and sums are fp32.
//
// A step is an affine map of the state, h -> (1 - w) h + w v, and affine maps
// compose to affine maps (A, B): h -> A h + B.  So the T tokens (the packed
// sequences laid end to end) are cut into chunks of a workgroup, 16 rows a wave,
// and one pass over the data does:
//   - every wave loads its rows into registers and composes their pair;
//   - the workgroup publishes the chunk's pair, and finds the state that enters
//     the chunk from the nearest chunk before it whose closing state is known
//     and the pairs in between;
//   - it publishes its own closing state, and every wave walks its rows again
//     in registers, from the state that enters them, and writes Y.
// K, V, R are read once and Y is written once: 32768 x 4096 bf16 in one sequence
// 305 us, 3.5 TB/s of the 5.1 of a copy; backward, with fp32 dY, 590 us, 3.6 TB/s.
// (With w as every step's factor, which loses what an open gate keeps, 289 and 560;
// so, with the pairs, the chain and the output in three launches, which read K and V
// twice, the forward took 345.)  What bounds it is the time a chunk's registers are
// held: the loads, about 3 us for the words of other chunks, the output.  Short
// calls (2048 x 512: 12 us) are two launches and one such chunk's time.
// The pairs in between are applied in order to the state found, the same
// operations whichever chunk that was: results do not depend on timing.
// A sequence's first token drops what came before: the composition restarts
// there with A = 0 and B = h0, and a pair with A = 0 returns B without
// multiplying, so nothing of one sequence (a NaN, an infinity) reaches the
// next.
//
// Backward, with u_t = dy_t s_t and g_t the gradient that reaches h_t:
//   g_t = u_t + (1 - w_{t+1}) g_{t+1}   (+ dhT behind the last token)
//   dv = g w,  dk = g (v - h_{t-1}) w (1 - w),  dr = dy h s (1 - s)
// p_t = (1 - w_t) g_t, the gradient of h_{t-1}, is again an affine chain, run
// from the last token to the first, through the same chunks in reverse.  The
// states h_{t-1} come from the forward's checkpoints (one row every 16 tokens).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

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
    int nch;                   // chunks
    unsigned wgs;              // workgroups that take chunks
    void *Y;                   // [T, C], row stride ldy
    int64_t ldy;
    float *hT;                 // [S, C] or null
    float *states;             // [ceil(T / 16), C]: the state before each 16-row block
    unsigned long long *agg;   // [nch][C]: pairs of the chunks, in chain order
    uint32_t *prefix;          // [nch][C]: states behind the chunks
    uint32_t *ticket;          // [ncb], 128 bytes apart
    const void *dY;            // [T, C], row stride lddy
    int64_t lddy;
    const float *dhT;          // [S, C] or null (zeros)
    void *dK, *dV, *dR;        // [T, C], row stride ldd
    int64_t ldd;
    float *dh0;                // [S, C] or null
};

// One lane's channels of a row: N of ES bytes.
__device__ inline uint32_t round_bf16(float f) {   // to nearest even (NaN stays NaN)
    return __builtin_bit_cast(unsigned short, (__bf16)f);
}
struct Bf {
    static constexpr int N = 2, ES = 2;
    using Raw = uint32_t;
    __device__ static void unpack(Raw x, float *f) {
        f[0] = __builtin_bit_cast(float, x << 16);
        f[1] = __builtin_bit_cast(float, x & 0xFFFF0000u);
    }
    __device__ static Raw pack(const float *f) { return round_bf16(f[0]) | round_bf16(f[1]) << 16; }
};
struct Bh {
    static constexpr int N = 1, ES = 2;
    using Raw = uint16_t;
    __device__ static void unpack(Raw x, float *f) { f[0] = __builtin_bit_cast(float, (uint32_t)x << 16); }
    __device__ static Raw pack(const float *f) { return (Raw)round_bf16(f[0]); }
};
struct Fp {
    static constexpr int N = 1, ES = 4;
    using Raw = float;
    __device__ static void unpack(Raw x, float *f) { f[0] = x; }
    __device__ static Raw pack(const float *f) { return f[0]; }
};

// a lane's channels of an fp32 row (8-byte aligned where there are two)
template <int N>
__device__ inline void load_f(const float *p, float *f) {
    if constexpr (N == 2) {
        const float2 v = *(const float2 *)p;
        f[0] = v.x, f[1] = v.y;
    } else {
        f[0] = *p;
    }
}
template <int N>
__device__ inline void store_f(float *p, const float *f) {
    if constexpr (N == 2) *(float2 *)p = float2{f[0], f[1]};
    else *p = f[0];
}

__device__ inline float exp_neg(float x) { return __builtin_amdgcn_exp2f(x * -1.44269504088896340736f); }
__device__ inline float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_neg(x)); }

// The smaller of sigmoid(x) and sigmoid(-x), negative (by its sign bit) where
// that is sigmoid(x): neither is made by a difference, which would cancel where
// the gate saturates.
__device__ inline float smaller(float x) {
    const float e = exp_neg(fabsf(x));
    return __builtin_copysignf(e * __builtin_amdgcn_rcpf(1.0f + e), x);
}
__device__ inline bool is_write(float g) { return __builtin_bit_cast(int, g) < 0; }
// a step of the state, and the kept share of x, by the smaller gate
__device__ inline float step(float g, float h, float v) { return fmaf(-g, v - h, is_write(g) ? h : v); }
__device__ inline float keep(float g, float x) { return fmaf(g, x, is_write(g) ? x : 0.0f); }

// sigmoid(x) and sigmoid(-x)
__device__ inline void gates(float x, float &on, float &off) {
    const float e = exp_neg(fabsf(x)), i = __builtin_amdgcn_rcpf(1.0f + e), j = e * i;
    on = x < 0.0f ? j : i;
    off = x < 0.0f ? i : j;
}

// A cursor among the rows from t0 on, with its sequence's borders as rows
// relative to t0 (clamped to [-1, 32]): comparing them costs one instruction a
// row, and the offsets in memory are read only where a border is crossed.
struct Span {
    Cursor c;
    int64_t t0;
    int b, e;
    bool live;
    __device__ int row_of(int64_t t) const { return t <= t0 - 1 ? -1 : t >= t0 + 32 ? 32 : (int)(t - t0); }
    __device__ void look() {
        b = row_of(c.begin());
        e = row_of(c.end());
        live = c.live();
    }
    __device__ Span(const RecurArgs &a, int64_t first) : c{a.off, a.S, a.T, 0}, t0(first) {
        c.seek(first);
        look();
    }
    __device__ void forth(int j) {
        if (j < e) return;
        c.forth(t0 + j);
        look();
    }
    __device__ void back(int j) {
        if (j >= b) return;
        c.back(t0 + j);
        look();
    }
};

// The rows of one checkpoint block (rows beyond the chunk's end repeat its
// last one), all loads issued together.
// A row's address is uniform in a wave, and lanes add 32 bits to it: that keeps
// the addresses of 16 rows out of the vector registers.
template <class T>
__device__ inline T *at_row(T *p, int64_t row, int64_t ld, int es, uint32_t lane_bytes) {
    using C = std::conditional_t<std::is_const_v<T>, const char, char>;
    return (T *)((C *)p + row * ld * es + lane_bytes);
}
template <class E>
__device__ inline void load_rows(typename E::Raw *x, const void *p, int64_t ld, int64_t tb, int64_t t1, uint32_t lane) {
#pragma unroll
    for (int j = 0; j < kBlk; j++)
        x[j] = *(const typename E::Raw *)at_row(p, tb + j < t1 ? tb + j : t1 - 1, ld, E::ES, lane);
}
template <class E>
__device__ inline void store_row(void *p, int64_t row, int64_t ld, uint32_t lane, const float *f) {
    *(typename E::Raw *)at_row(p, row, ld, E::ES, lane) = E::pack(f);
}

// Sequences without tokens pass their state through: dst[s] = src[s].
template <int N>
__device__ inline void copy_empty(const RecurArgs &a, int64_t group, int col, const float *src, float *dst) {
    const int64_t s = group * 64 + (threadIdx.x & 63);
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

// (A, B) applied to h, and the A of (A1, B1) after (A0, B0).  A = 0 means that a
// sequence starts among the rows, and forgets what came before, whatever it
// holds.  Without a start A stays above 0 where the product of the kept shares
// would reach it, so that a NaN or an infinity goes on to its sequence's end as it
// does token by token (a finite state adds 1e-45 of itself).
constexpr float kTiny = 1.401298464e-45f;
__device__ inline float kept(float A, bool restart) { return restart ? 0.0f : fmaxf(A, kTiny); }
__device__ inline float apply(float A, float B, float h) { return A == 0.0f ? B : fmaf(A, h, B); }
__device__ inline float compose(float A1, float A0) { return kept(A1 * A0, A1 == 0.0f || A0 == 0.0f); }

// ---------------------------------------------------------------------------
// The chain of chunks.  A pair (A, B) and a state are published as one 64-bit
// and one 32-bit word that validate themselves: the workspace is filled with
// ones beforehand (recur_init), and a value that would be all ones is stored
// as another NaN.  The words are written and read past the XCDs' L2 caches
// (agent scope), each by one access; nothing else has to be ordered with them.
//
// Workgroups take their chunk of a column block from a counter, in chain
// order, so whoever waits for an earlier chunk waits for a workgroup that runs
// already; that one publishes its pair before it waits for anything, and the
// first chunk waits for nothing: every wait ends.  Two calls at once that share
// a workspace against the rules wipe each other's words and tickets: a ticket
// past the last chunk has no work, and a wait gives up after a few seconds and
// goes on with a NaN.
// ---------------------------------------------------------------------------

constexpr uint32_t kEmpty = 0xFFFFFFFFu;
constexpr int kTicketStride = 32;   // words
constexpr int kBack = 16;           // chunks looked back over
constexpr int kPatience = 1 << 21;  // looks at other chunks' words, each above 1 us

__device__ inline uint32_t word_of(float x) {
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    return w == kEmpty ? 0x7FC00000u : w;
}
__device__ inline void publish_pair(unsigned long long *p, float A, float B) {
    __hip_atomic_store(p, (unsigned long long)word_of(A) | (unsigned long long)__builtin_bit_cast(uint32_t, B) << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void publish_state(uint32_t *p, float h) {
    __hip_atomic_store(p, word_of(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline unsigned long long pair_at(const unsigned long long *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint32_t state_at(const uint32_t *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__global__ __launch_bounds__(256) void recur_init_kernel(uint4 *empty, int64_t n16, uint32_t *ticket, int ncb) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n16) empty[i] = uint4{kEmpty, kEmpty, kEmpty, kEmpty};
    if (i < ncb) ticket[i * kTicketStride] = 0;
}

// Lanes 0 .. 15 watch one column of the 16 chunks before chunk i until one has
// its state and all chunks after that their pairs, or until `looks` reaches the
// limit.
__device__ inline void watch(const RecurArgs &a, int i, int col0, int &looks) {
    const int lane = threadIdx.x & 63, p = i - 1 - lane;
    while (looks++ < kPatience) {
        bool has_state = lane < kBack && p < 0, has_pair = false;   // before the first chunk the state is zero
        if (lane < kBack && p >= 0) {
            has_state = state_at(a.prefix + (int64_t)p * a.C + col0) != kEmpty;
            has_pair = (uint32_t)pair_at(a.agg + (int64_t)p * a.C + col0) != kEmpty;
        }
        const uint32_t states = (uint32_t)__ballot(has_state), pairs = (uint32_t)__ballot(has_pair);
        const int d = states ? __builtin_ctz(states) : kBack;   // chunks in between
        if (d < kBack && (~pairs & ((1u << d) - 1)) == 0) return;
        __builtin_amdgcn_s_sleep(1);
    }
}

// The state that enters each wave's rows; `order` is the wave's place in the
// chain.  The waves' pairs meet in shared memory; the first wave composes and
// publishes the chunk's.  A chunk in which a sequence starts (A = 0) closes with
// the state B whatever enters it, and publishes that at once; one that begins
// with a sequence's start (`fresh`) needs no state at all.  Work that does not
// need the state is done in `between`, while the other chunks' words arrive.
// Then all waves fetch the words of the 16 chunks before
// (one trip to memory), the first finds the state before the chunk in them and
// publishes the one behind it.
template <int N, int W, class Between>
__device__ inline void enter(const RecurArgs &a, int i, int order, bool fresh, int col, int col0, float *A, float *B,
                             float *h, Between between) {
    constexpr int J = kBack / W;   // chunks a wave fetches
    __shared__ float sA[W][64 * N], sB[W][64 * N], sH[64 * N];
    __shared__ unsigned long long sPair[kBack][64 * N];
    __shared__ uint32_t sState[kBack][64 * N];
    __shared__ int sKnown, sClosed, sHas[kBack];
    const int at = (threadIdx.x & 63) * N;
    store_f<N>(&sA[order][at], A);
    store_f<N>(&sB[order][at], B);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; k++) h[k] = 0.0f;
    if (a.nch > 1) {
        if (order == 0) {
#pragma unroll
            for (int q = 1; q < W; q++)
#pragma unroll
                for (int k = 0; k < N; k++) {
                    const float A1 = sA[q][at + k];
                    B[k] = apply(A1, sB[q][at + k], B[k]);
                    A[k] = compose(A1, A[k]);
                }
            bool closed = true;
#pragma unroll
            for (int k = 0; k < N; k++) closed = closed && A[k] == 0.0f;
            closed = i == 0 || fresh || __ballot(col < a.C && !closed) == 0;
            if (col < a.C)
#pragma unroll
                for (int k = 0; k < N; k++) {
                    if (closed) publish_state(a.prefix + (int64_t)i * a.C + col + k, apply(A[k], B[k], 0.0f));
                    else publish_pair(a.agg + (int64_t)i * a.C + col + k, A[k], B[k]);
                }
            sClosed = closed;
            sKnown = i == 0 || fresh;
            store_f<N>(&sH[at], h);   // zero; a fresh chunk does not use it
        }
        __syncthreads();
    }
    between();
    if (a.nch > 1) {
        // lanes past the last column take part with the last ones
        const int c = col < a.C ? col : a.C - N;
        int looks = 0;
        for (bool first = true; !sKnown; first = false) {
            if (!first) watch(a, i, col0, looks);
            unsigned long long pr[J][N];
            uint32_t st[J][N];
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int p = i - 1 - (order * J + j);
#pragma unroll
                for (int k = 0; k < N; k++) {
                    pr[j][k] = p < 0 ? 0 : pair_at(a.agg + (int64_t)p * a.C + c + k);
                    st[j][k] = p < 0 ? 0 : state_at(a.prefix + (int64_t)p * a.C + c + k);
                }
            }
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int d = order * J + j;
                bool has_state = true, has_pair = true;
#pragma unroll
                for (int k = 0; k < N; k++) {
                    sPair[d][at + k] = pr[j][k];
                    sState[d][at + k] = st[j][k];
                    has_state = has_state && st[j][k] != kEmpty;
                    has_pair = has_pair && (uint32_t)pr[j][k] != kEmpty;
                }
                const uint64_t no_state = __ballot(!has_state), no_pair = __ballot(!has_pair);
                if ((threadIdx.x & 63) == 0) sHas[d] = (no_state == 0) | (no_pair == 0) << 1;
            }
            __syncthreads();
            if (order == 0) {
                // the nearest chunk whose state is there for every column, and
                // the pairs of those behind it
                const int has = sHas[threadIdx.x & (kBack - 1)];
                const uint32_t states = (uint32_t)__ballot(has & 1) & ((1u << kBack) - 1);
                const uint32_t pairs = (uint32_t)__ballot(has & 2);
                const int from = states ? __builtin_ctz(states) : kBack;
                const bool all = from < kBack && (~pairs & ((1u << from) - 1)) == 0;
                if (all) {
#pragma unroll
                    for (int k = 0; k < N; k++) h[k] = __builtin_bit_cast(float, sState[from][at + k]);
#pragma unroll 4
                    for (int d = from - 1; d >= 0; d--)
#pragma unroll
                        for (int k = 0; k < N; k++) {
                            const unsigned long long pr = sPair[d][at + k];
                            h[k] = apply(__builtin_bit_cast(float, (uint32_t)pr),
                                         __builtin_bit_cast(float, (uint32_t)(pr >> 32)), h[k]);
                        }
                }
                const bool done = all || looks >= kPatience;
                if (!all)
#pragma unroll
                    for (int k = 0; k < N; k++) h[k] = __builtin_nanf("");
                if (done && !sClosed && col < a.C)
#pragma unroll
                    for (int k = 0; k < N; k++)
                        publish_state(a.prefix + (int64_t)i * a.C + col + k, apply(A[k], B[k], h[k]));
                if (done) store_f<N>(&sH[at], h);
                sKnown = done;
            }
            __syncthreads();
        }
        load_f<N>(&sH[at], h);
    }
    for (int q = 0; q < order; q++)
#pragma unroll
        for (int k = 0; k < N; k++) h[k] = apply(sA[q][at + k], sB[q][at + k], h[k]);
}

// The workgroup's next place in its column block's chain
__device__ inline int take_ticket(const RecurArgs &a, int cb) {
    __shared__ int t;
    if (a.nch == 1) return 0;
    if (threadIdx.x == 0)
        t = (int)__hip_atomic_fetch_add(a.ticket + cb * kTicketStride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(t);
}

template <class E, int W>
__device__ inline void fwd_chunk(const RecurArgs &a, int cb, int col, int wave, int ch) {
    constexpr int N = E::N;
    using Raw = typename E::Raw;
    const uint32_t lb = (uint32_t)col * E::ES;
    const int64_t t0 = ((int64_t)ch * W + wave) * kBlk, t1 = t0 + kBlk < a.T ? t0 + kBlk : a.T;
    const bool on = col < a.C && t0 < a.T;
    float w[kBlk][N];
    Raw k[kBlk], v[kBlk], r[kBlk];
    if (on) {
        load_rows<E>(k, a.K, a.ld, t0, t1, lb);
        load_rows<E>(v, a.V, a.ld, t0, t1, lb);
        load_rows<E>(r, a.R, a.ld, t0, t1, lb);
    }
    // the search among the offsets runs while the rows arrive
    Span at(a, t0);
    // the rows are all there and one sequence's, whose first they may be
    const int n = (int)(t1 - t0);   // rows
    const bool whole = at.live && at.e >= kBlk && n == kBlk, begins = whole && at.b == 0;
    float start[N] = {};
    if (begins && on && a.h0) load_f<N>(a.h0 + at.c.cur * a.C + col, start);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < kBlk; j++) {
        float kf[N];
        E::unpack(k[j], kf);
#pragma unroll
        for (int i = 0; i < N; i++) w[j][i] = smaller(kf[i]);
    }
    float A[N], B[N], h[N];
#pragma unroll
    for (int i = 0; i < N; i++) A[i] = 1.0f, B[i] = 0.0f;
    bool restart = false;
    if (on) {
        auto row = [&](int j) {
            float vf[N];
            E::unpack(v[j], vf);
#pragma unroll
            for (int i = 0; i < N; i++) {
                A[i] = keep(w[j][i], A[i]);
                B[i] = step(w[j][i], B[i], vf[i]);
            }
        };
        if (whole) {
            restart = begins;
            if (begins)
#pragma unroll
                for (int i = 0; i < N; i++) B[i] = start[i];
#pragma unroll
            for (int j = 0; j < kBlk; j++) row(j);
        } else {
            Span s = at;
#pragma unroll
            for (int j = 0; j < kBlk; j++) {
                if (j >= n) continue;
                s.forth(j);
                if (!s.live) continue;
                if (j == s.b) {
                    restart = true;
#pragma unroll
                    for (int i = 0; i < N; i++) B[i] = 0.0f;
                    if (a.h0) load_f<N>(a.h0 + s.c.cur * a.C + col, B);
                }
                row(j);
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++) A[i] = kept(A[i], restart);
    }
    // the first wave's answer counts: does the chunk begin with a sequence's start?
    enter<N, W>(a, ch, wave, at.b == 0, col, cb * 64 * N, A, B, h, [] {});
    if (!on) return;
    if (a.states) store_f<N>((float *)at_row(a.states, t0 / kBlk, a.C, 4, (uint32_t)col * 4), h);
    auto row = [&](int j) {
        float vf[N], rf[N], o[N];
        E::unpack(v[j], vf);
        E::unpack(r[j], rf);
#pragma unroll
        for (int i = 0; i < N; i++) {
            h[i] = step(w[j][i], h[i], vf[i]);
            o[i] = sigmoid(rf[i]) * h[i];
        }
        store_row<E>(a.Y, t0 + j, a.ldy, lb, o);
    };
    if (whole) {
        if (begins)
#pragma unroll
            for (int i = 0; i < N; i++) h[i] = start[i];
#pragma unroll
        for (int j = 0; j < kBlk; j++) row(j);
        if (a.hT && at.e == kBlk) store_f<N>(a.hT + at.c.cur * a.C + col, h);
    } else {
#pragma unroll
        for (int j = 0; j < kBlk; j++) {
            if (j >= n) continue;
            at.forth(j);
            if (!at.live) continue;
            if (j == at.b) {
#pragma unroll
                for (int i = 0; i < N; i++) h[i] = 0.0f;
                if (a.h0) load_f<N>(a.h0 + at.c.cur * a.C + col, h);
            }
            row(j);
            if (a.hT && j + 1 == at.e) store_f<N>(a.hT + at.c.cur * a.C + col, h);
        }
    }
}

// A workgroup for every chunk; behind those, one for every column block and 64
// sequences passes on the empty ones' states.
template <class E, int W>
__global__ __launch_bounds__(64 * W, 4) void recur_fwd_kernel(RecurArgs a) {
    const int b = blockIdx.x < a.wgs ? blockIdx.x : blockIdx.x - a.wgs, cb = b % a.ncb;
    const int col = (cb * 64 + (int)(threadIdx.x & 63)) * E::N;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x >= a.wgs) {
        if (wave == 0) copy_empty<E::N>(a, b / a.ncb, col, a.h0, a.hT);
        return;
    }
    const int i = take_ticket(a, cb);
    if (i < a.nch) fwd_chunk<E, W>(a, cb, col, wave, i);
}

// dY of one token, in the activations' type (D = E) or in fp32
template <class E, class D>
struct Grad {
    using Raw = std::conditional_t<std::is_same_v<D, E>, typename E::Raw, std::conditional_t<E::N == 2, float2, float>>;
    Raw x;
    __device__ void load(const RecurArgs &a, int64_t t, int col) {
        x = *(const Raw *)at_row(a.dY, t, a.lddy, D::ES, (uint32_t)col * D::ES);
    }
    __device__ void get(float *f) const {
        if constexpr (std::is_same_v<D, E>) E::unpack(x, f);
        else __builtin_memcpy(f, &x, sizeof x);
    }
};

template <class E, class D, int W>
__device__ inline void bwd_chunk(const RecurArgs &a, int cb, int col, int wave, int link) {
    constexpr int N = E::N;
    using Raw = typename E::Raw;
    const uint32_t lb = (uint32_t)col * E::ES;
    const int64_t t0 = ((int64_t)(a.nch - 1 - link) * W + wave) * kBlk, t1 = t0 + kBlk < a.T ? t0 + kBlk : a.T;
    const bool on = col < a.C && t0 < a.T;
    Raw k[kBlk], v[kBlk], r[kBlk];
    Grad<E, D> dy[kBlk];
    float h[N] = {};
    if (on) {
        load_rows<E>(k, a.K, a.ld, t0, t1, lb);
        load_rows<E>(r, a.R, a.ld, t0, t1, lb);
#pragma unroll
        for (int j = 0; j < kBlk; j++) dy[j].load(a, t0 + j < t1 ? t0 + j : t1 - 1, col);
        load_rows<E>(v, a.V, a.ld, t0, t1, lb);
        load_f<N>((float *)at_row(a.states, t0 / kBlk, a.C, 4, (uint32_t)col * 4), h);
    }
    Span at(a, t0);
    // the rows are all there and one sequence's, whose first and last they may hold
    const int n = (int)(t1 - t0);   // rows
    const bool whole = at.live && at.e >= kBlk && n == kBlk, begins = whole && at.b == 0,
               ends = whole && at.e == kBlk;
    float stop[N] = {};
    if (on && begins) {
        h[0] = h[N - 1] = 0.0f;
        if (a.h0) load_f<N>(a.h0 + at.c.cur * a.C + col, h);
    }
    if (on && ends && a.dhT) load_f<N>(a.dhT + at.c.cur * a.C + col, stop);
    Span last = at;   // at the last row
    if (on && !whole) last.forth(n - 1);
    __builtin_amdgcn_sched_barrier(0);
    float A[N], B[N];
#pragma unroll
    for (int i = 0; i < N; i++) A[i] = 1.0f, B[i] = 0.0f;
    bool restart = false;
    if (on) {
        auto row = [&](int j) {
            float kf[N], rf[N], d[N];
            E::unpack(k[j], kf);
            E::unpack(r[j], rf);
            dy[j].get(d);
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float w = smaller(kf[i]), g = fmaf(d[i], sigmoid(rf[i]), B[i]);
                A[i] = keep(w, A[i]);
                B[i] = keep(w, g);
            }
        };
        if (whole) {
            restart = ends;
            if (ends)
#pragma unroll
                for (int i = 0; i < N; i++) B[i] = stop[i];
#pragma unroll
            for (int j = kBlk - 1; j >= 0; j--) row(j);
        } else {
            Span s = last;
#pragma unroll
            for (int j = kBlk - 1; j >= 0; j--) {
                if (j >= n) continue;
                s.back(j);
                if (!s.live) continue;
                if (j + 1 == s.e) {
                    restart = true;
#pragma unroll
                    for (int i = 0; i < N; i++) B[i] = 0.0f;
                    if (a.dhT) load_f<N>(a.dhT + s.c.cur * a.C + col, B);
                }
                row(j);
            }
        }
#pragma unroll
        for (int i = 0; i < N; i++) A[i] = kept(A[i], restart);
    }
    float p[N], hb[kBlk][N];
    // the last wave's answer counts: does the chunk end with a sequence's last token?
    enter<N, W>(a, link, W - 1 - wave, last.e == kBlk, col, cb * 64 * N, A, B, p, [&] {
        // forward through the rows: the state before each
        if (!on) return;
        Span s = at;
#pragma unroll
        for (int j = 0; j < kBlk; j++) {
            if (!whole && j < n) {
                s.forth(j);
                if (s.live && j == s.b) {
#pragma unroll
                    for (int i = 0; i < N; i++) h[i] = 0.0f;
                    if (a.h0) load_f<N>(a.h0 + s.c.cur * a.C + col, h);
                }
            }
            float kf[N], vf[N];
            E::unpack(k[j], kf);
            E::unpack(v[j], vf);
#pragma unroll
            for (int i = 0; i < N; i++) {
                hb[j][i] = h[i];
                h[i] = step(smaller(kf[i]), h[i], vf[i]);
            }
        }
    });
    if (!on) return;
    auto row = [&](int j) {
        float kf[N], vf[N], rf[N], d[N], dk[N], dv[N], dr[N];
        E::unpack(k[j], kf);
        E::unpack(v[j], vf);
        E::unpack(r[j], rf);
        dy[j].get(d);
#pragma unroll
        for (int i = 0; i < N; i++) {
            float w, share, s, off;
            gates(kf[i], w, share);
            gates(rf[i], s, off);
            const float u = d[i] * s, g = u + p[i], x = vf[i] - hb[j][i];
            dr[i] = u * off * (kf[i] < 0.0f ? fmaf(w, x, hb[j][i]) : fmaf(-share, x, vf[i]));
            dv[i] = g * w;
            dk[i] = dv[i] * x * share;
            p[i] = kf[i] < 0.0f ? fmaf(-w, g, g) : share * g;
        }
        store_row<E>(a.dK, t0 + j, a.ldd, lb, dk);
        store_row<E>(a.dV, t0 + j, a.ldd, lb, dv);
        store_row<E>(a.dR, t0 + j, a.ldd, lb, dr);
    };
    if (whole) {
        if (ends)
#pragma unroll
            for (int i = 0; i < N; i++) p[i] = stop[i];
#pragma unroll
        for (int j = kBlk - 1; j >= 0; j--) row(j);
        if (a.dh0 && begins) store_f<N>(a.dh0 + at.c.cur * a.C + col, p);
    } else {
#pragma unroll
        for (int j = kBlk - 1; j >= 0; j--) {
            if (j >= n) continue;
            last.back(j);
            if (!last.live) continue;
            if (j + 1 == last.e) {
#pragma unroll
                for (int i = 0; i < N; i++) p[i] = 0.0f;
                if (a.dhT) load_f<N>(a.dhT + last.c.cur * a.C + col, p);
            }
            row(j);
            if (a.dh0 && j == last.b) store_f<N>(a.dh0 + last.c.cur * a.C + col, p);
        }
    }
}

template <class E, class D, int W>
__global__ __launch_bounds__(64 * W, 3) void recur_bwd_kernel(RecurArgs a) {
    const int b = blockIdx.x < a.wgs ? blockIdx.x : blockIdx.x - a.wgs, cb = b % a.ncb;
    const int col = (cb * 64 + (int)(threadIdx.x & 63)) * E::N;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (blockIdx.x >= a.wgs) {
        if (wave == 0) copy_empty<E::N>(a, b / a.ncb, col, a.dhT, a.dh0);
        return;
    }
    const int i = take_ticket(a, cb);
    if (i < a.nch) bwd_chunk<E, D, W>(a, cb, col, wave, i);   // the chain runs from the last chunk
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
    const int64_t o = (row * ld + col) * E::ES;
    float k[N], v[N], r[N], h[N], y[N];
    E::unpack(*(const typename E::Raw *)((const char *)K + o), k);
    E::unpack(*(const typename E::Raw *)((const char *)V + o), v);
    E::unpack(*(const typename E::Raw *)((const char *)R + o), r);
    load_f<N>(h_in + row * C + col, h);
#pragma unroll
    for (int j = 0; j < N; j++) {
        h[j] = step(smaller(k[j]), h[j], v[j]);
        y[j] = sigmoid(r[j]) * h[j];
    }
    store_f<N>(h_out + row * C + col, h);
    *(typename E::Raw *)((char *)Y + (row * ldy + col) * E::ES) = E::pack(y);
}

}  // namespace rdev

namespace {

using rdev::RecurArgs;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Waves of a chunk, and a lane's share of a bf16 row.  What decides is how many
// waves the registers leave room for while each holds 16 rows, and how many
// chunks the chain passes through:
//   forward   8 waves, two channels a lane (118 registers, 16 waves a compute
//             unit): 32768 x 4096 305 us;
//   backward  4 waves, one channel a lane (135 registers, 12 waves): 590 us.
// With w as every step's factor these were 289 and 560, and the others: forward with 4
// waves 377, 16 waves 385, one channel 309; backward with 8 waves 686, two channels 714.
// All are of this one size: smaller calls (2048 x 512: 64 workgroups for 256 units) take
// the same shape.
constexpr int kFwdWaves = 8, kBwdWaves = 4;
constexpr int kFwdCols = 128, kBwdCols = 64;   // columns of a workgroup, bf16 (fp32: 64)
struct RecurPlan {
    int64_t ncb, nch;
    size_t prefix, ticket, total;   // workspace: byte offsets
};
RecurPlan plan_recur(int64_t T, int64_t C, int cols, int waves) {
    RecurPlan p{};
    p.ncb = cdiv(C, cols);
    p.nch = cdiv(T, (int64_t)waves * TERN_RECUR_BLOCK);
    if (p.nch <= 1) return p;
    const size_t n = (size_t)p.nch * (size_t)C;
    p.prefix = n * 8;                      // C is a multiple of 8: 16-byte pieces
    p.ticket = n * 12;
    p.total = p.ticket + (size_t)p.ncb * rdev::kTicketStride * 4;
    return p;
}

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

// The chain's words, emptied by a launch of their own (none with one chunk).
void start_chain(RecurArgs &a, const RecurPlan &p, void *workspace, hipStream_t st) {
    if (!p.total) return;
    char *w = (char *)workspace;
    a.agg = (unsigned long long *)w;
    a.prefix = (uint32_t *)(w + p.prefix);
    a.ticket = (uint32_t *)(w + p.ticket);
    const int64_t n16 = (int64_t)(p.ticket / 16), n = n16 > p.ncb ? n16 : p.ncb;
    hipLaunchKernelGGL(rdev::recur_init_kernel, grid_of(cdiv(n, 256)), dim3(256), 0, st, (uint4 *)w, n16, a.ticket,
                       (int)p.ncb);
}
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
    size_t most = 0;
    for (int waves : {kFwdWaves, kBwdWaves}) most = std::max(most, plan_recur(T, C, 64, waves).total);
    return (most + 255) & ~size_t(255);
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
    const RecurPlan p = plan_recur(T, C, act_dtype == TERN_BF16 ? kFwdCols : 64, kFwdWaves);
    const size_t wsb = p.total;
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
    if (!grid_fits(p.ncb * (p.nch + empties), 64 * kFwdWaves)) return TERN_ERR_SHAPE;
    RecurArgs a{};
    a.K = K; a.V = V; a.R = R; a.ld = ld; a.h0 = h0; a.off = offsets; a.S = n_seq; a.T = T;
    a.C = (int)C; a.ncb = (int)p.ncb; a.nch = (int)p.nch;
    a.Y = Y; a.ldy = ldy; a.hT = hT; a.states = states;
    hipStream_t st = (hipStream_t)stream;
    start_chain(a, p, workspace, st);
    a.wgs = (unsigned)(p.ncb * p.nch);
    const dim3 g = grid_of(a.wgs + p.ncb * empties), b(64 * kFwdWaves);
    if (act_dtype == TERN_BF16) hipLaunchKernelGGL((rdev::recur_fwd_kernel<rdev::Bf, kFwdWaves>), g, b, 0, st, a);
    else hipLaunchKernelGGL((rdev::recur_fwd_kernel<rdev::Fp, kFwdWaves>), g, b, 0, st, a);
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
    const RecurPlan p = plan_recur(T, C, act_dtype == TERN_BF16 ? kBwdCols : 64, kBwdWaves);
    const size_t wsb = p.total;
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
    if (!grid_fits(p.ncb * (p.nch + empties), 64 * kBwdWaves)) return TERN_ERR_SHAPE;
    RecurArgs a{};
    a.K = K; a.V = V; a.R = R; a.ld = ld; a.h0 = h0; a.off = offsets; a.S = n_seq; a.T = T;
    a.C = (int)C; a.ncb = (int)p.ncb; a.nch = (int)p.nch;
    a.states = const_cast<float *>(states);
    a.dY = dY; a.lddy = lddy; a.dhT = dhT; a.dK = dK; a.dV = dV; a.dR = dR; a.ldd = ldd; a.dh0 = dh0;
    hipStream_t st = (hipStream_t)stream;
    start_chain(a, p, workspace, st);
    a.wgs = (unsigned)(p.ncb * p.nch);
    const dim3 g = grid_of(a.wgs + p.ncb * empties), b(64 * kBwdWaves);
    if (act_dtype == TERN_F32)
        hipLaunchKernelGGL((rdev::recur_bwd_kernel<rdev::Fp, rdev::Fp, kBwdWaves>), g, b, 0, st, a);
    else if (dy_dtype == TERN_F32)
        hipLaunchKernelGGL((rdev::recur_bwd_kernel<rdev::Bh, rdev::Fp, kBwdWaves>), g, b, 0, st, a);
    else
        hipLaunchKernelGGL((rdev::recur_bwd_kernel<rdev::Bh, rdev::Bh, kBwdWaves>), g, b, 0, st, a);
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
