// tern_logprob.hip -- log probabilities of given tokens, entropy and top
// alternatives of rows of logits (C ABI and formulas in include/tern.h).
//
// With m the row's largest logit and d = (Z - m) scale <= 0,
//   s = sum e^d,  u = sum e^d d:  logp = d[token] - log s,  entropy = log s - u / s.
// The exponentials are powers of two (d is carried in units of log 2).
//
// The k largest: 256 groups of elements (64, a lane's each, where one wave has the row
// and few are asked for) know their own largest element.  The k-th largest of those is a bound that at least k
// elements reach, and hardly more do; a bisection over its bits by one wave finds
// it.  The eights that hold an element which reaches it go to a list in shared
// memory, their elements that do to another, and each one's place is the
// number of greater keys there.  One alternative is the first element that equals the
// row's largest, without lists.  Where a list would overflow (ties, rows in which
// fewer than k tokens are allowed) the k-th largest value is found itself, by the same
// bisection over all elements unless the bound is it, and then the elements above it
// and the first of those equal to it, by their index.
//
// A row longer than a workgroup's registers is taken in segments, one after the
// other (the sums rescaled, the alternatives so far a bound for the next); where
// the rows are few, by workgroups that a second launch joins.
//
// 4096 rows of 131072 bf16 logits: 196 us without alternatives (5.5 TB/s: HBM bounds
// it), 221 with 20, 244 with 64 (the search among the lanes' largest, and one
// more look at the registers, about as long as a third of the sums).  (Every alternative
// by a maximum over the row: 43 ms.)  13 rows of 50021 in fp32, 20 alternatives: 12.5 us in
// two launches; 2048 rows of 256, the largest alone, 4.0.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tern_softmax.h"

namespace tern {
namespace hdev {

using namespace rows;

struct LogprobArgs {
    const void *Z;
    int64_t ld, T;
    int V, k, S;
    int part, seg;             // elements of a workgroup's part of a row, of a segment of it
    float scale, c;            // c = scale log2 e
    const int64_t *tokens;
    float *logp, *entropy, *lse;
    int64_t *top_ids;
    float *top_logp;
    float4 *sums;              // [T][S]: largest logit, s, u of a part
    uint64_t *keys;            // [T][S][k]: its alternatives, 0 behind the last
};

// (Rows of one stride and wave have 64 eights, all of which their list holds.)
template <int DT, int W, int NV>
struct Pick {
    static constexpr int kKeys = W >= 4 ? 1024 : 256;
    static constexpr int kEights = W >= 4 ? 512 : NV > 1 ? 128 : 64, kMasks = NV * W;
    uint64_t top[TERN_TOP_MAX];    // the largest so far, falling
    uint64_t key[kKeys];
    Raw8<DT> eight[kEights];
    int from[kEights];             // index of an eight's first element in its segment
    uint64_t mask[kMasks];         // lanes with an element equal to the k-th largest, stride by stride and wave by wave
    int before[kMasks];            // how many such lanes stand before a mask's
    uint32_t group[W >= 4 ? W * 64 : 1];
    float sum[2][W];
    uint32_t bound;
    int keys, eights;
};

struct MaxU {
    __device__ static uint32_t of(uint32_t a, uint32_t b) { return a > b ? a : b; }
};
struct MinU {
    __device__ static uint32_t of(uint32_t a, uint32_t b) { return a < b ? a : b; }
};
template <class Op>
__device__ inline uint32_t wave_all_u(uint32_t x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x = Op::of(x, (uint32_t)__shfl_xor((int)x, d));
    return x;
}
// A bound that at least k of the groups' largest reach, by one wave, of whose lanes
// each knows G of them (k <= 64 G).
template <int G>
__device__ inline uint32_t bound_of(const uint32_t (&g)[G], int k) {
    uint32_t most = g[0], least = g[0];
#pragma unroll
    for (int i = 1; i < G; i++) most = max(most, g[i]), least = min(least, g[i]);
    most = wave_all_u<MaxU>(most);
    auto reach = [&](uint32_t t) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < G; i++) c += __builtin_popcountll(__ballot(g[i] >= t));
        return c;
    };
    if (reach(most) >= k) return most;
    // at least k reach lo, fewer than k reach hi; a few more than k will do
    uint32_t lo = wave_all_u<MinU>(least), hi = most;
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int c = reach(mid);
        if (c >= k) {
            lo = mid;
            if (c <= k + k / 4 + 2) break;
        } else {
            hi = mid;
        }
    }
    return lo;
}

// The elements that the listed eights hold, as keys: those that `take` says.
template <int DT, int W, int NV, class F>
__device__ inline void keys_of_eights(Pick<DT, W, NV> &p, int eights, int n, uint32_t first, int tid, F take) {
    for (int q = tid; q < eights * 8; q += W * 64) {
        const int v = p.from[q >> 3] + (q & 7);
        const float f = at<DT>((const char *)&p.eight[q >> 3], q & 7);
        if (v < n && take(f)) {
            const int at = atomicAdd(&p.keys, 1);
            if (at < Pick<DT, W, NV>::kKeys) p.key[at] = key_of(f, first + v);
        }
    }
}

// The `want` largest of a segment as keys behind the `had` in p.key, whatever it holds
// (of NaNs, as of infinities, any).  `bound` is reached by that many at least.
template <int DT, int W, int NV>
__device__ inline void exact_keys(const Raw8<DT> (&x)[NV], int n, uint32_t first, int want, int had, uint32_t bound,
                                  Pick<DT, W, NV> &p, int tid) {
    constexpr int ST = W * 512, M = Pick<DT, W, NV>::kMasks;
    tid = fresh(tid);
    const int lane = tid & 63, wave = tid >> 6;
    auto number = [](float f) { return f != f ? kInf : f; };
    int turn = 0;
    auto above = [&](uint32_t t) {
        const float v = from_ordered(t);
        float c = 0.0f;
        each8<DT, W, NV>(x, n, [&](int i, const float *f) {
#pragma unroll
            for (int j = 0; j < 8; j++) c += number(f[j]) > v && i * ST + tid * 8 + j < n ? 1.0f : 0.0f;
        });
        turn ^= 1;
        return (int)row_all<Add, W>(c, p.sum[turn], tid);
    };
    const uint32_t least = ordered(-kInf), most = ordered(kInf);
    uint32_t value = min(max(bound, least), most);
    int more = above(value);
    if (more >= want) {   // fewer than want are above hi, more are above lo
        uint32_t lo = value, hi = most;
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (above(mid) < want) hi = mid;
            else lo = mid;
        }
        value = hi;
        more = above(value);
    }
    const float v = from_ordered(value);
    meet<W>();
    if (tid == 0) p.keys = had, p.eights = 0;
    if (tid < M) p.mask[tid] = 0;
    meet<W>();
    each8<DT, W, NV>(x, n, [&](int i, const float *f) {
        bool over = false, equal = false;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const bool in = i * ST + tid * 8 + j < n;
            over = over || (in && number(f[j]) > v);
            equal = equal || (in && number(f[j]) == v);
        }
        const uint64_t m = __ballot(equal);
        if (lane == 0) p.mask[i * W + wave] = m;
        if (over) {
            const int at = atomicAdd(&p.eights, 1);   // fewer than want
            p.eight[at] = x[i], p.from[at] = i * ST + tid * 8;
        }
    });
    meet<W>();
    keys_of_eights<DT, W, NV>(p, p.eights, n, first, tid, [&](float f) { return number(f) > v; });
    if (tid < 64) {
        const int mine = lane < M ? __builtin_popcountll(p.mask[lane]) : 0;
        int sum = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        if (lane < M) p.before[lane] = sum - mine;
    }
    meet<W>();
    const int ties = want - more;
    each8<DT, W, NV>(x, n, [&](int i, const float *f) {
        const uint64_t m = p.mask[i * W + wave];
        const int rank = p.before[i * W + wave] + __builtin_popcountll(m & ((1ull << lane) - 1));
        if ((m >> lane & 1) && rank < ties)   // the list's other eights have been taken
            p.eight[rank] = x[i], p.from[rank] = i * ST + tid * 8;
    });
    meet<W>();
    if (tid < 64) {   // the listed eights in order, 64 elements at a time
        const int eights = min(ties, p.before[M - 1] + __builtin_popcountll(p.mask[M - 1]));
        int taken = 0;
        for (int q = tid; q < (eights * 8 + 63) / 64 * 64; q += 64) {
            const int at8 = min(q >> 3, eights - 1), i = p.from[at8] + (q & 7);
            const float f = at<DT>((const char *)&p.eight[at8], q & 7);
            const bool tie = q < eights * 8 && i < n && number(f) == v;
            const uint64_t m = __ballot(tie);
            const int rank = taken + __builtin_popcountll(m & ((1ull << lane) - 1));
            if (tie && rank < ties) p.key[atomicAdd(&p.keys, 1)] = key_of(f, first + i);
            taken += __builtin_popcountll(m);
        }
    }
    meet<W>();
}

// The largest alone: the first of a segment's elements that equal its largest, m, and the
// one that p.top holds where one is had.  (A row of nothing but NaN: its first.)
template <int DT, int W, int NV>
__device__ inline int first_of_segment(const Raw8<DT> (&x)[NV], int n, uint32_t first, int had, float mine, float m,
                                       Pick<DT, W, NV> &p, int tid) {
    tid = fresh(tid);
    if (tid == 0) p.bound = 0xFFFFFFFFu;
    meet<W>();
    if (__ballot(mine == m)) {
        uint32_t at = 0xFFFFFFFFu;
        each8<DT, W, NV>(x, n, [&](int i, const float *f) {
            if (max8(f) < m) return;
#pragma unroll
            for (int j = 7; j >= 0; j--) {
                const uint32_t v = i * W * 512 + tid * 8 + j;
                if (f[j] == m && v < (uint32_t)n) at = min(at, v);
            }
        });
        if (at != 0xFFFFFFFFu) atomicMin(&p.bound, at);
    }
    meet<W>();
    if (tid == 0) {
        const uint64_t key = key_of(m, first + (p.bound == 0xFFFFFFFFu ? 0 : p.bound));
        p.top[0] = had ? max(p.top[0], key) : key;
    }
    meet<W>();
    return 1;
}

// The k largest (fewer where there are not so many) of the segment in x, n elements
// of which `first` is the first's index, and of the `had` that p.top holds already:
// to p.top.  Returns how many there are.
template <int DT, int W, int NV>
__device__ inline int top_of_segment(const Raw8<DT> (&x)[NV], int n, uint32_t first, int k, int had, float mine,
                                     Pick<DT, W, NV> &p, int tid) {
    using P = Pick<DT, W, NV>;
    constexpr int ST = W * 512;
    tid = fresh(tid);
    if (tid == 0) p.keys = had, p.eights = 0;
    for (int i = tid; i < had; i += W * 64) p.key[i] = p.top[i];
    uint32_t reached;
    if constexpr (W == 1) {
        // Groups of two where 64 would not do.  16384 rows of bf16, 64 groups and 256: of 512, 28
        // alternatives 22.9 us and 24.5, 32: 26.3 and 25.1; of 256, 16: 21.0 and 22.8, 24: 47 and 24;
        // of 4000, 64: 547 (the lists overflow) and 73.
        if (n < 2 * k) {   // most are asked for, and all are compared: of 64, 64: 40 us with a search, 24 without
            reached = ordered(-kInf);
        } else if (2 * k < min(64, (n + 7) / 8)) {
            const uint32_t g[1] = {ordered(mine)};
            reached = bound_of(g, k);
        } else {
            float m[4] = {-kInf, -kInf, -kInf, -kInf};
            each8<DT, W, NV>(x, n, [&](int, const float *f) {
#pragma unroll
                for (int j = 0; j < 4; j++) m[j] = max3(m[j], f[2 * j], f[2 * j + 1]);
            });
            const uint32_t g[4] = {ordered(m[0]), ordered(m[1]), ordered(m[2]), ordered(m[3])};
            reached = bound_of(g, k);
        }
        meet<W>();
    } else {
        static_assert(W == 4, "a group for each lane");
        p.group[tid] = ordered(mine);
        meet<W>();
        if (tid < 64) {
            const uint32_t g[4] = {p.group[tid], p.group[tid + 64], p.group[tid + 128], p.group[tid + 192]};
            const uint32_t b = bound_of(g, k);
            if (tid == 0) p.bound = b;
        }
        meet<W>();
        reached = p.bound;
    }
    // the last of the k so far is a bound as well
    const float bound = from_ordered(had == k ? max(reached, (uint32_t)(p.top[k - 1] >> 32)) : reached);
    if (__ballot(!(mine < bound)))
        each8<DT, W, NV>(x, n, [&](int i, const float *f) {
            if (max8(f) < bound) return;
            const int at = atomicAdd(&p.eights, 1);
            if (at < P::kEights) p.eight[at] = x[i], p.from[at] = i * ST + tid * 8;
        });
    meet<W>();
    const int eights = p.eights;
    if (eights <= P::kEights)
        keys_of_eights<DT, W, NV>(p, eights, n, first, tid, [&](float f) { return !(f < bound); });
    meet<W>();
    const int want = min(k, had + n);
    int keys = p.keys;
    if (eights > P::kEights || keys > P::kKeys || keys < want) {
        meet<W>();
        exact_keys<DT, W, NV>(x, n, first, min(k, n), had, reached, p, tid);
        keys = p.keys;
    }
    for (int q = tid; q < keys; q += W * 64) {
        const uint64_t key = p.key[q];
        int place = 0;
#pragma unroll 8
        for (int i = 0; i < keys; i++) place += p.key[i] > key;
        if (place < k) p.top[place] = key;
    }
    meet<W>();
    return want;
}

// what a row's sums say
struct RowEnd {
    float m0, s, logs, scale;
    __device__ float log_p(float z) const { return s == 0.0f ? -kInf : 2.0f * fmaf(half_apart(z, m0), scale, -0.5f * logs); }
};
__device__ inline RowEnd finish_row(const LogprobArgs &a, int64_t t, float m0, float s, float u, int tid) {
    s = at_least_one(s);
    RowEnd r{m0, s, logf(s), a.scale};
    if (tid == 0) {
        if (a.lse) a.lse[t] = fmaf(m0, a.scale, r.logs);
        if (a.entropy) {
            const float h = r.logs - u / s * kLn2;
            a.entropy[t] = s == 0.0f || h < 0.0f ? 0.0f : h;
        }
    }
    return r;
}

// The row's token (-1: none to tell of) and its logit.  (Fetched ahead of a whole row it
// costs registers and 1 to 8 per cent; where parts are joined it comes first.)
struct Token {
    int64_t id;
    float z;
};
template <int DT>
__device__ inline Token token_of(const LogprobArgs &a, int64_t t, int tid) {
    Token y{-1, 0.0f};
    if (a.tokens && tid == 0) y.id = a.tokens[t];
    if (y.id >= a.V) y.id = -1;
    if (y.id >= 0) y.z = at<DT>((const char *)a.Z + t * a.ld * esize<DT>(), y.id);
    return y;
}
__device__ inline void tell_token(const LogprobArgs &a, int64_t t, const RowEnd &r, const Token &y, int tid) {
    if (a.tokens && tid == 0) a.logp[t] = y.id >= 0 ? r.log_p(y.z) : 0.0f;
}

// s = sum e, u = sum e d over a lane's elements, m0 the segment's largest
template <int DT, int W, int NV>
__device__ inline void lane_sums(const char *z, const Raw8<DT> (&x)[NV], int n, float m0, const Exponent &e, int tid, float &s,
                                 float &u) {
    s = u = 0.0f;
    auto add = [&](float d) {
        const float p = exp2_(d);
        s += p;
        u = fmaf(p, fmaxf(d, -200.0f), u);   // (-inf: p is 0)
    };
    if (!e.far) {
        each8<DT, W, NV>(x, n, [&](int, const float *f) {
#pragma unroll
            for (int j = 0; j < 8; j++) add(e.of(f[j]));
        });
    } else {
        for (int v = fresh(tid); v < n; v += W * 64) add(apart(at<DT>(z, v), m0, e.c));
    }
}

template <int DT, int W, int NV>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W, 4) void logprob_kernel(LogprobArgs a) {
    constexpr int R = W == 1 ? 4 : 1;   // rows of a workgroup
    __shared__ Pick<DT, W, NV> picks[R];
    __shared__ float sh[3][W];
    const int slot = R > 1 ? threadIdx.x >> 6 : 0, tid = R > 1 ? threadIdx.x & 63 : threadIdx.x;
    Pick<DT, W, NV> &pick = picks[slot];
    const int64_t items = a.T * a.S;
    for (int64_t item = (int64_t)blockIdx.x * R + slot; item < items; item += (int64_t)gridDim.x * R) {
        const int64_t t = a.S == 1 ? item : item / a.S;
        const int begin = (int)(item - t * a.S) * a.part, end = min(begin + a.part, a.V);
        const char *row = (const char *)a.Z + t * a.ld * esize<DT>();
        float M = -kInf, s = 0.0f, u = 0.0f;   // of the segments so far
        int had = 0;
        for (int first = begin; first < end; first += a.seg) {
            const int n = min(a.seg, end - first);
            const char *z = row + (int64_t)first * esize<DT>();
            Raw8<DT> x[NV];
            load_row<DT, W, NV>(z, n, tid, x);
            const float mine = lane_max<DT, W, NV>(x, n);
            const float m = row_all<Max, W>(mine, sh[0], tid), m0 = m == -kInf ? 0.0f : m;
            const Exponent e(m0, a.c);
            float s1, u1;
            lane_sums<DT, W, NV>(z, x, n, m0, e, tid, s1, u1);
            row_sums<W>(s1, u1, &sh[1], tid);
            if (!e.far) {   // the exponents were e.off too large
                const float f = exp2_(-e.off);
                u1 = fmaf(-e.off, s1, u1) * f;
                s1 *= f;
            }
            const float both = fmaxf(M, m);
            if (first == begin) {
                s = s1, u = u1;
            } else {   // to the larger of the two largest
                const float b0 = both == -kInf ? 0.0f : both;
                const float d0 = apart(M, b0, a.c), d1 = apart(m, b0, a.c), f0 = exp2_(d0), f1 = exp2_(d1);
                u = f0 * fmaf(s, fmaxf(d0, -200.0f), u) + f1 * fmaf(s1, fmaxf(d1, -200.0f), u1);
                s = f0 * s + f1 * s1;
            }
            M = both;
            if (a.k == 1) had = first_of_segment<DT, W, NV>(x, n, first, had, mine, m, pick, tid);
            else if (a.k) had = top_of_segment<DT, W, NV>(x, n, first, a.k, had, mine, pick, tid);
            meet<W>();
        }
        const int l = fresh(tid);
        if (a.S == 1) {
            const RowEnd r = finish_row(a, t, M == -kInf ? 0.0f : M, s, u, l);
            tell_token(a, t, r, token_of<DT>(a, t, l), l);
            if (l < a.k) {
                a.top_ids[t * a.k + l] = index_of(pick.top[l]);
                a.top_logp[t * a.k + l] = r.log_p(value_of(pick.top[l]));
            }
        } else {
            if (l == 0) a.sums[item] = float4{M, s, u, 0.0f};
            if (l < a.k) a.keys[item * a.k + l] = l < had ? pick.top[l] : 0;
        }
        meet<W>();
    }
}

// Rows that were cut: the parts' sums meet, and their alternatives.  Each part's keys
// fall, so that k at least reach the k-th of any part, and, with r = ceil(k / S), the
// smallest of the parts' r-th: the larger of the two bounds leaves few to compare.
template <int DT>
__global__ __launch_bounds__(256) void logprob_join_kernel(LogprobArgs a) {
    __shared__ uint64_t list[kMaxSegments * TERN_TOP_MAX];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const Token y = token_of<DT>(a, t, tid);
        float4 q = lane < a.S ? a.sums[t * a.S + lane] : float4{-kInf, 0.0f, 0.0f, 0.0f};
        const float m = wave_all<Max>(q.x), m0 = m == -kInf ? 0.0f : m;
        const float d = apart(q.x, m0, a.c), f = exp2_(d);
        const float s = wave_all<Add>(f * q.y), u = wave_all<Add>(f * fmaf(q.y, fmaxf(d, -200.0f), q.z));
        const RowEnd r = finish_row(a, t, m0, s, u, tid);
        tell_token(a, t, r, y, tid);
        if (!a.k) continue;
        const uint64_t *keys = a.keys + t * a.S * a.k;
        const int rank = (a.k + a.S - 1) / a.S - 1;
        uint64_t low = lane < a.S ? keys[lane * a.k + rank] : ~(uint64_t)0;
        uint64_t high = lane < a.S ? keys[lane * a.k + a.k - 1] : 0;
#pragma unroll
        for (int i = 1; i < 64; i *= 2) {
            low = min(low, (uint64_t)__shfl_xor((unsigned long long)low, i));
            high = max(high, (uint64_t)__shfl_xor((unsigned long long)high, i));
        }
        const uint64_t bound = max(low, high);
        if (tid == 0) count = 0;
        __syncthreads();
        for (int i = tid; i < a.S * a.k; i += 256) {
            const uint64_t key = keys[i];
            if (key >= bound && key) list[atomicAdd(&count, 1)] = key;
        }
        __syncthreads();
        const int n = count;
        for (int i = tid; i < n; i += 256) {
            const uint64_t key = list[i];
            int place = 0;
#pragma unroll 8
            for (int j = 0; j < n; j++) place += list[j] > key;
            if (place < a.k) {
                a.top_ids[t * a.k + place] = index_of(key);
                a.top_logp[t * a.k + place] = r.log_p(value_of(key));
            }
        }
        __syncthreads();
    }
}

}  // namespace hdev

namespace {

using hdev::LogprobArgs;

int launched() { return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

// Segments of four waves, so that four workgroups share a compute unit and one loads
// while others compute.  (4096 rows of 131072 bf16, 64 alternatives: 252 us with 4
// waves, 287 with 8, 361 with 16.)
RowPlan plan_parts(int32_t dt, int64_t T, int64_t V) { return plan_rows(dt, T, V, 4, true); }

size_t workspace_of(const RowPlan &p, int64_t T, int32_t k) {
    return p.S == 1 ? 0 : (size_t)T * (size_t)p.S * (16 + 8 * (size_t)k);
}

template <int32_t DT>
struct Launch {
    LogprobArgs a;
    hipStream_t st;
    template <int W, int NV>
    void operator()() const {
        constexpr int R = W == 1 ? 4 : 1;
        const dim3 g((unsigned)std::min<int64_t>(cdiv_(a.T * a.S, R), kMaxGroups)), b(W == 1 ? 256 : 64 * W);
        hipLaunchKernelGGL((hdev::logprob_kernel<DT, W, NV>), g, b, 0, st, a);
    }
};

template <int32_t DT>
void run(const LogprobArgs &a, const RowPlan &p, hipStream_t st) {
    with_plan<DT, 1, 4>(p, Launch<DT>{a, st});
    if (a.S > 1)
        hipLaunchKernelGGL(hdev::logprob_join_kernel<DT>, dim3((unsigned)std::min<int64_t>(a.T, kMaxGroups)), dim3(256), 0,
                           st, a);
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

size_t tern_logprob_workspace_bytes(int64_t T, int64_t V, int32_t k) {
    if (!row_sizes_ok(T, V) || k < 0 || k > TERN_TOP_MAX) return 0;
    return std::max(workspace_of(plan_parts(TERN_F32, T, V), T, k), workspace_of(plan_parts(TERN_BF16, T, V), T, k));
}

int tern_logprob(const void *Z, int64_t ld, int32_t z_dtype, float scale, int64_t T, int64_t V, const int64_t *tokens,
                 float *logp, float *entropy, float *lse, int32_t k, int64_t *top_ids, float *top_logp,
                 void *workspace, size_t workspace_bytes, void *stream) {
    if (!row_sizes_ok(T, V) || !row_stride_ok(ld, V)) return TERN_ERR_SHAPE;
    if (z_dtype != TERN_F32 && z_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (!factor_ok(scale) || k < 0 || k > TERN_TOP_MAX || k > V) return TERN_ERR_VALUE;
    if (T == 0) return TERN_OK;
    if (!Z || !tokens != !logp || (k > 0 && (!top_ids || !top_logp))) return TERN_ERR_NULL;
    const RowPlan p = plan_parts(z_dtype, T, V);
    const size_t wsb = workspace_of(p, T, k);
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (off_by(Z, 16) || off_by(tokens, 8) || off_by(top_ids, 8) || off_by(logp, 4) || off_by(entropy, 4) ||
        off_by(lse, 4) || off_by(top_logp, 4) || off_by(workspace, 16))
        return TERN_ERR_ALIGN;
    const Mat outs[] = {vec(logp, T, 4), vec(entropy, T, 4), vec(lse, T, 4), vec(top_ids, T * k, 8),
                        vec(top_logp, T * k, 4), vec(workspace, (int64_t)wsb, 1)};
    const Mat ins[] = {{Z, T, V, ld, (size_t)(z_dtype == TERN_BF16 ? 2 : 4)}, vec(tokens, T, 8)};
    if (any_overlap(outs, 6, ins, 2)) return TERN_ERR_ALIAS;
    LogprobArgs a{Z, ld, T, (int)V, k, p.S, (int)p.part, (int)p.seg, scale, (float)(scale * rows::kLog2e), tokens, logp, entropy, lse,
                  top_ids, top_logp, (float4 *)workspace, nullptr};
    if (p.S > 1) a.keys = (uint64_t *)(a.sums + T * p.S);
    hipStream_t st = (hipStream_t)stream;
    if (z_dtype == TERN_BF16) run<TERN_BF16>(a, p, st);
    else run<TERN_F32>(a, p, st);
    return launched();
}

}  // extern "C"
