// tern_distill.hip -- the distillation loss of rows of logits against a
// teacher's top alternatives, mixed with the cross entropy of given targets, and
// its gradient (C ABI and formulas in include/tern.h).
//
// A row of logits is held in registers (tern_softmax.h): its largest element,
// then s1 = sum exp(Z - m) and st = sum exp((Z - m) / tau), then the gradient
//   dloss (alpha exp(Z - m) / s1 + (1 - alpha) tau exp((Z - m) / tau) / st)
// from the same registers, so that Z is read once and dZ written once.  The few
// elements that have a target or a teacher's probability to lose are written again,
// whole, by the wave that wrote them before.  Where one softmax serves both parts
// (tau = 1, or only one part) each element takes one exponential a pass; where tau is
// 2, exp(Z - m) is the square of the other; else two.
//
// Without dZ a row is taken in segments, one after the other, as tern_logprob takes
// it.  Rows that are cut (few rows, or with dZ longer than a workgroup's registers)
// take two launches: the parts' sums, and the logits of the named tokens, which dZ
// may overwrite; then the loss and the gradient, which reads the parts again.
//
// 8192 rows of 65536 bf16 logits, tau 2, loss and gradient: 413 to 440 us by the card, 4.9 to
// 5.2 TB/s; at tau 1.5, with two exponentials, 445 to 488.  Two workgroups of eight waves share a
// compute unit and load and compute in turn; rows of 131072 fill it alone and are not
// hidden (4096 of them 505 us, 4.3 TB/s).  fp32 rows of more than 65536 are read twice (2048
// of 131072: 590 to 646 us where one pass would take 440).  The loss alone: 1021 rows of 50021 23 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "tern_softmax.h"

namespace tern {
namespace kdev {

using namespace rows;

constexpr int kEntries = TERN_TOP_MAX + 1;   // the teacher's, and the target

struct DistillArgs {
    const void *Z;
    int64_t ld, lddz, T;
    int V, K, S;
    int part, seg;            // elements of a workgroup's part of a row, of a segment of it
    const int64_t *targets, *ids;
    const float *lp, *dloss;
    float alpha, tau;
    float c1, ct;             // log2 e, log2 e / tau
    float unit, rest;         // tau = 2 unit rest: unit a power of two, rest from 1 to 2
    bool ce, kl;              // which parts the call has
    float *loss;
    void *dZ;
    float4 *sums;             // [T][S]: largest logit, s1, st of a part
    float *named;             // [T][65]: logits of the teacher's tokens and of the target
};

// The tokens a row names.
struct Names {
    int id[kEntries];         // -1: none; the last is the target
    float z[kEntries];        // their logits
    float less[kEntries];     // what the gradient loses there, before dloss
    float p[kEntries], logp[kEntries];   // the teacher's
    uint8_t place[1024];      // which entry wrote here last, by its token's last ten bits
    bool kl, ce;
};

// An entry of a row as the caller gives it (-1 and -inf: none), and the row's target.
struct Given {
    int id, target;
    float lp;
};
__device__ inline Given given(const DistillArgs &a, int64_t t, int lane) {
    int64_t id = -1, y = a.ce ? a.targets[t] : -1;
    float lp = -kInf;
    if (a.kl && lane < a.K) {
        id = a.ids[t * a.K + lane];
        lp = a.lp[t * a.K + lane];
    }
    if (id < 0 || id >= a.V || lp == -kInf) id = -1, lp = -kInf;
    return Given{(int)id, y >= 0 && y < a.V ? (int)y : -1, lp};
}

// By the first wave of a row.  `z` is the row (its logits are read where `cut` is not
// set: in a row that is cut they come from the workspace).
template <int DT>
__device__ inline void read_names(const DistillArgs &a, int64_t t, const char *z, const Given &in, Names &e, int lane,
                                  bool cut) {
    const int me = in.id, target = in.target;
    const float lp = in.lp;
    float zid = 0.0f, zy = 0.0f;
    if (cut) {
        if (me >= 0) zid = a.named[t * kEntries + lane];
        if (target >= 0) zy = a.named[t * kEntries + kEntries - 1];
    } else {
        if (me >= 0) zid = at<DT>(z, me);
        if (target >= 0) zy = at<DT>(z, target);
    }
    const bool kl = __ballot(me >= 0) != 0;
    const float lm = wave_all<Max>(lp);
    float p = me < 0 ? 0.0f : exp2_((lp - lm) * a.c1);
    const float ps = wave_all<Add>(p);
    p = me < 0 ? 0.0f : p / ps;
    if (me >= 0) e.place[me & 1023] = (uint8_t)lane;
    meet<1>();
    float mine = p, its = 0.0f;
    if (__ballot(me >= 0 && e.place[me & 1023] != lane)) {
        // a token that is named twice (or two that share a place) loses the sum, in the order of the entries
        mine = 0.0f;
        for (int j = 0; j < a.K; j++) {
            const int o = __builtin_amdgcn_readlane(me, j);
            const float q = as_f(__builtin_amdgcn_readlane(as_u(p), j));
            mine += o == me ? q : 0.0f;
            its += o == target ? q : 0.0f;
        }
    } else {
        its = wave_all<Add>(me == target ? p : 0.0f);   // one entry at most
    }
    const float f = (1.0f - a.alpha) * a.tau;
    e.id[lane] = me;
    e.z[lane] = zid;
    e.p[lane] = p;
    e.logp[lane] = me < 0 ? 0.0f : lp - lm - logf(ps);
    e.less[lane] = kl ? fmaf(f, mine, me == target ? a.alpha : 0.0f) : 0.0f;
    if (lane == 0) {
        e.id[kEntries - 1] = target;
        e.z[kEntries - 1] = zy;
        e.less[kEntries - 1] = fmaf(kl ? f : 0.0f, its, a.alpha);
        e.kl = kl;
        e.ce = target >= 0;
    }
}

// How many exponentials an element takes: one softmax, two of which one is the square
// of the other, or two.
enum Kind { kOne, kSquare, kTwo };

// A row's exponents: of (Z - m) / tau, or of the one softmax there is, and of Z - m.
struct Exponents {
    Exponent t, one;
    float m0;
    bool far;
    __device__ Exponents(float m, float ct, float c1, Kind kind) : t(m, ct), one(m, c1), m0(m) {
        far = t.far || (kind == kTwo && one.far);
    }
};

// A lane's sums of exponentials: of Z - m (s1) and of (Z - m) / tau (st); where there is
// one softmax, st is its.
template <int DT, int W, int NV>
__device__ inline void sums_of(const char *z, const Raw8<DT> (&x)[NV], int n, const Exponents &e, Kind kind, int tid,
                               float &s1, float &st) {
    s1 = 0.0f, st = 0.0f;
    if (!e.far) {
        each8<DT, W, NV>(x, n, [&](int, const float *f) {
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; j++) st += p[j] = exp2_(e.t.of(f[j]));
            if (kind == kSquare)
#pragma unroll
                for (int j = 0; j < 8; j++) s1 = fmaf(p[j], p[j], s1);
            if (kind == kTwo)
#pragma unroll
                for (int j = 0; j < 8; j++) s1 += exp2_(e.one.of(f[j]));
        });
        // the exponents were `off` too large
        s1 *= exp2_(kind == kSquare ? -2.0f * e.t.off : -e.one.off);
        st *= exp2_(-e.t.off);
    } else {
        for (int v = fresh(tid); v < n; v += W * 64) {
            const float f = at<DT>(z, v);
            st += exp2_(apart(f, e.m0, e.t.c));
            s1 += exp2_(apart(f, e.m0, e.one.c));
        }
    }
}

struct Sums {
    float m0, s1, st;
};

// The loss of a row, by its first wave.  The KL is summed in units of 1 / unit, about tau / 2: neither it nor
// tau^2 alone has to fit fp32, but tau times a difference of logits.
__device__ inline void write_loss(const DistillArgs &a, int64_t t, const Names &e, const Sums &s, int lane) {
    float k = 0.0f;
    const float p = e.p[lane];
    if (e.id[lane] >= 0 && p != 0.0f)
        k = s.st == 0.0f ? kInf : p * fmaf(logf(s.st), a.unit, fmaf(e.logp[lane], a.unit, -half_apart(e.z[lane], s.m0) / a.rest));
    k = wave_all<Add>(k);
    if (lane != 0) return;
    float loss = 0.0f;
    if (e.ce)
        loss = s.s1 == 0.0f ? kInf : 2.0f * (a.alpha * fmaf(logf(s.s1), 0.5f, -half_apart(e.z[kEntries - 1], s.m0)));
    if (e.kl) loss = fmaf((1.0f - a.alpha) * a.tau * (2.0f * a.rest), k, loss);
    a.loss[t] = loss;
}

// the gradient of a segment's n elements, of which `first` is the row's index of the first
template <int DT, int W, int NV>
__device__ inline void write_grad(const DistillArgs &a, int64_t t, const char *z, const Raw8<DT> (&x)[NV], int first,
                                  int n, const Names &e, const Sums &s, float c, Kind kind, int tid) {
    constexpr int ST = W * 512, ES = esize<DT>();
    const float w = a.dloss ? a.dloss[t] : 1.0f;
    char *dz = (char *)a.dZ + (t * a.lddz + first) * ES;
    const bool zero = w == 0.0f || !(e.kl || e.ce);
    float f1 = e.ce && s.s1 != 0.0f ? w * a.alpha / s.s1 : 0.0f;
    float ft = e.kl && s.st != 0.0f ? w * (1.0f - a.alpha) * a.tau / s.st : 0.0f;
    if (kind == kOne) ft += f1;
    const int full = n & ~7, l = fresh(tid);
    const Exponents x2(s.m0, c, a.c1, kind);
    if (zero || x2.far) {
        // element by element, in the places of the pass below (a row of zeros takes nothing from Z), written in
        // eights (no row of 8192 x 65536 bf16 with a weight: 405 us, element by element 738)
        for (int v = l * 8; v < n; v += ST) {
            float g[8] = {};
#pragma unroll
            for (int j = 0; j < 8; j++) {
                if (zero || v + j >= n) continue;
                const float f = at<DT>(z, v + j);
                g[j] = ft * exp2_(apart(f, s.m0, c));
                if (kind != kOne) g[j] = fmaf(f1, exp2_(apart(f, s.m0, a.c1)), g[j]);
            }
            if (v < full) {
                store8<DT>(dz + (int64_t)v * ES, pack8<DT>(g));
            } else {
#pragma unroll
                for (int j = 0; j < 7; j++)
                    if (v + j < n) store1<DT>(dz + (int64_t)(v + j) * ES, g[j]);
            }
        }
        if (zero) return;
    } else {
        // the factors take off what the exponents are too large by
        const float ht = ft * exp2_(-x2.t.off);
        const float h1 = f1 * exp2_(kind == kSquare ? -2.0f * x2.t.off : -x2.one.off);
        const uint32_t off = (uint32_t)l * (8 * ES);
        float last[8] = {};   // of the stride with the last, partial eight
        each8<DT, W, NV>(x, n, [&](int i, const float *f) {
            float g[8];
#pragma unroll
            for (int j = 0; j < 8; j++) g[j] = exp2_(x2.t.of(f[j]));
            if (kind == kSquare) {
#pragma unroll
                for (int j = 0; j < 8; j++) g[j] *= fmaf(h1, g[j], ht);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++) g[j] *= ht;
                if (kind == kTwo)
#pragma unroll
                    for (int j = 0; j < 8; j++) g[j] = fmaf(h1, exp2_(x2.one.of(f[j])), g[j]);
            }
            if (l * 8 < full - i * ST) store8<DT>(dz + i * ST * ES + off, pack8<DT>(g));
            if (i == full / ST)
#pragma unroll
                for (int j = 0; j < 7; j++) last[j] = g[j];
        });
        if (n & 7 && l == full % ST / 8)
#pragma unroll
            for (int j = 0; j < 7; j++)
                if (full + j < n) store1<DT>(dz + (int64_t)full * ES + j * ES, last[j]);
    }
    // the named tokens, by the wave that has just written them
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int r = 0; r < 2; r++) {
        const int j = r == 0 ? lane : kEntries - 1;
        const int v = e.id[j] - first;
        if ((r == 1 && lane != 0) || e.id[j] < 0 || v < 0 || v >= n || (v / 512) % W != wave) continue;
        float g = ft * exp2_(apart(e.z[j], s.m0, c));
        if (kind != kOne) g = fmaf(f1, exp2_(apart(e.z[j], s.m0, a.c1)), g);
        store1<DT>(dz + (int64_t)v * ES, fmaf(-w, e.less[j], g));
    }
}

// The row's sums from its parts', by a wave.
__device__ inline Sums join_sums(const DistillArgs &a, int64_t t, float c, Kind kind, int lane) {
    const float4 r = lane < a.S ? a.sums[t * a.S + lane] : float4{-kInf, 0.0f, 0.0f, 0.0f};
    const float m = wave_all<Max>(r.x);
    Sums q;
    q.m0 = m == -kInf ? 0.0f : m;
    q.st = at_least_one(wave_all<Add>(r.z * exp2_(apart(r.x, q.m0, c))));
    q.s1 = kind == kOne ? q.st : at_least_one(wave_all<Add>(r.y * exp2_(apart(r.x, q.m0, a.c1))));
    return q;
}

__device__ inline Kind kind_of(const DistillArgs &a) {
    return !(a.ce && a.kl) || a.tau == 1.0f ? kOne : a.tau == 2.0f ? kSquare : kTwo;
}

// PHASE 0: whole rows with dZ, a segment each.  1: a part's sums and the named logits.
// 2: the row's sums from its parts', loss and gradient.  3: whole rows without dZ.
template <int DT, int W, int NV, int PHASE>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W, 4) void distill_kernel(DistillArgs a) {
    constexpr int R = W == 1 ? 4 : 1;   // rows of a workgroup
    __shared__ Names names[R];
    __shared__ float sh[3][W];
    const int slot = R > 1 ? threadIdx.x >> 6 : 0, tid = R > 1 ? threadIdx.x & 63 : threadIdx.x, lane = tid & 63;
    Names &e = names[slot];
    const Kind kind = kind_of(a);
    const float c = a.kl ? a.ct : a.c1;
    const int64_t items = a.T * a.S;
    for (int64_t item = (int64_t)blockIdx.x * R + slot; item < items; item += (int64_t)gridDim.x * R) {
        const bool whole = PHASE == 0 || PHASE == 3;
        const int64_t t = whole ? item : item / a.S;
        const int begin = whole ? 0 : (int)(item - t * a.S) * a.part, end = min(begin + a.part, a.V);
        const char *row = (const char *)a.Z + t * a.ld * esize<DT>();
        Raw8<DT> x[NV];
        Sums q;
        auto largest_and_sums = [&](const char *z, int n, float &m, float &s1, float &st) {
            m = row_all<Max, W>(lane_max<DT, W, NV>(x, n), sh[0], tid);
            const float m0 = m == -kInf ? 0.0f : m;
            sums_of<DT, W, NV>(z, x, n, Exponents(m0, c, a.c1, kind), kind, tid, s1, st);
            row_sums<W>(s1, st, &sh[1], tid);
        };
        // the row's names before the row: loads come back in order, and the first wave needs them for
        // further ones (which the others wait for)
        Given names_in{};
        if (tid < 64) names_in = given(a, t, lane);
        __builtin_amdgcn_sched_barrier(0);
        if (PHASE == 2) {
            load_row<DT, W, NV>(row + (int64_t)begin * esize<DT>(), end - begin, tid, x);
            if (tid < 64) read_names<DT>(a, t, row, names_in, e, lane, true);
            q = join_sums(a, t, c, kind, lane);
        } else if (PHASE == 0) {
            load_row<DT, W, NV>(row, a.V, tid, x);
            if (tid < 64) read_names<DT>(a, t, row, names_in, e, lane, false);
            float m;
            largest_and_sums(row, a.V, m, q.s1, q.st);
            q.m0 = m == -kInf ? 0.0f : m;
            q.st = at_least_one(q.st);
            q.s1 = kind == kOne ? q.st : at_least_one(q.s1);
        } else {
            float M = -kInf, s1 = 0.0f, st = 0.0f;   // of the segments so far
            for (int first = begin; first < end; first += a.seg) {
                const int n = min(a.seg, end - first);
                const char *z = row + (int64_t)first * esize<DT>();
                load_row<DT, W, NV>(z, n, tid, x);
                if (first == begin && tid < 64) {
                    if (PHASE == 3) {
                        read_names<DT>(a, t, row, names_in, e, lane, false);
                    } else {   // the logits of the tokens that are named of this part
                        const int v = names_in.id, y = names_in.target;
                        if (v >= begin && v < end) a.named[t * kEntries + lane] = at<DT>(row, v);
                        if (lane == 0 && y >= begin && y < end)
                            a.named[t * kEntries + kEntries - 1] = at<DT>(row, y);
                    }
                }
                float m, p1, pt;
                largest_and_sums(z, n, m, p1, pt);
                // to the larger of the two largest
                const float both = fmaxf(M, m), b0 = both == -kInf ? 0.0f : both;
                st = fmaf(exp2_(apart(M, b0, c)), st, exp2_(apart(m, b0, c)) * pt);
                if (kind != kOne) s1 = fmaf(exp2_(apart(M, b0, a.c1)), s1, exp2_(apart(m, b0, a.c1)) * p1);
                M = both;
                meet<W>();
            }
            q = Sums{M == -kInf ? 0.0f : M, at_least_one(kind == kOne ? st : s1), at_least_one(st)};
            if (PHASE == 1 && tid == 0) a.sums[item] = float4{M, s1, st, 0.0f};
        }
        if (PHASE != 1) {
            meet<W>();   // the names are there
            if (a.loss && begin == 0 && tid < 64) write_loss(a, t, e, q, lane);
            if (PHASE != 3)
                write_grad<DT, W, NV>(a, t, row + (int64_t)begin * esize<DT>(), x, begin, end - begin, e, q, c, kind,
                                      tid);
            meet<W>();
        }
    }
}

// The loss alone of rows that were cut: a wave each.
template <int DT>
__global__ __launch_bounds__(64) void distill_loss_kernel(DistillArgs a) {
    __shared__ Names e;
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        read_names<DT>(a, t, nullptr, given(a, t, lane), e, lane, true);
        const Sums q = join_sums(a, t, a.kl ? a.ct : a.c1, kind_of(a), lane);
        meet<1>();
        write_loss(a, t, e, q, lane);
        meet<1>();
    }
}

}  // namespace kdev

namespace {

using kdev::DistillArgs;

int launched() { return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

// With dZ a part has to fit a workgroup's registers: up to 16 waves.  Without, four
// waves take segments in turn.
RowPlan plan_call(int32_t dt, int64_t T, int64_t V, bool grad) {
    return plan_rows(dt, T, V, grad ? 16 : 4, !grad);
}

size_t workspace_of(const RowPlan &p, int64_t T) {
    return p.S == 1 ? 0 : (size_t)T * ((size_t)p.S * 16 + kdev::kEntries * 4);
}

template <int32_t DT, int PHASE>
struct Launch {
    DistillArgs a;
    hipStream_t st;
    template <int W, int NV>
    void operator()() const {
        constexpr int R = W == 1 ? 4 : 1;
        const dim3 g((unsigned)std::min<int64_t>(cdiv_(a.T * a.S, R), kMaxGroups)), b(W == 1 ? 256 : 64 * W);
        hipLaunchKernelGGL((kdev::distill_kernel<DT, W, NV, PHASE>), g, b, 0, st, a);
    }
};

template <int32_t DT>
void run(const DistillArgs &a, const RowPlan &p, hipStream_t st) {
    if (a.S == 1) {
        if (a.dZ) with_plan<DT, 1, 16>(p, Launch<DT, 0>{a, st});
        else with_plan<DT, 1, 4>(p, Launch<DT, 3>{a, st});
        return;
    }
    // (parts are longer than one wave takes, and take eight at most)
    with_plan<DT, 4, 8>(p, Launch<DT, 1>{a, st});
    if (a.dZ) with_plan<DT, 4, 8>(p, Launch<DT, 2>{a, st});
    else
        hipLaunchKernelGGL(kdev::distill_loss_kernel<DT>, dim3((unsigned)std::min<int64_t>(a.T, kMaxGroups)), dim3(64), 0,
                           st, a);
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

size_t tern_distill_workspace_bytes(int64_t T, int64_t V) {
    if (!row_sizes_ok(T, V)) return 0;
    size_t most = 0;
    for (int32_t dt : {TERN_F32, TERN_BF16})
        for (bool grad : {false, true}) most = std::max(most, workspace_of(plan_call(dt, T, V, grad), T));
    return most;
}

int tern_distill(const void *Z, int64_t ld, int32_t z_dtype, int64_t T, int64_t V, const int64_t *targets, int32_t K,
                 const int64_t *teacher_ids, const float *teacher_logp, float alpha, float tau, const float *dloss,
                 float *loss, void *dZ, int64_t lddz, void *workspace, size_t workspace_bytes, void *stream) {
    if (!row_sizes_ok(T, V) || !row_stride_ok(ld, V) || (dZ && !row_stride_ok(lddz, V))) return TERN_ERR_SHAPE;
    if (z_dtype != TERN_F32 && z_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (K < 0 || K > TERN_TOP_MAX || !(alpha >= 0.0f && alpha <= 1.0f) || !(tau > 0.0f) || !factor_ok(1.0 / tau) ||
        !std::isfinite(tau * tau))
        return TERN_ERR_VALUE;
    if (T == 0 || (!loss && !dZ)) return TERN_OK;
    if (!Z || (K > 0 && (!teacher_ids || !teacher_logp))) return TERN_ERR_NULL;
    const RowPlan p = plan_call(z_dtype, T, V, dZ != nullptr);
    const size_t wsb = workspace_of(p, T);
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (off_by(Z, 16) || off_by(dZ, 16) || off_by(targets, 8) || off_by(teacher_ids, 8) || off_by(teacher_logp, 4) ||
        off_by(dloss, 4) || off_by(loss, 4) || off_by(workspace, 16))
        return TERN_ERR_ALIGN;
    const size_t es = z_dtype == TERN_BF16 ? 2 : 4;
    // every element of Z is read before its place in dZ is written, so dZ may be Z
    const bool in_place = dZ == Z && lddz == ld;
    const Mat outs[] = {{dZ, T, V, lddz, es}, vec(loss, T, 4), vec(workspace, (int64_t)wsb, 1)};
    const Mat ins[] = {vec(targets, T, 8), vec(teacher_ids, T * K, 8), vec(teacher_logp, T * K, 4), vec(dloss, T, 4),
                       {in_place ? nullptr : Z, T, V, ld, es}};
    if (any_overlap(outs, 3, ins, 5)) return TERN_ERR_ALIAS;
    int exponent;
    const float rest = 2.0f * std::frexp(tau, &exponent);
    DistillArgs a{Z, ld, lddz, T, (int)V, K, p.S, (int)p.part, (int)p.seg, targets, teacher_ids, teacher_logp, dloss, alpha, tau,
                  (float)rows::kLog2e, (float)(rows::kLog2e / tau), std::ldexp(1.0f, exponent - 2), rest, alpha > 0.0f && targets, alpha < 1.0f && K > 0, loss,
                  dZ, (float4 *)workspace, nullptr};
    if (p.S > 1) a.named = (float *)(a.sums + T * p.S);
    hipStream_t st = (hipStream_t)stream;
    if (z_dtype == TERN_BF16) run<TERN_BF16>(a, p, st);
    else run<TERN_F32>(a, p, st);
    return launched();
}

}  // extern "C"
