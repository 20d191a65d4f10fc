// tern_head.hip -- what stands behind the head's logits: log probabilities of
// tokens with entropy and top alternatives, and the distillation loss with its
// gradient (C ABI and formulas in include/tern.h).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/tern.h"
#include "tern_mat.h"
#include "tern_plan.h"
#include "tern_rows.h"

namespace tern {
namespace hdev {

using namespace rows;

constexpr float kInf = __builtin_inff();
constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;
constexpr int kWaves = 4;

struct LogprobArgs {
    const void *Z;
    int64_t ld, T;
    int V, k;
    float scale, c;          // c = scale log2 e
    const int64_t *tokens;
    float *logp, *entropy, *lse;
    int64_t *top_ids;
    float *top_logp;
};

struct DistillArgs {
    const void *Z;
    int64_t ld, lddz, T;
    int V, K;
    const int64_t *targets, *ids;
    const float *lp, *dloss;
    float alpha, tau;
    float *loss;
    void *dZ;
};

__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Bits that order as the values do, -0 as +0, NaN outermost.
__device__ inline uint32_t ordered(float f) {
    const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float from_ordered(uint32_t o) {
    return __builtin_bit_cast(float, o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// The value, then the lower index.
__device__ inline uint64_t key_of(float f, uint32_t i) { return (uint64_t)ordered(f) << 32 | (0xFFFFFFFFu - i); }

__device__ inline uint64_t wave_max(uint64_t x) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint64_t y = __shfl_xor((unsigned long long)x, d);
        x = y > x ? y : x;
    }
    return x;
}

template <int DT>
__device__ inline float at(const void *z, int64_t v) { return load1<DT>((const char *)z + v * esize<DT>()); }

template <int DT>
__global__ __launch_bounds__(64 * kWaves) void logprob_kernel(LogprobArgs a) {
    __shared__ float sh[3][kWaves];
    __shared__ uint64_t sk[2][kWaves];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const char *z = (const char *)a.Z + t * a.ld * esize<DT>();
        float m = -kInf, s = 0.0f, u = 0.0f;
        for (int v = threadIdx.x; v < a.V; v += 64 * kWaves) m = fmaxf(m, at<DT>(z, v));
        m = group_all<Max, kWaves>(m, sh[0]);
        const float m0 = m == -kInf ? 0.0f : m;
        for (int v = threadIdx.x; v < a.V; v += 64 * kWaves) {
            // in units of log 2, from the largest on: no product of a large logit, which could overflow
            const float d = (at<DT>(z, v) - m0) * a.c, e = exp2_(d);
            s += e;
            u = fmaf(e, fmaxf(d, -200.0f), u);
        }
        s = group_all<Add, kWaves>(s, sh[1]);
        u = group_all<Add, kWaves>(u, sh[2]);
        const double logs = log2((double)s) * kLn2;
        if (threadIdx.x == 0) {
            if (a.lse) a.lse[t] = (float)((double)m0 * a.scale + logs);
            if (a.entropy) a.entropy[t] = s == 0.0f ? 0.0f : (float)(logs - (double)u / s * kLn2);
            if (a.tokens) {
                const int64_t y = a.tokens[t];
                float lp = 0.0f;
                if (y >= 0 && y < a.V) lp = s == 0.0f ? -kInf : (float)(((double)at<DT>(z, y) - m0) * a.scale - logs);
                a.logp[t] = lp;
            }
        }
        uint64_t last = ~(uint64_t)0;
        for (int j = 0; j < a.k; j++) {
            uint64_t best = 0;
            for (int v = threadIdx.x; v < a.V; v += 64 * kWaves) {
                const uint64_t key = key_of(at<DT>(z, v), v);
                if (key < last && key > best) best = key;
            }
            best = wave_max(best);
            if ((threadIdx.x & 63) == 0) sk[j & 1][threadIdx.x >> 6] = best;
            __syncthreads();
            for (int i = 0; i < kWaves; i++) best = sk[j & 1][i] > best ? sk[j & 1][i] : best;
            last = best;
            if (threadIdx.x == 0) {
                const float f = from_ordered((uint32_t)(best >> 32));
                a.top_ids[t * a.k + j] = 0xFFFFFFFFu - (uint32_t)best;
                a.top_logp[t * a.k + j] = s == 0.0f ? -kInf : (float)(((double)f - m0) * a.scale - logs);
            }
        }
        __syncthreads();
    }
}

template <int DT>
__global__ __launch_bounds__(64 * kWaves) void distill_kernel(DistillArgs a) {
    __shared__ float sh[3][kWaves];
    __shared__ float sz[TERN_TOP_MAX], sp[TERN_TOP_MAX], szy;
    __shared__ int sid[TERN_TOP_MAX];
    const int lane = threadIdx.x & 63;
    const float c1 = (float)kLog2e, ct = (float)(kLog2e / a.tau);
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const char *z = (const char *)a.Z + t * a.ld * esize<DT>();
        // the teacher's entries
        int64_t id = -1;
        float lp = -kInf;
        if (lane < a.K && a.alpha < 1.0f) {
            id = a.ids[t * a.K + lane];
            lp = a.lp[t * a.K + lane];
            if (id < 0 || id >= a.V || lp == -kInf) id = -1, lp = -kInf;
        }
        const float lm = wave_all<Max>(lp);
        float p = id < 0 ? 0.0f : exp2_((lp - lm) * c1);
        const float ps = wave_all<Add>(p);
        const bool kl = __ballot(id >= 0) != 0;
        p = id < 0 ? 0.0f : p / ps;
        const float logp = id < 0 ? 0.0f : lp - lm - logf(ps);
        int64_t y = a.targets && a.alpha > 0.0f ? a.targets[t] : -1;
        if (y >= a.V) y = -1;
        const bool ce = y >= 0;
        if (threadIdx.x < 64 && lane < TERN_TOP_MAX) {
            sid[lane] = (int)id;
            sp[lane] = p;
            sz[lane] = id >= 0 ? at<DT>(z, id) : 0.0f;
        }
        if (threadIdx.x == 0) szy = ce ? at<DT>(z, y) : 0.0f;
        float m = -kInf, s1 = 0.0f, st = 0.0f;
        for (int v = threadIdx.x; v < a.V; v += 64 * kWaves) m = fmaxf(m, at<DT>(z, v));
        m = group_all<Max, kWaves>(m, sh[0]);
        const float m0 = m == -kInf ? 0.0f : m;
        for (int v = threadIdx.x; v < a.V; v += 64 * kWaves) {
            const float x = at<DT>(z, v) - m0;
            s1 += exp2_(x * c1);
            st += exp2_(x * ct);
        }
        s1 = group_all<Add, kWaves>(s1, sh[1]);
        st = group_all<Add, kWaves>(st, sh[2]);
        const float zid = sz[lane], zy = szy;
        if (a.loss && threadIdx.x < 64) {
            double k = 0.0;
            if (kl && id >= 0 && p != 0.0f)
                k = st == 0.0f ? (double)kInf
                               : (double)p * ((double)logp - ((double)zid - m0) / a.tau + log2((double)st) * kLn2);
            for (int d = 1; d < 64; d *= 2) k += __shfl_xor(k, d);
            double h = 0.0;
            if (ce) h = s1 == 0.0f ? (double)kInf : log2((double)s1) * kLn2 - ((double)zy - m0);
            if (lane == 0)
                a.loss[t] = (float)((ce ? a.alpha * h : 0.0) + (kl ? (1.0 - a.alpha) * (double)a.tau * a.tau * k : 0.0));
        }
        if (a.dZ) {
            const float w = a.dloss ? a.dloss[t] : 1.0f;
            const bool zero = w == 0.0f || !(kl || ce);
            const float f1 = ce ? (s1 == 0.0f ? 0.0f : w * a.alpha / s1) : 0.0f;
            const float ft = kl ? (st == 0.0f ? 0.0f : w * (1.0f - a.alpha) * a.tau / st) : 0.0f;
            char *dz = (char *)a.dZ + t * a.lddz * esize<DT>();
            for (int v = threadIdx.x; v < a.V; v += 64 * kWaves) {
                const float x = at<DT>(z, v) - m0;
                float g = ce ? f1 * exp2_(x * c1) : 0.0f;
                if (kl) g += ft * exp2_(x * ct);
                if (v == y) g -= w * a.alpha;
                if (kl)
                    for (int j = 0; j < a.K; j++)
                        if (sid[j] == v) g -= w * (1.0f - a.alpha) * a.tau * sp[j];
                store1<DT>(dz + (int64_t)v * esize<DT>(), zero ? 0.0f : g);
            }
        }
        __syncthreads();
    }
}

}  // namespace hdev

namespace {

using hdev::DistillArgs;
using hdev::LogprobArgs;

bool misaligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) != 0; }
size_t esize(int32_t dt) { return dt == TERN_BF16 ? 2 : 4; }
int launched() { return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

bool sizes_ok(int64_t T, int64_t V) { return T >= 0 && T <= kMaxT && V >= 1 && V <= kMaxInOut; }
bool stride_ok(int64_t ld, int64_t V) { return ld >= V && ld % 8 == 0 && ld <= kMaxInOut * 8; }
// a factor of the logits and its product with log2 e, above 0 and finite
bool factor_ok(double x) { return x > 0.0 && x * hdev::kLog2e <= 3.4e38; }

Mat vec(const void *p, int64_t n, size_t es) { return {p, 1, n, n, es}; }

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

size_t tern_logprob_workspace_bytes(int64_t T, int64_t V, int32_t k) {
    (void)T, (void)V, (void)k;
    return 0;
}

int tern_logprob(const void *Z, int64_t ld, int32_t z_dtype, float scale, int64_t T, int64_t V, const int64_t *tokens,
                 float *logp, float *entropy, float *lse, int32_t k, int64_t *top_ids, float *top_logp,
                 void *workspace, size_t workspace_bytes, void *stream) {
    if (!sizes_ok(T, V) || !stride_ok(ld, V)) return TERN_ERR_SHAPE;
    if (z_dtype != TERN_F32 && z_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (!factor_ok(scale) || k < 0 || k > TERN_TOP_MAX || k > V) return TERN_ERR_VALUE;
    if (T == 0) return TERN_OK;
    if (!Z || !tokens != !logp || (k > 0 && (!top_ids || !top_logp))) return TERN_ERR_NULL;
    const size_t wsb = tern_logprob_workspace_bytes(T, V, k);
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (misaligned(Z, 16) || misaligned(tokens, 8) || misaligned(top_ids, 8) || misaligned(logp, 4) ||
        misaligned(entropy, 4) || misaligned(lse, 4) || misaligned(top_logp, 4) || misaligned(workspace, 16))
        return TERN_ERR_ALIGN;
    const Mat outs[] = {vec(logp, T, 4), vec(entropy, T, 4), vec(lse, T, 4), vec(top_ids, T * k, 8),
                        vec(top_logp, T * k, 4), vec(workspace, (int64_t)wsb, 1)};
    const Mat ins[] = {{Z, T, V, ld, esize(z_dtype)}, vec(tokens, T, 8)};
    if (any_overlap(outs, 6, ins, 2)) return TERN_ERR_ALIAS;
    LogprobArgs a{Z, ld, T, (int)V, k, scale, (float)(scale * hdev::kLog2e), tokens, logp, entropy, lse, top_ids,
                  top_logp};
    const dim3 g((unsigned)std::min<int64_t>(T, 65536)), b(64 * hdev::kWaves);
    hipStream_t st = (hipStream_t)stream;
    if (z_dtype == TERN_BF16) hipLaunchKernelGGL(hdev::logprob_kernel<TERN_BF16>, g, b, 0, st, a);
    else hipLaunchKernelGGL(hdev::logprob_kernel<TERN_F32>, g, b, 0, st, a);
    return launched();
}

size_t tern_distill_workspace_bytes(int64_t T, int64_t V) {
    (void)T, (void)V;
    return 0;
}

int tern_distill(const void *Z, int64_t ld, int32_t z_dtype, int64_t T, int64_t V, const int64_t *targets, int32_t K,
                 const int64_t *teacher_ids, const float *teacher_logp, float alpha, float tau, const float *dloss,
                 float *loss, void *dZ, int64_t lddz, void *workspace, size_t workspace_bytes, void *stream) {
    if (!sizes_ok(T, V) || !stride_ok(ld, V) || (dZ && !stride_ok(lddz, V))) return TERN_ERR_SHAPE;
    if (z_dtype != TERN_F32 && z_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (K < 0 || K > TERN_TOP_MAX || !(alpha >= 0.0f && alpha <= 1.0f) || !(tau > 0.0f) ||
        !factor_ok(1.0 / tau) || !std::isfinite(tau * tau))
        return TERN_ERR_VALUE;
    if (T == 0 || (!loss && !dZ)) return TERN_OK;
    if (!Z || (K > 0 && (!teacher_ids || !teacher_logp))) return TERN_ERR_NULL;
    const size_t wsb = tern_distill_workspace_bytes(T, V);
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (misaligned(Z, 16) || misaligned(dZ, 16) || misaligned(targets, 8) || misaligned(teacher_ids, 8) ||
        misaligned(teacher_logp, 4) || misaligned(dloss, 4) || misaligned(loss, 4) || misaligned(workspace, 16))
        return TERN_ERR_ALIGN;
    const size_t es = esize(z_dtype);
    // every element of Z is read before its place in dZ is written, so dZ may be Z
    const bool in_place = dZ == Z && lddz == ld;
    const Mat outs[] = {{dZ, T, V, lddz, es}, vec(loss, T, 4), vec(workspace, (int64_t)wsb, 1)};
    const Mat ins[] = {vec(targets, T, 8), vec(teacher_ids, T * K, 8), vec(teacher_logp, T * K, 4), vec(dloss, T, 4),
                       {in_place ? nullptr : Z, T, V, ld, es}};
    if (any_overlap(outs, 3, ins, 5)) return TERN_ERR_ALIAS;
    DistillArgs a{Z, ld, lddz, T, (int)V, K, targets, teacher_ids, teacher_logp, dloss, alpha, tau, loss, dZ};
    const dim3 g((unsigned)std::min<int64_t>(T, 65536)), b(64 * hdev::kWaves);
    hipStream_t st = (hipStream_t)stream;
    if (z_dtype == TERN_BF16) hipLaunchKernelGGL(hdev::distill_kernel<TERN_BF16>, g, b, 0, st, a);
    else hipLaunchKernelGGL(hdev::distill_kernel<TERN_F32>, g, b, 0, st, a);
    return launched();
}

}  // extern "C"
