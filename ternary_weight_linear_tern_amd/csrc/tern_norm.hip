// tern_norm.hip -- layer norm of rows, forward and backward, with the residual
// add in front of it (C ABI in include/tern.h).
//
//   S = X + A,  mu = mean S,  r = 1 / sqrt(mean (S - mu)^2 + eps),
//   Y = (S - mu) r w + b
//   xh = (S - mu) r,  g = dY w:
//   dX = dS + r (g - mean g - xh mean (g xh)),  dw = sum_t dY xh,  db = sum_t dY
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
namespace ndev {

using namespace rows;

constexpr int kNone = 2;   // type code of an array that is not there

struct FwdArgs {
    const void *X, *A;
    const float *w, *b;
    void *S, *Y;
    float *stats;
    int64_t ldx, lda, lds, ldy, T;
    int C;
    float eps;
};

struct BwdArgs {
    const void *S, *dY, *dS;
    const float *stats, *w;
    void *dX;
    float *dw, *db;
    float *part;             // [groups][2][C]: dw and db of the groups' rows
    int64_t lds, lddy, ldds, lddx, T;
    int64_t groups, per;     // row groups and rows of a group
    int C;
};

template <int DT>
__device__ inline void get8(const void *p, int64_t row, int64_t ld, int c, float *f) {
    unpack8<DT>(load8<DT>((const char *)p + (row * ld + c) * esize<DT>()), f);
}
template <int DT>
__device__ inline void put8(void *p, int64_t row, int64_t ld, int c, const float *f) {
    store8<DT>((char *)p + (row * ld + c) * esize<DT>(), pack8<DT>(f));
}
__device__ inline void coef8(const float *p, int c, float fill, float *f) {
    if (p) {
        unpack8<TERN_F32>(load8<TERN_F32>(p + c), f);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j++) f[j] = fill;
    }
}

// Rows of any length: a workgroup a row, which it reads three times.
template <int XD, int AD, int YD>
__global__ __launch_bounds__(256) void norm_fwd_kernel(FwdArgs a) {
    __shared__ float sh[2][4];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float sum = 0.0f, sq = 0.0f;
        const void *src = a.X;
        int64_t ld = a.ldx;
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8];
            get8<XD>(a.X, t, a.ldx, c, x);
            if constexpr (AD != kNone) {
                float y[8];
                get8<AD>(a.A, t, a.lda, c, y);
#pragma unroll
                for (int j = 0; j < 8; j++) x[j] += y[j];
                put8<XD>(a.S, t, a.lds, c, x);
                unpack8<XD>(pack8<XD>(x), x);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) sum += x[j];
        }
        if constexpr (AD != kNone) src = a.S, ld = a.lds;   // each lane reads what it wrote
        const float mu = group_all<Add, 4>(sum, sh[0]) / (float)a.C;
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8];
            get8<XD>(src, t, ld, c, x);
#pragma unroll
            for (int j = 0; j < 8; j++) sq = fmaf(x[j] - mu, x[j] - mu, sq);
        }
        const float r = 1.0f / sqrtf(group_all<Add, 4>(sq, sh[1]) / (float)a.C + a.eps);
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8], w[8], b[8];
            get8<XD>(src, t, ld, c, x);
            coef8(a.w, c, 1.0f, w);
            coef8(a.b, c, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = fmaf((x[j] - mu) * r, w[j], b[j]);
            put8<YD>(a.Y, t, a.ldy, c, x);
        }
        if (a.stats && threadIdx.x == 0) *(float2 *)(a.stats + 2 * t) = float2{mu, r};
        __syncthreads();
    }
}

template <int SD, int DY, int DX>
__global__ __launch_bounds__(256) void norm_dx_kernel(BwdArgs a) {
    __shared__ float sh[2][4];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float2 st = *(const float2 *)(a.stats + 2 * t);
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8], g[8], w[8];
            get8<SD>(a.S, t, a.lds, c, x);
            get8<DY>(a.dY, t, a.lddy, c, g);
            coef8(a.w, c, 1.0f, w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                s1 = fmaf(g[j], w[j], s1);
                s2 = fmaf(g[j] * w[j], (x[j] - st.x) * st.y, s2);
            }
        }
        const float m1 = group_all<Add, 4>(s1, sh[0]) / (float)a.C, m2 = group_all<Add, 4>(s2, sh[1]) / (float)a.C;
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8], g[8], w[8], d[8] = {};
            get8<SD>(a.S, t, a.lds, c, x);
            get8<DY>(a.dY, t, a.lddy, c, g);
            coef8(a.w, c, 1.0f, w);
            if (a.dS) get8<DX>(a.dS, t, a.ldds, c, d);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float xh = (x[j] - st.x) * st.y;
                d[j] = fmaf(st.y, fmaf(g[j], w[j], -m1) - xh * m2, d[j]);
            }
            put8<DX>(a.dX, t, a.lddx, c, d);
        }
        __syncthreads();
    }
}

// dw and db of a group's rows, 64 columns a wave.
template <int SD, int DY>
__global__ __launch_bounds__(64) void norm_dw_kernel(BwdArgs a) {
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= a.C) return;
    for (int64_t g = blockIdx.y; g < a.groups; g += gridDim.y) {
        float dw = 0.0f, db = 0.0f;
        const int64_t t1 = min((g + 1) * a.per, a.T);
        for (int64_t t = g * a.per; t < t1; t++) {
            const float2 st = *(const float2 *)(a.stats + 2 * t);
            const float x = load1<SD>((const char *)a.S + (t * a.lds + c) * esize<SD>());
            const float d = load1<DY>((const char *)a.dY + (t * a.lddy + c) * esize<DY>());
            dw = fmaf(d, (x - st.x) * st.y, dw);
            db += d;
        }
        a.part[(g * 2) * a.C + c] = dw;
        a.part[(g * 2 + 1) * a.C + c] = db;
    }
}

// The groups' sums, in order.
__global__ __launch_bounds__(64) void norm_dw_sum_kernel(const float *part, int64_t groups, int C, float *dw, float *db) {
    const int c = blockIdx.x * 64 + threadIdx.x;
    if (c >= C) return;
    double s = 0.0, u = 0.0;
    for (int64_t g = 0; g < groups; g++) {
        s += part[(g * 2) * C + c];
        u += part[(g * 2 + 1) * C + c];
    }
    if (dw) dw[c] = (float)s;
    if (db) db[c] = (float)u;
}

}  // namespace ndev

namespace {

using ndev::BwdArgs;
using ndev::FwdArgs;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }
bool type_ok(int32_t dt) { return dt == TERN_F32 || dt == TERN_BF16; }
size_t esize(int32_t dt) { return dt == TERN_BF16 ? 2 : 4; }
int launched() { return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

bool sizes_ok(int64_t T, int64_t C) { return T >= 0 && T <= kMaxT && C >= 0 && C <= kMaxInOut && C % 8 == 0; }
bool stride_ok(int64_t ld, int64_t C) { return ld >= C && ld % 8 == 0 && ld <= kMaxInOut * 8; }

struct BwdPlan {
    int64_t groups, per;   // row groups of the weight's gradient, rows of one
};
BwdPlan plan_bwd(int64_t T) {
    BwdPlan p;
    p.per = std::max<int64_t>(8, cdiv(T, 512));
    p.groups = cdiv(T, p.per);
    return p;
}

// f with a type code as a compile-time constant
template <class F>
void with_type(int32_t dt, F f) {
    if (dt == TERN_BF16) f(std::integral_constant<int, TERN_BF16>{});
    else f(std::integral_constant<int, TERN_F32>{});
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

size_t tern_norm_bwd_workspace_bytes(int64_t T, int64_t C) {
    if (!sizes_ok(T, C)) return 0;
    return (size_t)plan_bwd(T).groups * (size_t)C * 8;
}

int tern_norm_fwd(const void *X, int64_t ldx, int32_t x_dtype, const void *A, int64_t lda, int32_t a_dtype,
                  const float *w, const float *b, float eps, int64_t T, int64_t C, void *S, int64_t lds, void *Y,
                  int64_t ldy, int32_t y_dtype, float *stats, void *stream) {
    if (!sizes_ok(T, C) || !stride_ok(ldx, C) || !stride_ok(ldy, C)) return TERN_ERR_SHAPE;
    if ((A || S) && (!stride_ok(lda, C) || !stride_ok(lds, C))) return TERN_ERR_SHAPE;
    if (!type_ok(x_dtype) || !type_ok(y_dtype) || (A && !type_ok(a_dtype))) return TERN_ERR_DTYPE;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return TERN_ERR_VALUE;
    if (T == 0 || C == 0) return TERN_OK;
    if (!X || !Y || !A != !S) return TERN_ERR_NULL;
    if (misaligned(X) || misaligned(A) || misaligned(S) || misaligned(Y) || misaligned(w) || misaligned(b) ||
        ((uintptr_t)stats & 7u))
        return TERN_ERR_ALIGN;
    const size_t xs = esize(x_dtype);
    // every lane reads its elements of X before it writes them to S, so S may be X
    const bool in_place = S == X && lds == ldx;
    const Mat outs[] = {{Y, T, C, ldy, esize(y_dtype)}, {S, T, C, lds, xs}, {stats, 1, 2 * T, 2 * T, 4}};
    const Mat ins[] = {{A, T, C, lda, A ? esize(a_dtype) : 0}, {w, 1, C, C, 4}, {b, 1, C, C, 4},
                       {in_place ? nullptr : X, T, C, ldx, xs}};
    if (any_overlap(outs, 3, ins, 4)) return TERN_ERR_ALIAS;
    FwdArgs a{X, A, w, b, S, Y, stats, ldx, lda, lds, ldy, T, (int)C, eps};
    hipStream_t st = (hipStream_t)stream;
    const dim3 grid((unsigned)std::min<int64_t>(T, 65536));
    with_type(x_dtype, [&](auto xd) {
        with_type(y_dtype, [&](auto yd) {
            constexpr int XD = decltype(xd)::value, YD = decltype(yd)::value;
            if (!A) hipLaunchKernelGGL((ndev::norm_fwd_kernel<XD, ndev::kNone, YD>), grid, dim3(256), 0, st, a);
            else
                with_type(a_dtype, [&](auto ad) {
                    constexpr int AD = decltype(ad)::value;
                    hipLaunchKernelGGL((ndev::norm_fwd_kernel<XD, AD, YD>), grid, dim3(256), 0, st, a);
                });
        });
    });
    return launched();
}

int tern_norm_bwd(const void *S, int64_t lds, int32_t s_dtype, const float *stats, const float *w, const void *dY,
                  int64_t lddy, int32_t dy_dtype, const void *dS, int64_t ldds, int64_t T, int64_t C, void *dX,
                  int64_t lddx, int32_t dx_dtype, float *dw, float *db, void *workspace, size_t workspace_bytes,
                  void *stream) {
    if (!sizes_ok(T, C) || !stride_ok(lds, C) || !stride_ok(lddy, C) || !stride_ok(lddx, C) ||
        (dS && !stride_ok(ldds, C)))
        return TERN_ERR_SHAPE;
    if (!type_ok(s_dtype) || !type_ok(dy_dtype) || !(dx_dtype == TERN_F32 || (dx_dtype == TERN_BF16 && s_dtype == TERN_BF16)))
        return TERN_ERR_DTYPE;
    if (C == 0) return TERN_OK;
    if (T > 0 && (!S || !stats || !dY || !dX)) return TERN_ERR_NULL;
    const bool weights = dw || db;
    const BwdPlan p = plan_bwd(T);
    const size_t wsb = weights ? (size_t)p.groups * (size_t)C * 8 : 0;
    if (wsb && (!workspace || workspace_bytes < wsb)) return TERN_ERR_WORKSPACE;
    if (misaligned(S) || misaligned(w) || misaligned(dY) || misaligned(dS) || misaligned(dX) || misaligned(dw) ||
        misaligned(db) || misaligned(workspace) || ((uintptr_t)stats & 7u))
        return TERN_ERR_ALIGN;
    const size_t xs = esize(dx_dtype);
    // every lane reads its elements of dS before it writes them to dX, so dX may be dS
    const bool in_place = dS == dX && ldds == lddx;
    const Mat outs[] = {{dX, T, C, lddx, xs}, {dw, 1, C, C, 4}, {db, 1, C, C, 4},
                        {workspace, 1, (int64_t)wsb, (int64_t)wsb, 1}};
    const Mat ins[] = {{S, T, C, lds, esize(s_dtype)}, {stats, 1, 2 * T, 2 * T, 4}, {w, 1, C, C, 4},
                       {dY, T, C, lddy, esize(dy_dtype)}, {in_place ? nullptr : dS, T, C, ldds, xs}};
    if (any_overlap(outs, 4, ins, 5)) return TERN_ERR_ALIAS;
    if (T == 0 && !weights) return TERN_OK;
    BwdArgs a{S, dY, dS, stats, w, dX, dw, db, (float *)workspace, lds, lddy, ldds, lddx, T, p.groups, p.per, (int)C};
    hipStream_t st = (hipStream_t)stream;
    const unsigned cols = (unsigned)cdiv(C, 64);
    if (T > 0) {
        const dim3 grid((unsigned)std::min<int64_t>(T, 65536)), gw(cols, (unsigned)std::min<int64_t>(p.groups, 65535));
        with_type(s_dtype, [&](auto sd) {
            with_type(dy_dtype, [&](auto yd) {
                constexpr int SD = decltype(sd)::value, DY = decltype(yd)::value;
                with_type(dx_dtype, [&](auto xd) {
                    constexpr int DX = decltype(xd)::value;
                    if constexpr (DX == TERN_F32 || SD == TERN_BF16)
                        hipLaunchKernelGGL((ndev::norm_dx_kernel<SD, DY, DX>), grid, dim3(256), 0, st, a);
                });
                if (weights) hipLaunchKernelGGL((ndev::norm_dw_kernel<SD, DY>), gw, dim3(64), 0, st, a);
            });
        });
    }
    if (weights)
        hipLaunchKernelGGL(ndev::norm_dw_sum_kernel, dim3(cols), dim3(64), 0, st, a.part, p.groups, a.C, dw, db);
    return launched();
}

}  // extern "C"
