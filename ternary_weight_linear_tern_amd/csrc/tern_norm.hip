// tern_norm.hip -- layer norm of rows, forward and backward, with the residual
// add in front of it (C ABI in include/tern.h).
//
//   S = X + A,  mu = mean S,  r = 1 / sqrt(mean (S - mu)^2 + eps),
//   Y = (S - mu) r w + b
//   xh = (S - mu) r,  g = dY w:
//   dX = dS + r (g - mean g - xh mean (g xh)),  dw = sum_t dY xh,  db = sum_t dY
//
// Some ten operations an element: HBM bounds both, as long as each row is read once.
// So rows of up to 16384 columns stay in registers between their sums and their
// results, the backward sums dw and db from the same registers, and the next rows are
// loaded meanwhile.  Forward, 16384 x 2048, fp32 + fp32 to fp32 and bf16: 91 us, 5.1 TB/s;
// backward, 32768 x 4096, bf16 with fp32 dY, dS and dX: 357 us, 5.3 TB/s, of which 5 are the
// second launch, which adds up the groups' dw and db.  (Three passes over each row, and
// dw and db from passes of their own: 109 and 721.)  Few rows are bound by the launches:
// 32 x 2048 forward 3.4 us, 2048 x 512 backward 7.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/tern.h"
#include "tern_mat.h"
#include "tern_plan.h"
#include "tern_rows.h"

namespace tern {
namespace ldev {

using namespace rows;

struct FwdArgs {
    const void *X, *A;
    const float *w, *b;
    void *S, *Y;
    float *stats;
    int64_t ldx, lda, lds, ldy, T;
    int C, W, P, a_dtype;
    float eps;
};

struct BwdArgs {
    const void *S, *dY, *dS;
    const float *stats, *w;
    void *dX;
    float *dw, *db;
    float *part;             // [groups][2][C]: dw and db of the groups' rows
    int64_t lds, lddy, ldds, lddx, T;
    int64_t groups;          // row groups, a workgroup each
    int C, W, P;
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

// An eight of A, which has a type of its own: told by a uniform branch.
struct RawA {
    Raw8<TERN_F32> r;
    __device__ void load(const void *A, int dt, int64_t row, int64_t ld, int c) {
        if (dt == TERN_BF16) r.v[0] = load8<TERN_BF16>((const char *)A + (row * ld + c) * 2).v[0];
        else r = load8<TERN_F32>((const char *)A + (row * ld + c) * 4);
    }
    __device__ void add_to(int dt, float *x) const {
        float f[8];
        if (dt == TERN_BF16) unpack8<TERN_BF16>(Raw8<TERN_BF16>{{r.v[0]}}, f);
        else unpack8<TERN_F32>(r, f);
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] += f[j];
    }
};

// How a workgroup takes rows of up to 16 * 512 * CV columns: W waves a row, eight
// neighbours a lane, CV times; rows of 256 columns and fewer take P = 8, 16 or 32
// lanes of one wave (65536 rows of 64 in bf16: forward 30.6 us with a
// wave each, 10.0 with 8 lanes; backward 30.7 and 16.0).  R rows at once.
// (P is a variable in kernels of their own: that costs the others some per cent.)
template <bool NARROW>
struct Lanes {
    int W, P, R, slot, tid, wave;   // this lane's row among the R, its number and its wave in the row
    __device__ Lanes(int waves, int lanes) : W(NARROW ? 1 : waves), P(NARROW ? lanes : 64) {
        R = (int)blockDim.x / (P * W);
        if (!NARROW) {
            const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
            slot = w / W;
            wave = w - slot * W;
            tid = wave * 64 + (int)(threadIdx.x & 63);
        } else {
            slot = (int)threadIdx.x / P;
            wave = 0;
            tid = (int)threadIdx.x & (P - 1);
        }
    }
    __device__ int col(int v) const { return (v * W * P + tid) * 8; }
    // columns of wave w of a row
    template <int CV>
    __device__ float columns(int w, int C) const {
        int n = 0;
#pragma unroll
        for (int v = 0; v < CV; v++) n += min(max(C - (v * W + w) * 512, 0), 512);
        return (float)n;
    }
};
// Rows whose squares pass fp32's range (differences above about 1e19), told by sums that do, take
// them of their values times 2^-80: squares of any differences, and sums of 2^20 of those, fit.
constexpr float kFar = 0x1p-80f;
constexpr float kFarSquares = 0x1p-33f, kFarSum = 0x1p47f;   // of those values: half of what passes the range
constexpr float kInf = __builtin_inff();

// xh = (x k - mu) r: a row's mean and 1 / deviation in units of 1 / k, in which the difference of any two
// numbers and 1 / deviation fit: k is 1, or 1/16 for a far row (sq: of its values times 2^-80).
struct RowStats {
    float k, mu, r;
    __device__ RowStats(float mean, float sq, float C, float eps, bool far) : k(1.0f), mu(mean) {
        if (far) {
            k = 0.0625f, mu = mean * 0x1p76f;
            // deviation and sqrt(eps) times 2^-68 (equal values leave no deviation, and no eps that has a square)
            const float e = fmaxf(sqrtf(eps) * 0x1p-68f, 0x1p-126f), q = fmaf(sq / C, 0x1p24f, e * e);
            r = 0x1p-64f / (q == 0.0f ? e : sqrtf(q));
        } else {
            r = 1.0f / sqrtf(sq / C + eps);
        }
    }
    __device__ float of(float x) const { return fmaf(x, k, -mu) * r; }
    __device__ float2 as_stored() const { return float2{mu / k, r * k}; }
};
// xh in the backward, by halves: the difference of any two numbers fits
struct Hat {
    float mu, r;   // -mu / 2, 2 r
    __device__ Hat(float2 stats) : mu(-0.5f * stats.x), r(2.0f * stats.y) {}
    __device__ float of(float x) const { return fmaf(x, 0.5f, mu) * r; }
};

constexpr int kMaxWaves = 16;
constexpr int kTogether = 8;   // waves of a backward workgroup that has several rows

// The far rows of a wave, after the others: once more, from what is stored of them (a row's S by all its
// waves, before they met).  Each wave takes the sums over all columns, and writes its own columns again.
template <int XD, int YD, int CV, bool NARROW>
__device__ void norm_far_rows(const FwdArgs &a, const Lanes<NARROW> &l) {
    const void *src = a.A ? a.S : a.X;
    const int64_t ld = a.A ? a.lds : a.ldx, step = (int64_t)gridDim.x * l.R;
    const int lane = l.tid & (l.P - 1);
    for (int64_t t0 = (int64_t)blockIdx.x * l.R; t0 < a.T; t0 += step) {
        const int64_t t = t0 + l.slot;
        const bool here = t < a.T;
        auto sum = [&](auto of) {
            float s = 0.0f;
            for (int c = lane * 8; here && c < a.C; c += l.P * 8) {
                float x[8];
                get8<XD>(src, t, ld, c, x);
#pragma unroll
                for (int j = 0; j < 8; j++) s += of(x[j] * kFar);
            }
            return lanes_all<Add>(s, l.P);
        };
        const float all = sum([](float x) { return x; }), mu = all / (float)a.C;
        const float sq = sum([&](float x) { return (x - mu) * (x - mu); });
        if (!here || (sq < kFarSquares && fabsf(all) < kFarSum)) continue;
        const RowStats st(mu, sq, (float)a.C, a.eps, true);
#pragma unroll 1
        for (int v = 0; v < CV; v++) {
            int c = l.col(v);
            asm volatile("" : "+v"(c));   // (w and b are loaded again, not kept from the rows before)
            if (c >= a.C) continue;
            float x[8], w[8], b[8];
            get8<XD>(src, t, ld, c, x);
            coef8(a.w, c, 1.0f, w);
            coef8(a.b, c, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = fmaf(st.of(x[j]), w[j], b[j]);
            put8<YD>(a.Y, t, a.ldy, c, x);
        }
        if (a.stats && l.tid == 0) *(float2 *)(a.stats + 2 * t) = st.as_stored();
    }
}

// Rows in registers.  A workgroup goes on to further rows, with w and b in
// registers and, where they leave room (CV 1), the next rows' loads under way.  Each
// wave takes the mean of its columns and the squares around that; the waves'
// meet by n_i (mu_i - mu)^2: one barrier for R rows.
template <int XD, int YD, int CV, bool NARROW>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_fwd_rows_kernel(FwdArgs a) {
    __shared__ float2 sh[2][kMaxWaves];
    const Lanes<NARROW> l(a.W, a.P);
    float w[CV][8], b[CV][8];
#pragma unroll
    for (int v = 0; v < CV; v++)
        if (l.col(v) < a.C) {
            coef8(a.w, l.col(v), 1.0f, w[v]);
            coef8(a.b, l.col(v), 0.0f, b[v]);
        }
    Raw8<XD> nx[CV];
    RawA na[CV];
    auto fetch = [&](int64_t t) {
        if (t >= a.T) return;
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (l.col(v) < a.C) {
                nx[v] = load8<XD>((const char *)a.X + (t * a.ldx + l.col(v)) * esize<XD>());
                if (a.A) na[v].load(a.A, a.a_dtype, t, a.lda, l.col(v));
            }
    };
    const int64_t step = (int64_t)gridDim.x * l.R;
    const float n = l.template columns<CV>(l.wave, a.C);
    if (CV == 1) fetch((int64_t)blockIdx.x * l.R + l.slot);
    int turn = 0;
    uint64_t far = 0;   // (told, not taken here: a branch in this loop costs 2 to 6 per cent)
    for (int64_t t0 = (int64_t)blockIdx.x * l.R; t0 < a.T; t0 += step, turn ^= 1) {
        const int64_t t = t0 + l.slot;
        const bool here = t < a.T;
        if (CV > 1) fetch(t);
        float x[CV][8], sum = 0.0f, sq = 0.0f;
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (here && l.col(v) < a.C) {
                unpack8<XD>(nx[v], x[v]);
                if (a.A) {
                    na[v].add_to(a.a_dtype, x[v]);
                    const Raw8<XD> s = pack8<XD>(x[v]);   // the norm is that of S as stored
                    store8<XD>((char *)a.S + (t * a.lds + l.col(v)) * esize<XD>(), s);
                    unpack8<XD>(s, x[v]);
                }
#pragma unroll
                for (int j = 0; j < 8; j++) sum += x[v][j];
            }
        if (CV == 1) fetch(t + step);
        float mu = lanes_all<Add>(sum, l.P) / fmaxf(n, 1.0f);
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (here && l.col(v) < a.C)
#pragma unroll
                for (int j = 0; j < 8; j++) sq = fmaf(x[v][j] - mu, x[v][j] - mu, sq);
        sq = lanes_all<Add>(sq, l.P);
        if (!NARROW && l.W > 1) {
            const float2 *of = &sh[turn][l.slot * l.W];
            if ((threadIdx.x & 63) == 0) sh[turn][l.slot * l.W + l.wave] = float2{mu, sq};
            __syncthreads();
            float m = 0.0f;
            for (int i = 0; i < l.W; i++) m = fmaf(l.template columns<CV>(i, a.C), of[i].x, m);
            mu = m / (float)a.C;
            sq = 0.0f;
            for (int i = 0; i < l.W; i++) {
                const float d = of[i].x - mu;
                sq += fmaf(l.template columns<CV>(i, a.C) * d, d, of[i].y);
            }
        }
        far |= __ballot(!(sq < kInf));
        const float r = 1.0f / sqrtf(sq / (float)a.C + a.eps);
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (here && l.col(v) < a.C) {
#pragma unroll
                for (int j = 0; j < 8; j++) x[v][j] = fmaf((x[v][j] - mu) * r, w[v][j], b[v][j]);
                store8<YD>((char *)a.Y + (t * a.ldy + l.col(v)) * esize<YD>(), pack8<YD>(x[v]));
            }
        if (a.stats && here && l.tid == 0) *(float2 *)(a.stats + 2 * t) = float2{mu, r};
    }
    if (far) norm_far_rows<XD, YD, CV, NARROW>(a, l);
}

// Rows of any length: a workgroup a row, which it reads three times.
template <int XD, int YD>
__global__ __launch_bounds__(256) void norm_fwd_kernel(FwdArgs a) {
    __shared__ float sh[2][4];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float sum = 0.0f;
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8];
            get8<XD>(a.X, t, a.ldx, c, x);
            if (a.A) {
                RawA y;
                y.load(a.A, a.a_dtype, t, a.lda, c);
                y.add_to(a.a_dtype, x);
                put8<XD>(a.S, t, a.lds, c, x);
                unpack8<XD>(pack8<XD>(x), x);
            }
#pragma unroll
            for (int j = 0; j < 8; j++) sum += x[j];
        }
        const void *src = a.A ? a.S : a.X;   // each lane reads what it wrote
        const int64_t ld = a.A ? a.lds : a.ldx;
        float mu = group_all<Add, 4>(sum, sh[0]) / (float)a.C;
        auto squares = [&](float k) {   // of the values times k
            float s = 0.0f;
            for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
                float x[8];
                get8<XD>(src, t, ld, c, x);
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float d = fmaf(x[j], k, -mu);
                    s = fmaf(d, d, s);
                }
            }
            return group_all<Add, 4>(s, sh[1]);
        };
        float sq = squares(1.0f);
        const bool far = !(sq < kInf);   // (the same in all lanes)
        if (far) {
            sum = 0.0f;
            for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
                float x[8];
                get8<XD>(src, t, ld, c, x);
#pragma unroll
                for (int j = 0; j < 8; j++) sum = fmaf(x[j], kFar, sum);
            }
            mu = group_all<Add, 4>(sum, sh[0]) / (float)a.C;
            sq = squares(kFar);
        }
        const RowStats st(mu, sq, (float)a.C, a.eps, far);
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8], w[8], b[8];
            get8<XD>(src, t, ld, c, x);
            coef8(a.w, c, 1.0f, w);
            coef8(a.b, c, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; j++) x[j] = fmaf(st.of(x[j]), w[j], b[j]);
            put8<YD>(a.Y, t, a.ldy, c, x);
        }
        if (a.stats && threadIdx.x == 0) *(float2 *)(a.stats + 2 * t) = st.as_stored();
        __syncthreads();
    }
}

// The backward of rows in registers, as the forward's: S and dY are read once, for
// dX and for the sums of dw and db, which a lane keeps for its columns over all
// rows of its workgroup.
template <int SD, int DY, int DX, int CV, bool NARROW>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_bwd_rows_kernel(BwdArgs a) {
    __shared__ float2 sh[2][kMaxWaves];
    __shared__ float4 meet[kTogether * 128];   // [R][C / 4] where there are several rows
    const Lanes<NARROW> l(a.W, a.P);
    float w[CV][8], dw[CV][8] = {}, db[CV][8] = {};
#pragma unroll
    for (int v = 0; v < CV; v++)
        if (l.col(v) < a.C) coef8(a.w, l.col(v), 1.0f, w[v]);
    Raw8<SD> nx[CV];
    Raw8<DY> ny[CV];
    Raw8<DX> nd[CV];
    float2 ns{};
    auto fetch = [&](int64_t t) {
        if (t >= a.T) return;
        ns = *(const float2 *)(a.stats + 2 * t);
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (l.col(v) < a.C) {
                nx[v] = load8<SD>((const char *)a.S + (t * a.lds + l.col(v)) * esize<SD>());
                ny[v] = load8<DY>((const char *)a.dY + (t * a.lddy + l.col(v)) * esize<DY>());
                if (a.dS) nd[v] = load8<DX>((const char *)a.dS + (t * a.ldds + l.col(v)) * esize<DX>());
            }
    };
    const int64_t step = a.groups * l.R;
    if (CV == 1) fetch((int64_t)blockIdx.x * l.R + l.slot);
    int turn = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * l.R; t0 < a.T; t0 += step, turn ^= 1) {
        const int64_t t = t0 + l.slot;
        const bool here = t < a.T;
        if (CV > 1) fetch(t);
        float xh[CV][8], g[CV][8], s1 = 0.0f, s2 = 0.0f;
        const Hat hat(ns);
        Raw8<DX> d[CV];
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (here && l.col(v) < a.C) {
                unpack8<SD>(nx[v], xh[v]);
                unpack8<DY>(ny[v], g[v]);
                d[v] = nd[v];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    xh[v][j] = hat.of(xh[v][j]);
                    dw[v][j] = fmaf(g[v][j], xh[v][j], dw[v][j]);
                    db[v][j] += g[v][j];
                    g[v][j] *= w[v][j];
                    s1 += g[v][j];
                    s2 = fmaf(g[v][j], xh[v][j], s2);
                }
            }
        if (CV == 1) {
            fetch(t + step);
        } else {   // nothing is kept for a turn without a row: up to 34 registers (4096 x 16384 bf16 177 us, 136 without)
            ns = float2{};
#pragma unroll
            for (int v = 0; v < CV; v++) nx[v] = Raw8<SD>{}, ny[v] = Raw8<DY>{};
        }
        s1 = lanes_all<Add>(s1, l.P);
        s2 = lanes_all<Add>(s2, l.P);
        if (!NARROW && l.W > 1) {
            const float2 *of = &sh[turn][l.slot * l.W];
            if ((threadIdx.x & 63) == 0) sh[turn][l.slot * l.W + l.wave] = float2{s1, s2};
            __syncthreads();
            s1 = s2 = 0.0f;
            for (int i = 0; i < l.W; i++) s1 += of[i].x, s2 += of[i].y;
        }
        const float m1 = 0.5f * (s1 / (float)a.C), m2 = 0.5f * (s2 / (float)a.C);   // (halves, for 2 r)
#pragma unroll
        for (int v = 0; v < CV; v++)
            if (here && l.col(v) < a.C) {
                float o[8] = {};
                if (a.dS) unpack8<DX>(d[v], o);
#pragma unroll
                for (int j = 0; j < 8; j++)
                    o[j] = fmaf(hat.r, fmaf(-xh[v][j], m2, fmaf(g[v][j], 0.5f, -m1)), o[j]);
                store8<DX>((char *)a.dX + (t * a.lddx + l.col(v)) * esize<DX>(), pack8<DX>(o));
            }
    }
    if (!a.part) return;
    // the workgroup's sums: the R rows' in order
#pragma unroll
    for (int which = 0; which < 2; which++) {
        float *out = a.part + ((int64_t)blockIdx.x * 2 + which) * a.C;
        if (l.R == 1) {
#pragma unroll
            for (int v = 0; v < CV; v++)
                if (l.col(v) < a.C) store8<TERN_F32>(out + l.col(v), pack8<TERN_F32>(which ? db[v] : dw[v]));
        } else if (CV == 1) {
            const int n4 = a.C / 4;   // at most W * 128
            __syncthreads();
            if (l.col(0) < a.C)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float *f = which ? &db[0][4 * h] : &dw[0][4 * h];
                    meet[l.slot * n4 + l.tid * 2 + h] = float4{f[0], f[1], f[2], f[3]};
                }
            __syncthreads();
            for (int i = threadIdx.x; i < n4; i += blockDim.x) {
                float4 q = meet[i];
                for (int k = 1; k < l.R; k++) {
                    const float4 o = meet[k * n4 + i];
                    q.x += o.x, q.y += o.y, q.z += o.z, q.w += o.w;
                }
                *(float4 *)(out + i * 4) = q;
            }
        }
    }
}

template <int SD, int DY, int DX>
__global__ __launch_bounds__(256) void norm_dx_kernel(BwdArgs a) {
    __shared__ float sh[2][4];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float2 st = *(const float2 *)(a.stats + 2 * t);
        const Hat hat(st);
        float s1 = 0.0f, s2 = 0.0f;
        for (int c = threadIdx.x * 8; c < a.C; c += 2048) {
            float x[8], g[8], w[8];
            get8<SD>(a.S, t, a.lds, c, x);
            get8<DY>(a.dY, t, a.lddy, c, g);
            coef8(a.w, c, 1.0f, w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                s1 = fmaf(g[j], w[j], s1);
                s2 = fmaf(g[j] * w[j], hat.of(x[j]), s2);
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
                const float xh = hat.of(x[j]);
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
        for (int64_t t = g; t < a.T; t += a.groups) {
            const Hat hat(*(const float2 *)(a.stats + 2 * t));
            const float x = load1<SD>((const char *)a.S + (t * a.lds + c) * esize<SD>());
            const float d = load1<DY>((const char *)a.dY + (t * a.lddy + c) * esize<DY>());
            dw = fmaf(d, hat.of(x), dw);
            db += d;
        }
        a.part[(g * 2) * a.C + c] = dw;
        a.part[(g * 2 + 1) * a.C + c] = db;
    }
}

// The groups' sums: 32 columns a workgroup, of [2][C]; 32 strands of groups, each in
// order, then the strands.  (512 groups of 1032 columns: 3.0 us, with 8 strands 4.8;
// a number of strands chosen by the groups costs 0.4 us in every call.)
constexpr int kStrands = 32;
__global__ __launch_bounds__(32 * kStrands) void norm_dw_sum_kernel(const float *part, int groups, int C, float *dw,
                                                                    float *db) {
    __shared__ double sh[kStrands][32];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    double s = 0.0;
    if (c < 2 * C) {
#pragma unroll 8
        for (int g = y; g < groups; g += kStrands) s += part[(int64_t)g * 2 * C + c];
    }
    sh[y][x] = s;
    __syncthreads();
    if (y != 0 || c >= 2 * C) return;
#pragma unroll
    for (int i = 1; i < kStrands; i++) s += sh[i][x];
    float *out = c < C ? dw : db;
    if (out) out[c < C ? c : c - C] = (float)s;
}

}  // namespace ldev

namespace {

using ldev::BwdArgs;
using ldev::FwdArgs;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }
bool type_ok(int32_t dt) { return dt == TERN_F32 || dt == TERN_BF16; }
size_t esize(int32_t dt) { return dt == TERN_BF16 ? 2 : 4; }
int launched() { return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP; }

bool sizes_ok(int64_t T, int64_t C) { return T >= 0 && T <= kMaxT && C >= 0 && C <= kMaxInOut && C % 8 == 0; }
bool stride_ok(int64_t ld, int64_t C) { return ld >= C && ld % 8 == 0 && ld <= kMaxInOut * 8; }

// Waves of a row, eights of a lane and lanes of a wave; waves 0: rows too long for
// registers.
struct RowShape {
    int W, CV, P;
};
RowShape shape_of(int64_t C) {
    const int64_t most = ldev::kMaxWaves * 512;
    if (C <= 512) return {1, 1, C <= 64 ? 8 : C <= 128 ? 16 : C <= 256 ? 32 : 64};
    if (C <= most) return {(int)cdiv(C, 512), 1, 64};
    if (C <= 2 * most) return {(int)cdiv(C, 1024), 2, 64};
    return {0, 0, 64};
}
// rows of a workgroup of about `waves` waves
int rows_at_once(const RowShape &s, int waves) { return std::max(1, waves / std::max(s.W, 1)) * (64 / s.P); }

// Row groups of the backward, a workgroup each: at most 512, which fill the chip.
// With few long rows the groups' sums are as large as the rows: a group that takes
// `turns` times its rows costs about 2 us a turn and saves 16 C bytes of sums, written and
// read, so that their total is least at turns^2 = 16 C T / (R 4.9 TB/s 2 us).  (bf16, 300
// rows of 16384: 29 us with a group each, 23 with this; 1000 rows 44 and 36.  4096 rows are taken by 410
// groups, of which a unit holds one: 136 us, and 131 with 512.)
int64_t groups_of(int64_t T, int64_t C) {
    const int64_t R = rows_at_once(shape_of(C), ldev::kTogether);
    const int64_t turns = std::max<int64_t>(1, (int64_t)std::sqrt(1.6e-6 * (double)T * (double)C / (double)R));
    return std::max<int64_t>(1, std::min<int64_t>(512, cdiv(T, R * turns)));
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
    return (size_t)groups_of(T, C) * (size_t)C * 8;
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
    const RowShape shape = shape_of(C);
    FwdArgs a{X, A, w, b, S, Y, stats, ldx, lda, lds, ldy, T, (int)C, shape.W, shape.P, a_dtype, eps};
    hipStream_t st = (hipStream_t)stream;
    with_type(x_dtype, [&](auto xd) {
        with_type(y_dtype, [&](auto yd) {
            constexpr int XD = decltype(xd)::value, YD = decltype(yd)::value;
            if (shape.W == 0) {
                hipLaunchKernelGGL((ldev::norm_fwd_kernel<XD, YD>), dim3((unsigned)std::min<int64_t>(T, 65536)),
                                   dim3(256), 0, st, a);
                return;
            }
            const int R = rows_at_once(shape, 4);
            const dim3 g((unsigned)std::min<int64_t>(cdiv(T, R), 2048)), bl(shape.P * shape.W * R);
            if (shape.P < 64) hipLaunchKernelGGL((ldev::norm_fwd_rows_kernel<XD, YD, 1, true>), g, bl, 0, st, a);
            else if (shape.CV == 1) hipLaunchKernelGGL((ldev::norm_fwd_rows_kernel<XD, YD, 1, false>), g, bl, 0, st, a);
            else hipLaunchKernelGGL((ldev::norm_fwd_rows_kernel<XD, YD, 2, false>), g, bl, 0, st, a);
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
    const int64_t groups = groups_of(T, C);
    const size_t wsb = weights ? (size_t)groups * (size_t)C * 8 : 0;
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
    const RowShape shape = shape_of(C);
    BwdArgs a{S, dY, dS, stats, w, dX, dw, db, weights ? (float *)workspace : nullptr, lds, lddy, ldds, lddx, T, groups,
              (int)C, shape.W, shape.P};
    hipStream_t st = (hipStream_t)stream;
    const unsigned cols = (unsigned)cdiv(C, 64);
    if (T > 0) {
        with_type(s_dtype, [&](auto sd) {
            with_type(dy_dtype, [&](auto yd) {
                constexpr int SD = decltype(sd)::value, DY = decltype(yd)::value;
                with_type(dx_dtype, [&](auto xd) {
                    constexpr int DX = decltype(xd)::value;
                    if constexpr (DX == TERN_F32 || SD == TERN_BF16) {
                        if (shape.W == 0) {
                            hipLaunchKernelGGL((ldev::norm_dx_kernel<SD, DY, DX>),
                                               dim3((unsigned)std::min<int64_t>(T, 65536)), dim3(256), 0, st, a);
                            return;
                        }
                        const dim3 g((unsigned)groups), bl(shape.P * shape.W * rows_at_once(shape, ldev::kTogether));
                        if (shape.P < 64)
                            hipLaunchKernelGGL((ldev::norm_bwd_rows_kernel<SD, DY, DX, 1, true>), g, bl, 0, st, a);
                        else if (shape.CV == 1)
                            hipLaunchKernelGGL((ldev::norm_bwd_rows_kernel<SD, DY, DX, 1, false>), g, bl, 0, st, a);
                        else hipLaunchKernelGGL((ldev::norm_bwd_rows_kernel<SD, DY, DX, 2, false>), g, bl, 0, st, a);
                    }
                });
                if (weights && shape.W == 0)
                    hipLaunchKernelGGL((ldev::norm_dw_kernel<SD, DY>), dim3(cols, (unsigned)groups), dim3(64), 0, st, a);
            });
        });
    }
    if (weights)
        hipLaunchKernelGGL(ldev::norm_dw_sum_kernel, dim3((unsigned)cdiv(2 * C, 32)),
                           dim3(32 * ldev::kStrands), 0, st, a.part,
                           T > 0 ? (int)groups : 0, a.C, dw, db);
    return launched();
}

}  // extern "C"
