// tern_ortho.hip -- a weight update orthogonalised by Newton-Schulz products
// (C ABI in include/tern.h).
//
// With X = G / (|G|_F + 1e-7), transposed first if it has more rows than
// columns (m <= n), each step is
//   A = X X^T,   B = b A + c A^2,   X <- a X + B X
// which moves every singular value x of X to a x + b x^3 + c x^5 and leaves
// the singular vectors alone: after a few steps all are near 1.
//
// The products run on the fp16 matrix cores with fp32 sums.  fp16 and not
// bf16: X, A and B have known ranges (the polynomial keeps every singular
// value, and so every element of X, below 1.2025; |A| <= 1.45, |B| <= 2.9), so
// scaled by powers of two they fit fp16, whose three more bits make the
// result's error that of its own rounding to bf16 (measured on gradients of
// full rank: 0.0020 rms against the 0.0017 of the rounding alone; with bf16
// operands 0.010).
//   X is held as 2^14 X, A as 2^14 A, B as 2^13 B.
// A and A^2 are symmetric: only the tiles on and above the diagonal are
// computed, and each is written twice.  Every product is of the form P Q^T
// with both operands contiguous along the sum: X is kept beside its transpose
// (two of those, since a step reads one while it writes the other).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tern.h"
#include "tern_plan.h"

namespace tern {
namespace ndev {

typedef _Float16 h16;
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 b16x4 __attribute__((ext_vector_type(4)));
#define LDS_AS __attribute__((address_space(3)))

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kEps = 1e-7f;
constexpr float kXScale = 16384.0f;
constexpr int kPad = 64;        // rows and columns of the working matrices: multiples of this, zeros
constexpr int kParts = 256;     // partial sums of |G|^2
constexpr int kChunk = 32;      // K of a stage: 64 bytes a row
constexpr int kStages = 4;

struct OrthoOne {
    const void *G;
    void *O;
    h16 *X, *XT[2], *A, *B;   // [mp][np], [np][mp] twice, [mp][mp] twice
    double *part;             // [kParts]
    int64_t rows, cols;       // of G and O
    int m, n, mp, np;         // of X: m <= n; padded
    float gain;
    int tall;                 // X = G^T
    int start;                // first workgroup of the launch
};
struct OrthoArgs {
    OrthoOne p[kMaxGroup];
    int n;
    int g_bf16;
    int flip;                 // XT[flip] is current
    int last;                 // the last step writes O
};

__device__ inline int problem_of(const OrthoArgs &a, int wg) {
    int pi = 0;
    while (pi + 1 < a.n && wg >= a.p[pi + 1].start) pi++;
    return pi;
}

__device__ inline float g_at(const void *G, int bf, int64_t i) {
    return bf ? (float)((const __bf16 *)G)[i] : ((const float *)G)[i];
}

// |G|^2 in f64, one partial a workgroup, in a fixed order
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoArgs a) {
    __shared__ double red[256];
    const OrthoOne &p = a.p[blockIdx.y];
    const int64_t n8 = p.rows * p.cols / 8;
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += kParts * 256) {
        float f[8];
        if (a.g_bf16) {
            const u32x4 v = ((const u32x4 *)p.G)[i];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                f[2 * j] = __builtin_bit_cast(float, v[j] << 16);
                f[2 * j + 1] = __builtin_bit_cast(float, v[j] & 0xFFFF0000u);
            }
        } else {
            const float4 v0 = ((const float4 *)p.G)[2 * i], v1 = ((const float4 *)p.G)[2 * i + 1];
            f[0] = v0.x; f[1] = v0.y; f[2] = v0.z; f[3] = v0.w;
            f[4] = v1.x; f[5] = v1.y; f[6] = v1.z; f[7] = v1.w;
        }
#pragma unroll
        for (int j = 0; j < 8; j++) s += (double)f[j] * (double)f[j];
    }
    red[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d; d >>= 1) {
        if ((int)threadIdx.x < d) red[threadIdx.x] += red[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) p.part[blockIdx.x] = red[0];
}

// X and its transpose from G, 64 x 64 tiles, zeros in the padding
__global__ __launch_bounds__(256) void ortho_load_kernel(OrthoArgs a) {
    __shared__ double red[256];
    __shared__ h16 tile[64][66];
    const OrthoOne &p = a.p[problem_of(a, blockIdx.x)];
    red[threadIdx.x] = p.part[threadIdx.x];
    __syncthreads();
    for (int d = 128; d; d >>= 1) {
        if ((int)threadIdx.x < d) red[threadIdx.x] += red[threadIdx.x + d];
        __syncthreads();
    }
    const float f = (float)(16384.0 / (sqrt(red[0]) + (double)kEps));
    const int t = blockIdx.x - p.start, tn = p.np / 64;
    // tile (gi, gj) of G
    const int xi = t / tn, xj = t % tn;
    const int64_t r0 = (int64_t)(p.tall ? xj : xi) * 64, c0 = (int64_t)(p.tall ? xi : xj) * 64;
    const int c = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int r = (threadIdx.x >> 6) * 16 + i;
        float v = 0.0f;
        if (r0 + r < p.rows && c0 + c < p.cols) v = g_at(p.G, a.g_bf16, (r0 + r) * p.cols + c0 + c) * f;
        tile[r][c] = (h16)v;
    }
    __syncthreads();
    // the tile as it lies and transposed, into X and X^T (or the other way round)
    h16 *same = p.tall ? p.XT[0] : p.X, *flip = p.tall ? p.X : p.XT[0];
    const int64_t lds = p.tall ? p.mp : p.np, ldf = p.tall ? p.np : p.mp;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int r = (threadIdx.x >> 6) * 16 + i;
        same[(r0 + r) * lds + c0 + c] = tile[r][c];
        flip[(c0 + r) * ldf + r0 + c] = tile[c][r];
    }
}

// ---------------------------------------------------------------------------
// P Q^T: a workgroup of 2 x 2 waves computes a (2 WT)^2 tile, each wave
// WT x WT in 32 x 32 blocks.  Stages of 32 K go to LDS by direct loads, three
// ahead; the fragments of a stage are read into registers one stage ahead, so
// the matrix cores run over the barrier (one a stage).  A row's four 16-byte
// pieces lie permuted by its index, (row / 2) % 4, so that eight consecutive
// rows' pieces fall in different banks.
// ---------------------------------------------------------------------------

enum { GRAM = 0, POLY = 1, APPLY = 2 };

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *p, int64_t bytes) {
    const int n = __builtin_amdgcn_readfirstlane((int)(bytes < 0 ? 0 : bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : bytes));
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, n, 0x00020000);
}

// 16 bytes a lane to LDS, at lds + 16 lane; reads outside the resource give zeros
__device__ inline void load_lds(__amdgpu_buffer_rsrc_t rs, char *lds, uint32_t voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_AS void *)lds, 16, voff, 0, 0, 0);
}

template <int N>
__device__ inline void wait_loads_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);   // vmcnt(N), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

__device__ inline f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h16x8, a), __builtin_bit_cast(h16x8, b), c, 0, 0,
                                                  0);
}

template <int WT>
struct Frags {
    u32x4 a[2][WT / 32], b[2][WT / 32];   // [K half]
};

template <int WT, int MODE>
__global__ __launch_bounds__(256) void ortho_gemm_kernel(OrthoArgs a) {
    constexpr int BT = 2 * WT, F = WT / 32;
    constexpr int kOperand = BT * 64, kStage = 2 * kOperand;
    constexpr int NL = kStage / 1024 / 4;   // direct loads a wave and stage
    __shared__ __attribute__((aligned(16))) char lds[kStages * kStage];
    const OrthoOne &p = a.p[problem_of(a, blockIdx.x)];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // the tile: rows ti of P, rows tj of Q
    int ti, tj, t = blockIdx.x - p.start;
    const int nt = (p.mp + BT - 1) / BT;
    if (MODE == APPLY) {
        const int ntn = (p.np + BT - 1) / BT;
        ti = t / ntn;
        tj = t % ntn;
    } else {
        ti = 0;
        while (t >= nt - ti) {
            t -= nt - ti;
            ti++;
        }
        tj = ti + t;
    }
    const h16 *P = MODE == GRAM ? p.X : MODE == POLY ? p.A : p.B;
    const h16 *Q = MODE == GRAM ? p.X : MODE == POLY ? p.A : p.XT[a.flip];
    const int K = MODE == GRAM ? p.np : p.mp;
    const int64_t ld = K;
    const int nk = K / kChunk;
    const int prow = ti * BT, qrow = tj * BT;
    const int pall = p.mp, qall = MODE == APPLY ? p.np : p.mp;
    const char *pb = (const char *)(P + (int64_t)prow * ld), *qb = (const char *)(Q + (int64_t)qrow * ld);
    const int64_t pbytes = (int64_t)(pall - prow) * ld * 2, qbytes = (int64_t)(qall - qrow) * ld * 2;

    // load i of a wave: 16 rows of 64 bytes; rows past the matrix read zeros
    uint32_t voff[NL / 2];
#pragma unroll
    for (int i = 0; i < NL / 2; i++) {
        const int row = (wave * (NL / 2) + i) * 16 + (lane >> 2);
        voff[i] = (uint32_t)(row * ld * 2 + (((lane & 3) ^ ((row >> 1) & 3)) * 16));
    }
    auto issue = [&](int s) {
        char *st = lds + (s & (kStages - 1)) * kStage;
        const int64_t k = (int64_t)s * kChunk * 2;
        const __amdgpu_buffer_rsrc_t rp = rsrc(pb + (s < nk ? k : 0), s < nk ? pbytes - k : 0);
        const __amdgpu_buffer_rsrc_t rq = rsrc(qb + (s < nk ? k : 0), s < nk ? qbytes - k : 0);
#pragma unroll
        for (int i = 0; i < NL / 2; i++)
            load_lds(rp, st + (wave * (NL / 2) + i) * 1024, voff[i]);
#pragma unroll
        for (int i = 0; i < NL / 2; i++)
            load_lds(rq, st + kOperand + (wave * (NL / 2) + i) * 1024, voff[i]);
    };
    const int lr = lane & 31, lh = lane >> 5;
    auto read = [&](Frags<WT> &f, int s) {
        const char *st = lds + (s & (kStages - 1)) * kStage;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int piece = ((h * 2 + lh) ^ ((lr >> 1) & 3)) * 16;
#pragma unroll
            for (int i = 0; i < F; i++) {
                f.a[h][i] = *(const u32x4 *)(st + (wm * WT + i * 32 + lr) * 64 + piece);
                f.b[h][i] = *(const u32x4 *)(st + kOperand + (wn * WT + i * 32 + lr) * 64 + piece);
            }
        }
    };
    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
        for (int j = 0; j < F; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

    Frags<WT> f0, f1;
    auto mma = [&](const Frags<WT> &f) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int i = 0; i < F; i++)
#pragma unroll
                for (int j = 0; j < F; j++)
                    acc[i][j] = mfma(f.a[h][i], f.b[h][j], acc[i][j]);
    };
    issue(0);
    issue(1);
    issue(2);
    wait_loads_barrier<2 * NL>();
    read(f0, 0);
    // nk is even (K is a multiple of 64)
    for (int s = 0; s < nk; s += 2) {
        wait_loads_barrier<NL>();
        issue(s + 3);
        read(f1, s + 1);
        mma(f0);
        wait_loads_barrier<NL>();
        issue(s + 4);
        read(f0, s + 2);
        mma(f1);
    }
    wait_loads_barrier<0>();   // nothing in flight into LDS past the kernel's end

    // Results: a lane holds columns (of Q) lr of each block and rows
    // 8 g + 4 lh + 0..3 (of P), g < 4.
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
        for (int j = 0; j < F; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int row = prow + wm * WT + i * 32 + g * 8 + lh * 4, col = qrow + wn * WT + j * 32 + lr;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; r++) v[r] = acc[i][j][g * 4 + r];
                if (row >= p.mp || col >= qall) continue;
                if (MODE == APPLY) {
                    const int64_t at = (int64_t)col * p.mp + row;
                    const h16x4 x = *(const h16x4 *)(p.XT[a.flip] + at);
#pragma unroll
                    for (int r = 0; r < 4; r++) v[r] = fmaf(kA, (float)x[r], v[r] * (1.0f / 8192.0f));
                    if (!a.last) {
                        h16x4 o;
#pragma unroll
                        for (int r = 0; r < 4; r++) o[r] = (h16)v[r];
                        *(h16x4 *)(p.XT[a.flip ^ 1] + at) = o;
#pragma unroll
                        for (int r = 0; r < 4; r++) p.X[(int64_t)(row + r) * p.np + col] = o[r];
                    } else if (col < p.n && row < p.m) {
                        // row is a multiple of 4 and m of 8: all four rows exist
                        b16x4 o;
#pragma unroll
                        for (int r = 0; r < 4; r++) o[r] = (__bf16)(v[r] * (1.0f / kXScale) * p.gain);
                        if (p.tall) {
                            *(b16x4 *)((__bf16 *)p.O + (int64_t)col * p.cols + row) = o;
                        } else {
#pragma unroll
                            for (int r = 0; r < 4; r++) ((__bf16 *)p.O)[(int64_t)(row + r) * p.cols + col] = o[r];
                        }
                    }
                } else {
                    h16x4 o;
                    const int64_t at = (int64_t)col * p.mp + row;   // the mirrored place
                    if (MODE == POLY) {
                        const h16x4 x = *(const h16x4 *)(p.A + at);   // A is symmetric
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            o[r] = (h16)fmaf(0.5f * kB, (float)x[r], v[r] * (kC / 32768.0f));
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; r++) o[r] = (h16)(v[r] * (1.0f / 16384.0f));
                    }
                    h16 *out = MODE == POLY ? p.B : p.A;
                    *(h16x4 *)(out + at) = o;
                    if (ti != tj) {
#pragma unroll
                        for (int r = 0; r < 4; r++) out[(int64_t)(row + r) * p.mp + col] = o[r];
                    }
                }
            }
}

}  // namespace ndev

namespace {

using ndev::OrthoArgs;
using ndev::OrthoOne;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }
size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

struct OrthoLayout {
    int64_t m, n, mp, np;
    size_t x, xt0, xt1, a, b, part, total;   // byte offsets
};
OrthoLayout layout(int64_t rows, int64_t cols) {
    OrthoLayout L{};
    L.m = rows < cols ? rows : cols;
    L.n = rows < cols ? cols : rows;
    L.mp = cdiv(L.m, ndev::kPad) * ndev::kPad;
    L.np = cdiv(L.n, ndev::kPad) * ndev::kPad;
    const size_t mn = al256((size_t)L.mp * L.np * 2), mm = al256((size_t)L.mp * L.mp * 2);
    L.x = 0;
    L.xt0 = mn;
    L.xt1 = 2 * mn;
    L.a = 3 * mn;
    L.b = 3 * mn + mm;
    L.part = 3 * mn + 2 * mm;
    L.total = L.m ? L.part + al256(ndev::kParts * 8) : 0;
    return L;
}

bool sizes_ok(int64_t r, int64_t c) {
    // a launch counts its threads in 32 bits: 64 x 64 tiles of 256 threads
    return r >= 0 && c >= 0 && r <= kMaxInOut && c <= kMaxInOut && r % 8 == 0 && c % 8 == 0 &&
           cdiv(r, 64) * cdiv(c, 64) <= (1 << 20);
}

// tiles of a product with edge bt
int64_t tri_tiles(int64_t mp, int64_t bt) {
    const int64_t t = cdiv(mp, bt);
    return t * (t + 1) / 2;
}

template <int MODE>
void launch_product(int wt, int64_t wgs, const OrthoArgs &a, hipStream_t st) {
    const dim3 g((unsigned)wgs), b(256);
    if (wt == 128) hipLaunchKernelGGL((ndev::ortho_gemm_kernel<128, MODE>), g, b, 0, st, a);
    else if (wt == 64) hipLaunchKernelGGL((ndev::ortho_gemm_kernel<64, MODE>), g, b, 0, st, a);
    else hipLaunchKernelGGL((ndev::ortho_gemm_kernel<32, MODE>), g, b, 0, st, a);
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

size_t tern_layer_orthogonalize_workspace_bytes(const tern_ortho_t *mats, int32_t n) {
    if (n < 1 || n > kMaxGroup || !mats) return 0;
    size_t s = 0;
    for (int i = 0; i < n; i++) {
        if (!sizes_ok(mats[i].rows, mats[i].cols)) return 0;
        s += layout(mats[i].rows, mats[i].cols).total;
    }
    return s;
}

int tern_layer_orthogonalize(const tern_ortho_t *mats, int32_t n, int32_t g_dtype, int32_t steps, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (n < 1 || n > kMaxGroup) return TERN_ERR_SHAPE;
    if (!mats) return TERN_ERR_NULL;
    for (int i = 0; i < n; i++)
        if (!sizes_ok(mats[i].rows, mats[i].cols)) return TERN_ERR_SHAPE;
    if (g_dtype != TERN_F32 && g_dtype != TERN_BF16) return TERN_ERR_DTYPE;
    if (steps < 1 || steps > 64) return TERN_ERR_VALUE;
    const size_t need = tern_layer_orthogonalize_workspace_bytes(mats, n);
    for (int i = 0; i < n; i++) {
        const size_t c = (size_t)mats[i].rows * mats[i].cols;
        if (c && (!mats[i].G || !mats[i].O)) return TERN_ERR_NULL;
    }
    if (need && (!workspace || workspace_bytes < need)) return TERN_ERR_WORKSPACE;
    if (misaligned(workspace)) return TERN_ERR_ALIGN;
    const size_t es = g_dtype == TERN_BF16 ? 2 : 4;
    for (int i = 0; i < n; i++) {
        if (misaligned(mats[i].G) || misaligned(mats[i].O)) return TERN_ERR_ALIGN;
        const size_t c = (size_t)mats[i].rows * mats[i].cols;
        if (ranges_overlap(mats[i].O, c * 2, workspace, need)) return TERN_ERR_ALIAS;
        for (int j = 0; j < n; j++) {
            const size_t d = (size_t)mats[j].rows * mats[j].cols;
            if (ranges_overlap(mats[i].O, c * 2, mats[j].G, d * es)) return TERN_ERR_ALIAS;
            if (j != i && ranges_overlap(mats[i].O, c * 2, mats[j].O, d * 2)) return TERN_ERR_ALIAS;
        }
        if (ranges_overlap(mats[i].G, c * es, workspace, need)) return TERN_ERR_ALIAS;
    }
    OrthoArgs a{};
    a.g_bf16 = g_dtype == TERN_BF16;
    size_t at = 0;
    int64_t tiles = 0;
    for (int i = 0; i < n; i++) {
        if (mats[i].rows == 0 || mats[i].cols == 0) continue;
        const OrthoLayout L = layout(mats[i].rows, mats[i].cols);
        char *w = (char *)workspace + at;
        at += L.total;
        OrthoOne &p = a.p[a.n++];
        p.G = mats[i].G; p.O = mats[i].O;
        p.X = (ndev::h16 *)(w + L.x);
        p.XT[0] = (ndev::h16 *)(w + L.xt0);
        p.XT[1] = (ndev::h16 *)(w + L.xt1);
        p.A = (ndev::h16 *)(w + L.a);
        p.B = (ndev::h16 *)(w + L.b);
        p.part = (double *)(w + L.part);
        p.rows = mats[i].rows; p.cols = mats[i].cols;
        p.m = (int)L.m; p.n = (int)L.n; p.mp = (int)L.mp; p.np = (int)L.np;
        p.gain = mats[i].gain;
        p.tall = mats[i].rows > mats[i].cols;
    }
    if (a.n == 0) return TERN_OK;
    hipStream_t st = (hipStream_t)stream;
    hipLaunchKernelGGL(ndev::ortho_norm_kernel, dim3(ndev::kParts, (unsigned)a.n), dim3(256), 0, st, a);
    // the first workgroup of every problem in each kind of launch
    auto starts = [&](int kind, int bt) {
        int64_t s = 0;
        for (int i = 0; i < a.n; i++) {
            OrthoOne &p = a.p[i];
            p.start = (int)s;
            s += kind == ndev::APPLY ? cdiv(p.mp, bt) * cdiv(p.np, bt) : tri_tiles(p.mp, bt);
        }
        return s;
    };
    tiles = starts(ndev::APPLY, 64);
    hipLaunchKernelGGL(ndev::ortho_load_kernel, dim3((unsigned)tiles), dim3(256), 0, st, a);
    auto tile_for = [&](int kind) {
        for (int wt : {128, 64})
            if (starts(kind, 2 * wt) >= 192) return wt;
        return 32;
    };
    const int wt_tri = tile_for(ndev::GRAM), wt_app = tile_for(ndev::APPLY);
    for (int s = 0; s < steps; s++) {
        a.flip = s & 1;
        a.last = s == steps - 1;
        const int64_t tri = starts(ndev::GRAM, 2 * wt_tri);
        launch_product<ndev::GRAM>(wt_tri, tri, a, st);
        launch_product<ndev::POLY>(wt_tri, tri, a, st);
        const int64_t app = starts(ndev::APPLY, 2 * wt_app);
        launch_product<ndev::APPLY>(wt_app, app, a, st);
    }
    return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP;
}

size_t tern_orthogonalize_workspace_bytes(int64_t rows, int64_t cols) {
    const tern_ortho_t m = {rows, cols, nullptr, nullptr, 1.0f};
    return tern_layer_orthogonalize_workspace_bytes(&m, 1);
}

int tern_orthogonalize(const void *G, int32_t g_dtype, int64_t rows, int64_t cols, int32_t steps, float gain, void *O,
                       void *workspace, size_t workspace_bytes, void *stream) {
    const tern_ortho_t m = {rows, cols, G, O, gain};
    return tern_layer_orthogonalize(&m, 1, g_dtype, steps, workspace, workspace_bytes, stream);
}

}  // extern "C"
