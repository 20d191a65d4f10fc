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
// scaled by powers of two they fit fp16, whose three more bits count (bf16
// operands: an error of 0.010 where fp16 ones leave 0.0012).
//   X is held as 2^14 X, A as 2^14 A, B as 2^13 B.
//
// What is rounded, and what is not.  A rounding of X itself would be noise in
// every direction, and a direction in which G has next to nothing grows 3.44
// times a step: over five steps such noise reaches 0.02 of O for a G of rank 64
// of 512, and 0.15 for rank one.  So X = H + L is held in two terms of fp16, 22
// bits, and a X takes both; the products take H, whose rounding they pass on only
// to the directions in which B is large, where X has stopped growing.  There
// B L, the part left out, is most of the error.  Its largest part, that of B's
// diagonal, is put back in the last two steps (before them it would take from
// the weak directions what it gives to the strong ones), and so is in every step
// what the rounding of B's diagonal loses.  With d = diag(B) in fp32, e = d less
// its fp16 value:
//   X <- (a + e) H + (a + d or a) L + B H
// leaves, before O's rounding, 0.0007 of O for a flat spectrum, 0.0002 to 0.0009
// for decaying and low-rank ones (emulated, 512 x 1024); O's rounding to bf16 is
// 0.0017.
// A and A^2 are symmetric: only the tiles on and above the diagonal are
// computed, and each is written twice.  Every product is of the form P Q^T
// with both operands contiguous along the sum: X is kept beside its transpose
// (two of those, since a step reads one while it writes the other).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/tern.h"
#include "tern_plan.h"

namespace tern {
namespace ndev {

typedef _Float16 h16;
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
#define LDS_AS __attribute__((address_space(3)))

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kEps = 1e-7f;
constexpr float kXScale = 16384.0f;
constexpr int kPad = 64;        // rows and columns of the working matrices: multiples of this, zeros
constexpr int kParts = 256;     // partial sums of |G|^2
constexpr float kLow = 2048.0f; // of X's low term, which is half a step of the high one at most

struct OrthoOne {
    const void *G;
    void *O;
    h16 *X, *XT[2], *A, *B;   // [mp][np], [np][mp] twice, [mp][mp] twice
    h16 *XL;                  // X's low term, 2^25 L, in the order of low_block()
    float2 *diag;             // [mp]: a + e, a + d (or a)
    double *part;             // [kParts]
    int64_t rows, cols;       // of G and O
    int m, n, mp, np;         // of X: m <= n; padded
    float gain;
    int tall;                 // X = G^T
    int start, tiles;         // first workgroup of the launch; workgroups
};
struct OrthoArgs {
    OrthoOne p[kMaxGroup];
    int n;
    int g_bf16;
    int flip;                 // XT[flip] is current
    int last;                 // the last step writes O
    int near;                 // one of the last two steps
};

// X's low term is read and written where X is computed, by the lane that holds the
// element among the sums of a 32 x 32 block: it lies in that order, whatever the
// tiles.  Blocks by rows, 1024 elements each: two pieces (g = 0, 1 and 2, 3) of 8 a
// lane, element 4 (g & 1) + r of lane l being X's row 8 g + 4 (l / 32) + r and
// column l % 32 of the block.
__device__ inline h16 *low_block(const OrthoOne &p, int row, int col) {
    return p.XL + ((int64_t)(row / 32) * (p.np / 32) + col / 32) * 1024 + (threadIdx.x & 63) * 8;
}

// A value whose fp16 rounding and remainder are both taken.  Left to itself the
// compiler rounds twice, once within the operation that made the value and once
// from its fp32 result, and where these fall on either side of a tie the two
// terms do not belong together.
__device__ inline float once(float x) {
    asm("" : "+v"(x));
    return x;
}

__device__ inline int problem_of(const OrthoArgs &a, int wg) {
    int pi = 0;
    while (pi + 1 < a.n && wg >= a.p[pi + 1].start) pi++;
    return pi;
}

__device__ inline void load4(const void *G, int bf, int64_t i, float *f) {
    if (bf) {
        const uint2 v = *(const uint2 *)((const uint16_t *)G + i);
        f[0] = __builtin_bit_cast(float, v.x << 16);
        f[1] = __builtin_bit_cast(float, v.x & 0xFFFF0000u);
        f[2] = __builtin_bit_cast(float, v.y << 16);
        f[3] = __builtin_bit_cast(float, v.y & 0xFFFF0000u);
    } else {
        const float4 v = *(const float4 *)((const float *)G + i);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
}

// |G|^2 in f64, one partial a workgroup, in a fixed order
__global__ __launch_bounds__(256) void ortho_norm_kernel(OrthoArgs a) {
    __shared__ double red[4];
    const OrthoOne &p = a.p[blockIdx.y];
    const int64_t n8 = p.rows * p.cols / 8;
    double s = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += kParts * 256) {
        float f[8];
        load4(p.G, a.g_bf16, 8 * i, f);
        load4(p.G, a.g_bf16, 8 * i + 4, f + 4);
#pragma unroll
        for (int j = 0; j < 8; j++) s += (double)f[j] * (double)f[j];
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) p.part[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X, its transpose and its low term from G, 64 x 64 tiles, zeros in the padding
__global__ __launch_bounds__(256) void ortho_load_kernel(OrthoArgs a) {
    __shared__ h16 tile[64][68], low[64][68];
    const OrthoOne &p = a.p[problem_of(a, blockIdx.x)];
    // every wave adds up the partials (in the same order)
    const int lane = threadIdx.x & 63;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kParts / 64; i++) sum += p.part[lane + 64 * i];
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
    const float f = (float)(16384.0 / (sqrt(sum) + (double)kEps));
    const int t = blockIdx.x - p.start, tn = p.np / 64;
    // tile (xi, xj) of X, at (r0, c0) of G
    const int xi = t / tn, xj = t % tn;
    const int64_t r0 = (int64_t)(p.tall ? xj : xi) * 64, c0 = (int64_t)(p.tall ? xi : xj) * 64;
    // G's sides are multiples of 8: four columns are inside or outside together
    const int c4 = (threadIdx.x & 15) * 4;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = (threadIdx.x >> 4) + 16 * i;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (r0 + r < p.rows && c0 + c4 < p.cols) load4(p.G, a.g_bf16, (r0 + r) * p.cols + c0 + c4, v);
        h16x4 o, l;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float x = once(v[j] * f);
            o[j] = (h16)x;
            l[j] = (h16)((x - (float)o[j]) * kLow);
        }
        *(h16x4 *)&tile[r][c4] = o;
        *(h16x4 *)&low[r][c4] = l;
    }
    __syncthreads();
    // the tile as it lies and transposed, into X and X^T (or the other way round)
    h16 *same = p.tall ? p.XT[0] : p.X, *flip = p.tall ? p.X : p.XT[0];
    const int64_t lds = p.tall ? p.mp : p.np, ldf = p.tall ? p.np : p.mp;
    const int c8 = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int r = (threadIdx.x >> 3) + 32 * i;
        const h16x4 lo = *(const h16x4 *)&tile[r][c8], hi = *(const h16x4 *)&tile[r][c8 + 4];
        h16x8 s, q;
#pragma unroll
        for (int j = 0; j < 4; j++) s[j] = lo[j], s[4 + j] = hi[j];
#pragma unroll
        for (int j = 0; j < 8; j++) q[j] = tile[c8 + j][r];
        *(h16x8 *)(same + (r0 + r) * lds + c0 + c8) = s;
        *(h16x8 *)(flip + (c0 + r) * ldf + r0 + c8) = q;
    }
    // a block of the low term a wave
    const int w = threadIdx.x >> 6, br = (w >> 1) * 32, bc = (w & 1) * 32, xc = bc + (lane & 31);
    h16 *out = low_block(p, xi * 64 + br, xj * 64 + bc);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        h16x8 v;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int xr = br + 16 * h + 8 * (j >> 2) + 4 * (lane >> 5) + (j & 3);
            v[j] = p.tall ? low[xc][xr] : low[xr][xc];
        }
        *(h16x8 *)(out + 512 * h) = v;
    }
}

// ---------------------------------------------------------------------------
// P Q^T: a workgroup of 2 x 2 waves computes a (2 WT)^2 tile, each wave
// WT x WT in 32 x 32 blocks.  Stages of KC K go to LDS by direct loads, ST - 1
// ahead; the fragments of a stage are read into registers one stage ahead, so
// the matrix cores run over the barrier (one a stage).
//
// What bounds it.  4096 x 16384: A 290 us, its polynomial 84, B X 577, five steps
// 4.9 ms.  B X runs at 0.95 PFLOP/s (the vendor's plain product of that size 1.2):
// the board is at its power cap (with zeros in all operands it takes 485 us), and
// between the tiles the matrix cores wait for about 15 us while 256 KiB of the old X are read and 384 KiB of the new one written
// (128 KiB each are the low term's, which costs 40 us of the 577).  Small matrices
// (six of 512 x 512 to 512 x 2048, 169 us) are fifteen products of 5 to 15 us each, of
// which the launch, the first loads and the results are 4 to 5.
// ---------------------------------------------------------------------------

enum { GRAM = 0, POLY = 1, APPLY = 2 };

__device__ inline __amdgpu_buffer_rsrc_t rsrc(const void *p, int64_t bytes) {
    const int n = __builtin_amdgcn_readfirstlane((int)(bytes < 0 ? 0 : bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : bytes));
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, n, 0x00020000);
}

// 16 bytes a lane to LDS, at lds + 16 lane; reads outside the resource give zeros
__device__ inline void load_lds(__amdgpu_buffer_rsrc_t rs, char *lds, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LDS_AS void *)lds, 16, voff, soff, 0, 0);
}

__device__ inline u32x4 load16(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0);
}
__device__ inline void store16(u32x4 v, __amdgpu_buffer_rsrc_t rs, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, off, 0, 0);
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

// 4 x 4 transpose of 16-bit values among the 16 lanes of a group while reading
__device__ inline u32x2 transposed(const char *at) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS v4i16 *)at));
}

template <int WT, int KC>
struct Frags {
    u32x4 a[KC / 16][WT / 32], b[KC / 16][WT / 32];
};

template <int WT, int KC, int ST, int MODE>
__global__ __launch_bounds__(256) void ortho_gemm_kernel(OrthoArgs a) {
    constexpr int BT = 2 * WT, F = WT / 32, H = KC / 16;
    constexpr int kRow = KC * 2, kPieces = KC / 8;
    constexpr int kOperand = BT * kRow, kStage = 2 * kOperand;
    constexpr int NL = kStage / 1024 / 4;   // direct loads a wave and stage
    constexpr int kOut = 4 * WT * (WT * 2 + 16);
    __shared__ __attribute__((aligned(16))) char lds[ST * kStage > kOut ? ST * kStage : kOut];
    using Fr = Frags<WT, KC>;
    // the place of a row's 16-byte piece: equal pieces of 16 consecutive rows
    // fall in the 16 places of a 256-byte window of banks
    auto swz = [](int row, int piece) { return piece ^ (row / (256 / kRow) % kPieces); };
    const OrthoOne &p = a.p[problem_of(a, blockIdx.x)];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;

    // the tile: rows ti of P, rows tj of Q
    // (workgroups go round the 8 XCDs: each XCD takes one run of a problem's
    // tiles, whose operands then meet in its L2)
    const int wg = blockIdx.x - p.start, per = p.tiles >> 3, more = p.tiles & 7, run = wg & 7;
    int ti, tj, t = (wg >> 3) + run * per + (run < more ? run : more);
    const int nt = (p.mp + BT - 1) / BT;
    if (MODE == APPLY) {
        // down panels of 8 rows of tiles
        const int ntn = (p.np + BT - 1) / BT;
        const int g = t / (8 * ntn), h = nt - 8 * g < 8 ? nt - 8 * g : 8;
        t -= 8 * g * ntn;
        ti = 8 * g + t % h;
        tj = t / h;
    } else {
        // the triangle tj >= ti, down panels of 4 rows of tiles
        int r = 0;
        while (true) {
            const int h = nt - r < 4 ? nt - r : 4, n = h * (nt - r) - h * (h - 1) / 2;
            if (t < n) break;
            t -= n;
            r += 4;
        }
        tj = r;
        for (int h = 1; t >= h; tj++, h += h < 4 && h < nt - r) t -= h;
        ti = r + t;
    }
    const h16 *P = MODE == GRAM ? p.X : MODE == POLY ? p.A : p.B;
    const h16 *Q = MODE == GRAM ? p.X : MODE == POLY ? p.A : p.XT[a.flip];
    const int K = MODE == GRAM ? p.np : p.mp;
    const int64_t ld = K;
    const int nk = K / KC;
    const int prow = ti * BT, qrow = tj * BT;
    const int pall = p.mp, qall = MODE == APPLY ? p.np : p.mp;
    const char *pb = (const char *)(P + (int64_t)prow * ld), *qb = (const char *)(Q + (int64_t)qrow * ld);
    const int64_t pbytes = (int64_t)(pall - prow) * ld * 2, qbytes = (int64_t)(qall - qrow) * ld * 2;

    // load i of a wave: 1 KiB, whole rows; rows past the matrix read zeros
    uint32_t voff[NL / 2];
#pragma unroll
    for (int i = 0; i < NL / 2; i++) {
        const int row = (wave * (NL / 2) + i) * (64 / kPieces) + lane / kPieces;
        voff[i] = (uint32_t)(row * ld * 2 + swz(row, lane % kPieces) * 16);
    }
    const __amdgpu_buffer_rsrc_t rp = rsrc(pb, pbytes), rq = rsrc(qb, qbytes);
    // load i of stage s into its place (a stage past the last one loads that
    // again, unread)
    auto issue = [&](int s, int place, int i) {
        char *st = lds + place + (wave * (NL / 2) + i % (NL / 2)) * 1024;
        const uint32_t k = (uint32_t)(s < nk ? s : nk - 1) * kRow;
        if (i < NL / 2) load_lds(rp, st, voff[i % (NL / 2)], k);
        else load_lds(rq, st + kOperand, voff[i % (NL / 2)], k);
    };
    const int lr = lane & 31, lh = lane >> 5;
    const int aoff = (wm * WT + lr) * kRow, boff = kOperand + (wn * WT + lr) * kRow;
    int piece[H];
#pragma unroll
    for (int h = 0; h < H; h++) piece[h] = swz(lr, h * 2 + lh) * 16;   // rows 32 apart share their permutation
    // read i of a stage's fragments: those of K 16 h first, P's before Q's
    auto read = [&](Fr &f, const char *st, int i) {
        const int h = i / (2 * F), j = i % F;
        if (i % (2 * F) < F) f.a[h][j] = *(const u32x4 *)(st + aoff + j * 32 * kRow + piece[h]);
        else f.b[h][j] = *(const u32x4 *)(st + boff + j * 32 * kRow + piece[h]);
    };
    f32x16 acc[F][F];
#pragma unroll
    for (int i = 0; i < F; i++)
#pragma unroll
        for (int j = 0; j < F; j++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[i][j][r] = 0.0f;

    Fr f0, f1;
    constexpr int nm = H * F * F, nr = 2 * H * F;
    auto product = [&](const Fr &f, int k) {
        const int h = k / (F * F), i = k / F % F, j = k % F;
        acc[i][j] = mfma(f.a[h][i], f.b[h][j], acc[i][j]);
    };
    // The products of stage s, already in registers, with the reads of the
    // next stage and the loads of the one ST - 1 ahead dealt out between them
    // (in a burst they fill the address units' queue and the matrix cores wait
    // behind it).  The reads are over after three quarters of the products.
    int here = kStage, there = (ST - 1) * kStage;   // places of stages s + 1 and s + ST - 1
    auto step = [&](const Fr &f, Fr &next, int s) {
        wait_loads_barrier<(ST - 3) * NL>();
        const char *st = lds + here;
#pragma unroll
        for (int k = 0; k < nm; k++) {
            product(f, k);
            constexpr int span = nm * 3 / 4;
#pragma unroll
            for (int i = k * nr / span; i < (k + 1) * nr / span && i < nr; i++) read(next, st, i);
#pragma unroll
            for (int i = k * NL / nm; i < (k + 1) * NL / nm; i++) issue(s + ST - 1, there, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        here = here == (ST - 1) * kStage ? 0 : here + kStage;
        there = there == (ST - 1) * kStage ? 0 : there + kStage;
    };
#pragma unroll
    for (int s = 0; s < ST - 1; s++)
#pragma unroll
        for (int i = 0; i < NL; i++) issue(s, s * kStage, i);
    wait_loads_barrier<(ST - 2) * NL>();
#pragma unroll
    for (int i = 0; i < nr; i++) read(f0, lds, i);
    for (int s = 0; s + 1 < nk; s += 2) {
        step(f0, f1, s);
        step(f1, f0, s + 1);
    }
    if (nk & 1)
#pragma unroll
        for (int k = 0; k < nm; k++) product(f0, k);
    wait_loads_barrier<0>();   // every load has landed and every read is done

    // Results.  A lane holds columns (of Q) lr of each block and rows
    // 8 g + 4 lh + 0..3 (of P), g < 4.  Each wave brings its part through its own
    // piece of shared memory, T[column][row], from where both orders leave in
    // 16-byte pieces: T's rows as they lie, and transposed by the transposing
    // reads.  (Stored from the registers, 8 and 2 bytes a lane, a 256 x 256 tile
    // took 20 us.)
    constexpr int kT = WT * 2 + 16;   // bytes of a column of T
    char *T = lds + wave * WT * kT;
    const int row0 = prow + wm * WT, col0 = qrow + wn * WT;
    // A piece outside the matrix is loaded as zeros and not stored: its offset
    // lies behind the resource's end (columns past the last do by themselves).
    constexpr uint32_t kNone = 0x7FFFFFF0u;
    constexpr int kAll = WT * WT / 8 / 64;                             // pieces a lane
    constexpr int NB = kAll % 8 == 0 ? 8 : kAll % 6 == 0 ? 6 : kAll;   // and how many at a time
    // The low term and the diagonal's factors, of row of blocks i: on the way while
    // the old matrix is read, all of a small tile's, of a large one's the first and then
    // the next row's (read in turn, 4096 x 16384 takes 596 us a product, not 577).
    h16x8 low[F][F][2];
    float2 d[F][16];   // of rows 8 g + 4 lh + r, at 4 g + r
    const __amdgpu_buffer_rsrc_t rdiag = rsrc(p.diag, (int64_t)p.mp * 8);
    auto load_low = [&](int i) {
        const int row = row0 + i * 32;
#pragma unroll
        for (int j = 0; j < F; j++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                low[i][j][h] = h16x8{};
                if (row < p.mp && col0 + j * 32 < p.np)
                    low[i][j][h] = *(const h16x8 *)(low_block(p, row, col0 + j * 32) + 512 * h);
            }
#pragma unroll
        for (int g = 0; g < 4; g++)
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                const u32x4 v = load16(rdiag, (uint32_t)(row + 8 * g + 4 * lh + r) * 8);
                d[i][4 * g + r] = __builtin_bit_cast(float2, u32x2{v[0], v[1]});
                d[i][4 * g + r + 1] = __builtin_bit_cast(float2, u32x2{v[2], v[3]});
            }
    };
    if (MODE == APPLY)
#pragma unroll
        for (int i = 0; i < (F > 2 ? 1 : F); i++) load_low(i);
    if (MODE != GRAM) {
        // the old matrix's term at [column][row] (A is symmetric)
        const h16 *old = (MODE == APPLY ? p.XT[a.flip] : p.A) + (int64_t)col0 * p.mp;
        const __amdgpu_buffer_rsrc_t ro = rsrc(old, (int64_t)(qall - col0) * p.mp * 2);
#pragma unroll 1
        for (int n = 0; n < kAll; n += NB) {
            u32x4 v[NB];
#pragma unroll
            for (int m = 0; m < NB; m++) {
                const int i = lane + (n + m) * 64, c = i / (WT / 8), r = row0 + i % (WT / 8) * 8;
                v[m] = load16(ro, r < p.mp ? (uint32_t)(c * p.mp + r) * 2 : kNone);
            }
#pragma unroll
            for (int m = 0; m < NB; m++) {
                const int i = lane + (n + m) * 64;
                *(u32x4 *)(T + i / (WT / 8) * kT + i % (WT / 8) * 16) = v[m];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < F; i++) {
        char *at = T + lr * kT + (i * 32 + lh * 4) * 2;
        const int row = row0 + i * 32;
        if (MODE == APPLY && F > 2 && i + 1 < F) load_low(i + 1);
        h16x4 x[F][4];
        if (MODE != GRAM)
#pragma unroll
            for (int j = 0; j < F; j++)
#pragma unroll
                for (int g = 0; g < 4; g++) x[j][g] = *(const h16x4 *)(at + j * 32 * kT + g * 16);
#pragma unroll
        for (int j = 0; j < F; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                h16x4 o;
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const float v = acc[i][j][g * 4 + r];
                    if (MODE == GRAM) o[r] = (h16)(v * (1.0f / 16384.0f));
                    else if (MODE == POLY) {
                        const float b = once(fmaf(0.5f * kB, (float)x[j][g][r], v * (kC / 32768.0f)));   // 2^13 B
                        o[r] = (h16)b;
                        const int k = 8 * g + 4 * lh + r;
                        if (ti == tj && wm == wn && i == j && k == lr && row + k < p.mp)
                            p.diag[row + k] = float2{kA + (b - (float)o[r]) * (1.0f / 8192.0f),
                                                     a.near ? kA + b * (1.0f / 8192.0f) : kA};
                    } else {
                        const int e = 4 * (g & 1) + r;
                        const float2 c = d[i][4 * g + r];
                        const float y = once(fmaf(
                            c.x, (float)x[j][g][r],
                            fmaf(c.y * (1.0f / kLow), (float)low[i][j][g >> 1][e], v * (1.0f / 8192.0f))));
                        if (a.last) {
                            o[r] = __builtin_bit_cast(h16, (__bf16)(y * (1.0f / kXScale) * p.gain));
                        } else {
                            o[r] = (h16)y;
                            low[i][j][g >> 1][e] = (h16)((y - (float)o[r]) * kLow);
                        }
                    }
                }
                *(h16x4 *)(at + j * 32 * kT + g * 16) = o;
            }
        if (MODE == APPLY && !a.last)
#pragma unroll
            for (int j = 0; j < F; j++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    if (row < p.mp && col0 + j * 32 < p.np)
                        *(h16x8 *)(low_block(p, row, col0 + j * 32) + 512 * h) = low[i][j][h];
    }
    const bool out = MODE == APPLY && a.last;   // into O, without the padding
    const int rows = out ? p.m : p.mp, cols = out ? p.n : qall;
    // [column][row]: X^T, the mirrored tile of A or B, or O of a tall G
    if (!out || p.tall) {
        const int64_t ldd = out ? p.cols : p.mp;
        h16 *dst = (MODE == GRAM ? p.A : MODE == POLY ? p.B : out ? (h16 *)p.O : p.XT[a.flip ^ 1]) + col0 * ldd;
        const __amdgpu_buffer_rsrc_t rd = rsrc(dst, (cols - col0) * ldd * 2);
#pragma unroll 1
        for (int n = 0; n < kAll; n += NB) {
            u32x4 v[NB];
#pragma unroll
            for (int m = 0; m < NB; m++) {
                const int i = lane + (n + m) * 64;
                v[m] = *(const u32x4 *)(T + i / (WT / 8) * kT + i % (WT / 8) * 16);
            }
#pragma unroll
            for (int m = 0; m < NB; m++) {
                const int i = lane + (n + m) * 64, c = i / (WT / 8), r = row0 + i % (WT / 8) * 8;
                store16(v[m], rd, r < rows ? (uint32_t)(c * ldd + r) * 2 : kNone);
            }
        }
    }
    // [row][column]: X, the tile of A or B itself, or O of a wide G
    if (MODE == APPLY ? !out || !p.tall : ti != tj) {
        const int64_t ldd = MODE != APPLY ? p.mp : out ? p.cols : p.np;
        h16 *dst = (MODE == GRAM ? p.A : MODE == POLY ? p.B : out ? (h16 *)p.O : p.X) + row0 * ldd;
        const __amdgpu_buffer_rsrc_t rd = rsrc(dst, (rows - row0) * ldd * 2);
        // 16 lanes: 16 rows of 8 columns, four columns a read (lane 4 e + q reads
        // rows 4 q .. 4 q + 3 of column e and receives row 4 e + q)
        const int e = lane >> 2 & 3, q = lane & 3, g = lane >> 4;
#pragma unroll 1
        for (int n = 0; n < kAll; n += NB) {
            u32x4 v[NB];
#pragma unroll
            for (int m = 0; m < NB; m++) {
                const int i = n + m, r = i / (WT / 32) * 16, c = i % (WT / 32) * 32 + g * 8;
                const char *at = T + (c + e) * kT + (r + 4 * q) * 2;
                const u32x2 lo = transposed(at), hi = transposed(at + 4 * kT);
                v[m] = u32x4{lo[0], lo[1], hi[0], hi[1]};
            }
#pragma unroll
            for (int m = 0; m < NB; m++) {
                const int i = n + m, r = i / (WT / 32) * 16 + (lane & 15), col = col0 + i % (WT / 32) * 32 + g * 8;
                store16(v[m], rd, col < cols ? (uint32_t)(r * ldd + col) * 2 : kNone);
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
    size_t x, xt0, xt1, xl, a, b, diag, part, total;   // byte offsets
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
    L.xl = 3 * mn;
    L.a = 4 * mn;
    L.b = 4 * mn + mm;
    L.diag = 4 * mn + 2 * mm;
    L.part = L.diag + al256((size_t)L.mp * 8);
    L.total = L.m ? L.part + al256(ndev::kParts * 8) : 0;
    return L;
}

bool sizes_ok(int64_t r, int64_t c) {
    // a launch counts its threads in 32 bits: 64 x 64 tiles of 256 threads
    return r >= 0 && c >= 0 && r <= kMaxInOut && c <= kMaxInOut && r % 8 == 0 && c % 8 == 0 &&
           cdiv(r, 64) * cdiv(c, 64) <= (1 << 20);
}

int64_t tiles_of(int mode, const OrthoOne &p, int wt) {
    const int64_t r = cdiv(p.mp, 2 * wt);
    return mode == ndev::APPLY ? r * cdiv(p.np, 2 * wt) : r * (r + 1) / 2;
}

// The tile shapes, and what a tile costs: us for its first loads, its results
// and the launch, and us per 32 K, alone on the chip and with every unit busy
// (measured on the products of 512 x 2048 to 4096 x 16384).  Large tiles need
// half the operand traffic a flop; small ones fill the chip sooner and
// start and end faster.
struct Shape {
    int wt, per_cu;
    double fixed, alone, busy;
};
constexpr Shape kShapes[] = {{128, 1, 14.0, 0.44, 1.10}, {96, 1, 9.0, 0.32, 0.65}, {64, 1, 6.0, 0.17, 0.33},
                             {32, 2, 4.5, 0.09, 0.21}};

// The cheapest shape.  Units that are all busy take the tiles in full rounds, and
// what is left over (the shortest sums, which come last) in one with less
// company; and the launch ends no sooner than its longest tile.  (Over 19 sizes,
// single and of six matrices, 128 x 8192 to 4096 x 16384, the choice is within
// 0.9 % of the best shape in the mean and 3 % but for four, all of the last product,
// whose low term the figures do not know: 1000 x 12000 takes 60 us where 256 x 256
// tiles take 52.  With full rounds only, 2048 x 2048 took the smallest tiles, 24 us
// against 18.)
int choose_shape(int mode, const OrthoArgs &a) {
    int best = 0;
    double least = 0.0;
    for (const Shape &s : kShapes) {
        double sum = 0.0, longest = 0.0, shortest = 0.0;
        int64_t tiles = 0;
        for (int i = 0; i < a.n; i++) {
            const int64_t n = tiles_of(mode, a.p[i], s.wt);
            const double k = (mode == ndev::GRAM ? a.p[i].np : a.p[i].mp) / 32.0;
            tiles += n;
            sum += (double)n * k;
            longest = k > longest ? k : longest;
            shortest = i == 0 || k < shortest ? k : shortest;
        }
        const int slots = 256 * s.per_cu;
        auto rate = [&](int64_t n) { return s.alone + (s.busy - s.alone) * (double)(n < slots ? n : slots) / slots; };
        const int64_t left = tiles % slots;
        const double rounds = (sum - (double)left * shortest) / slots * s.busy + (left ? shortest * rate(left) : 0.0);
        const double t = s.fixed + std::max(rounds, longest * rate(tiles));
        if (!best || t < least) best = s.wt, least = t;
    }
    return best;
}

template <int MODE>
void launch_product(int wt, OrthoArgs &a, hipStream_t st) {
    int64_t wgs = 0;
    for (int i = 0; i < a.n; i++) {
        a.p[i].start = (int)wgs;
        a.p[i].tiles = (int)tiles_of(MODE, a.p[i], wt);
        wgs += a.p[i].tiles;
    }
    const dim3 g((unsigned)wgs), b(256);
    if (wt == 128) hipLaunchKernelGGL((ndev::ortho_gemm_kernel<128, 32, 4, MODE>), g, b, 0, st, a);
    else if (wt == 96) hipLaunchKernelGGL((ndev::ortho_gemm_kernel<96, 32, 4, MODE>), g, b, 0, st, a);
    else if (wt == 64) hipLaunchKernelGGL((ndev::ortho_gemm_kernel<64, 64, 5, MODE>), g, b, 0, st, a);
    else hipLaunchKernelGGL((ndev::ortho_gemm_kernel<32, 64, (MODE == ndev::APPLY ? 3 : 5), MODE>), g, b, 0, st, a);
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
        p.XL = (ndev::h16 *)(w + L.xl);
        p.A = (ndev::h16 *)(w + L.a);
        p.B = (ndev::h16 *)(w + L.b);
        p.diag = (float2 *)(w + L.diag);
        p.part = (double *)(w + L.part);
        p.rows = mats[i].rows; p.cols = mats[i].cols;
        p.m = (int)L.m; p.n = (int)L.n; p.mp = (int)L.mp; p.np = (int)L.np;
        p.gain = mats[i].gain;
        p.tall = mats[i].rows > mats[i].cols;
    }
    if (a.n == 0) return TERN_OK;
    hipStream_t st = (hipStream_t)stream;
    hipLaunchKernelGGL(ndev::ortho_norm_kernel, dim3(ndev::kParts, (unsigned)a.n), dim3(256), 0, st, a);
    int64_t tiles = 0;
    for (int i = 0; i < a.n; i++) {
        a.p[i].start = (int)tiles;
        tiles += (int64_t)(a.p[i].mp / 64) * (a.p[i].np / 64);
    }
    hipLaunchKernelGGL(ndev::ortho_load_kernel, dim3((unsigned)tiles), dim3(256), 0, st, a);
    // the longest sums first
    std::stable_sort(a.p, a.p + a.n, [](const OrthoOne &x, const OrthoOne &y) { return x.np > y.np; });
    const int gram = choose_shape(ndev::GRAM, a), poly = choose_shape(ndev::POLY, a),
              apply = choose_shape(ndev::APPLY, a);
    for (int s = 0; s < steps; s++) {
        a.flip = s & 1;
        a.last = s == steps - 1;
        a.near = s >= steps - 2;
        launch_product<ndev::GRAM>(gram, a, st);
        launch_product<ndev::POLY>(poly, a, st);
        launch_product<ndev::APPLY>(apply, a, st);
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
