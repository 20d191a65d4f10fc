// tern_q4.hip -- products of a few rows with 4-bit weights and group scales
// (C ABI in include/tern.h):
//
//   Y[t, c] = sum_r X[t, r] q[r, c] s[r / group, c],   -8 <= q <= 7
//
// With few rows the weights' bytes are the work: every wave streams them once,
// 16 bytes a lane, and the matrix cores do the sums, so that decoding is all
// the vector units have to do.
//
// Decoding.  A code u = q + 8 placed in the top four mantissa bits of the
// bf16 16.0 is the bf16 16 + u = 24 + q: a shift and one and-or give two
// weights.  The products of 24 + q with bf16 activations are exact in fp32;
// the 24 sum_r X[t, r] too much is taken off by the start of the sum, the
// same sum made by a matrix instruction with -24 in the place of every weight
// (one for all column blocks of a wave).  So a sum of 32 products holds terms up to
// 31 |x| where q x is meant.  Of activations within some 6 binary orders of each
// other it is exact all the same (8 bits times 5, 32 of them), and what it is added to
// no longer holds the 24 x: results are nearer than a plain fp32 sum's (16384 rows:
// 1.1e-7 to 4e-7 against 1.1e-6, activations of one sign included; over 6 decimal orders
// 1.8e-6).
//
// fp32 activations are cut into three bf16 terms of 8 significant bits each,
// exactly, and multiplied term by term: the first terms' sum as above, the small
// ones' in a sum of their own, added to it once nothing is left of its 24 x (all in one
// sum, which rounds at 24 sum x from the second term on, gave 0.4e-6 to 3.2e-6).
//
// What bounds it (times of a call in a recorded chain of eight, each with weights of its
// own): one bf16 token of 4096 x 16384 takes 13.8 us, 2.7 TB/s of the 5.1 of a copy
// (about 3 us are the launch's start and the first loads); three 2048 x 2048 6.4 us, two
// thirds of it that latency.  The rows are split among the waves of one workgroup only,
// so narrow matrices leave units idle: 8192 x 2048 (128 workgroups for 256 units) takes
// 7.6 us, 16384 x 512 10.4.  More tokens read the activations once a column block, through
// shared memory (16 bf16 tokens of 16384 x 4096 17.5 us); fp32 ones pass it as 12 KiB a
// block and wave and are cut there, in every workgroup anew, which bounds one token of
// 16384 x 4096 at 19 us and 13 at 27, 1.4 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/tern.h"
#include "tern_plan.h"

namespace tern {
namespace qdev {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kCols = 16, kRows = 128;          // a block of the packed matrix: 1 KiB
constexpr int kBlockWords = kCols * kRows / 8;
// waves of a workgroup, at most: 16 where 128 registers a lane are enough; with fp32
// activations shared memory holds 12
constexpr int max_waves(int terms, int nb) { return nb == 1 ? (terms == 1 ? 16 : 12) : 8; }

// Word w of lane l of a block: rows 32 w + 8 (l / 16) + e (e < 8), column
// l % 16.  Rows e = 2 d and 2 d + 1 stand at bits 4 d + 3 and 4 d + 19 (mod 32), so
// that a rotation by 4 d brings both into place.
__global__ __launch_bounds__(256) void q4_pack_kernel(const int8_t *__restrict__ q, int64_t in, int64_t out,
                                                      int64_t nkb, int64_t words, uint32_t *__restrict__ packed) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= words) return;
    const int64_t blk = i / kBlockWords;
    const int in_blk = (int)(i % kBlockWords), l = in_blk >> 2, w = in_blk & 3;
    const int64_t cb = blk / nkb, kb = blk - cb * nkb;
    const int64_t c = cb * kCols + (l & 15), r0 = kb * kRows + w * 32 + (l >> 4) * 8;
    uint32_t x = 0;
    for (int e = 0; e < 8; e++) {
        int v = 0;
        if (c < out && r0 + e < in) v = q[(r0 + e) * out + c];
        v = v < -8 ? -8 : v > 7 ? 7 : v;
        const uint32_t u = (uint32_t)(v + 8);
        const int sh = (e & 1) * 16 + (e >> 1) * 4 + 3;
        x |= u << (sh & 31);
        if (sh > 28) x |= u >> (32 - sh);   // the last code wraps into bits 0..2
    }
    packed[i] = x;
}

struct Q4One {
    const void *X;
    const uint32_t *packed;
    const void *gscale;
    void *Y;
    int in, out, nkb, group_chunks;   // group_chunks: 32-row chunks of a group (1, 2, 4)
    int runs, per, more;              // runs of row blocks: nkb = runs * per + more
    int wave_runs;                    // runs a wave takes
    int inv;                          // 2^16 / runs, rounded up
    int start;                        // first workgroup
    // of the row blocks that are over, how many runs before run r take one more:
    // floor(r more / runs), exact for up to 16 runs
    __device__ int over(int r) const { return (int)((unsigned)(r * more * inv) >> 16); }
};
struct Q4Args {
    Q4One p[kMaxGroup];
    int n, T, waves, y_bf16;
    int rows;                         // tokens of a workgroup, at most 16
};

// A projection's row blocks are cut into runs.  The sum of a run and the order in
// which they are added are the projection's alone; which wave takes which runs is
// the call's.  So the result is the same, bit for bit, whatever else the call holds.
// Runs: about 4 row blocks each, what a wave needs to hide its loads (one bf16 token
// of 4096 x 4096 6.3 us, runs of 8 7.9; 2600 x 2600 5.4 and 6.4; 5000 x 5000, with
// more column blocks than units, 10.7 and 8.5), in fours, so that 4 waves share them
// evenly, and no more than one a wave of the largest workgroup.  A projection whose
// columns alone fill the chip (pair() below) needs only 4.  A wave that takes 4 runs
// spends about 0.2 us on each: the six matrices of d = 2048 14.9 us (split for the
// whole call, with bits that follow the company, 14.1).
constexpr int kPairFrom = 1024;   // column blocks
inline bool pair(int64_t column_blocks) { return column_blocks >= kPairFrom; }
inline int64_t runs_of(int64_t nkb, int64_t ncb, int terms) {
    int64_t runs = pair(ncb) || nkb < 16 ? 4 : (nkb + 15) / 16 * 4;
    if (runs > max_waves(terms, 1)) runs = max_waves(terms, 1);
    return runs < nkb ? runs : nkb;
}

__device__ inline f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ inline bf16x8 weights(uint32_t w) {
    u32x4 r;
#pragma unroll
    for (int d = 0; d < 4; d++) {
        const uint32_t x = d ? __builtin_amdgcn_alignbit(w, w, 4 * d) : w;
        r[d] = (x & 0x00780078u) | 0x41804180u;
    }
    return __builtin_bit_cast(bf16x8, r);
}

// A wave's activations of 128 rows.  They are loaded in whole lines, a lane 16
// bytes of a token's row, and brought through shared memory into the order of the
// matrix instruction, whose lanes stand at 16 different tokens (loaded in that order,
// every lane's 16 bytes cost the L1 cache an access of their own, which bound the
// kernel: 13 rows of 16384 x 4096 in fp32 took 33.7 us, 16 in bf16 23.8).
// fp32 ones are cut on the way, TERMS matrices of bf16, for the tokens that are
// there; the places of other tokens hold anything, and spoil only results that are
// not written.
// The 16-byte pieces of a token's row are permuted by its number, so that
// equal pieces of the 16 tokens fall in different banks.
template <int TERMS>
struct Rows {
    static constexpr int ES = TERMS == 1 ? 2 : 4, kTerm = 16 * kRows * 2, kBytes = TERMS * kTerm;
    static constexpr int kPieces = kRows * ES / 16, kPer = 64 / kPieces, kLoads = 16 / kPer;   // kPer: tokens a load
    u32x4 v[kLoads];
    __device__ static char *place(char *lds, int tok, int piece) { return lds + tok * kRows * 2 + (piece ^ tok) * 16; }
    // rows r0 .. of the tokens at X (nt of them)
    __device__ void load(const char *X, int nt, int in, int r0, int lane) {
        const int t = lane / kPieces, piece = lane % kPieces;
        const uint32_t at = (uint32_t)(t * in * ES + piece * 16);
        const bool ok = r0 + piece * (16 / ES) < in;
        const char *p = X + (int64_t)r0 * ES;
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            v[j] = u32x4{0, 0, 0, 0};
            if (ok && j * kPer + t < nt) v[j] = *(const u32x4 *)(p + (int64_t)j * kPer * in * ES + at);
        }
    }
    __device__ void store(char *lds, int nt, int lane) const {
        const int t = lane / kPieces, piece = lane % kPieces;
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            if (j * kPer >= nt) continue;
            if constexpr (TERMS == 1) {
                *(u32x4 *)place(lds, j * kPer + t, piece) = v[j];
            } else {
                // 4 values, each cut into terms of 8 significant bits
                uint32_t x[4] = {v[j][0], v[j][1], v[j][2], v[j][3]};
                char *at = place(lds, j * kPer + t, piece >> 1) + (piece & 1) * 8;
#pragma unroll
                for (int i = 0; i < TERMS; i++) {
                    *(u32x2 *)(at + i * kTerm) = u32x2{__builtin_amdgcn_perm(x[1], x[0], 0x07060302u),   // upper halves
                                                       __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        x[e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, x[e]) -
                                                                __builtin_bit_cast(float, x[e] & 0xFFFF0000u));
                }
            }
        }
    }
    // 8 activations of a token, rows 32 ck + 8 sub .., of one term
    __device__ static bf16x8 read(const char *lds, int term, int tok, int ck, int sub) {
        return *(const bf16x8 *)place(const_cast<char *>(lds) + term * kTerm, tok, ck * 4 + sub);
    }
};

// the 4 scales of a lane's columns: as loaded, and as fp32
template <bool SBF>
struct Scales {
    using Raw = std::conditional_t<SBF, u32x2, f32x4>;
    __device__ static Raw load(const void *s, int64_t at) {
        return *(const Raw *)((const char *)s + at * (SBF ? 2 : 4));
    }
    __device__ static f32x4 get(Raw v) {
        if constexpr (SBF)
            return f32x4{__builtin_bit_cast(float, v[0] << 16), __builtin_bit_cast(float, v[0] & 0xFFFF0000u),
                         __builtin_bit_cast(float, v[1] << 16), __builtin_bit_cast(float, v[1] & 0xFFFF0000u)};
        else
            return v;
    }
};

// Blocks k0 .. k1 - 1 of a wave's NB column blocks, whole runs from r0 on, of each of
// which `done` takes the sums (GC: 32-row chunks of a scale group).  The weights, which come from HBM, are loaded kAhead blocks ahead, the
// activations and scales, which mostly come from L2, one block ahead.
constexpr int kAhead = 2;
template <int TERMS, bool SBF, int NB, int GC, class Done>
__device__ inline void run_blocks(const Q4One &p, const char *X, int nt, int lane, char *lds, const u32x4 *const (&W)[NB],
                                  const int (&col)[NB], int r0, int k0, int k1, Done done) {
    using Sc = typename Scales<SBF>::Raw;
    const int ng = (p.in + GC * 32 - 1) / (GC * 32), tok = lane & 15, sub = lane >> 4;
    u32x4 w[kAhead][NB];
    f32x4 y[NB];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < NB; i++) y[i] = f32x4{0, 0, 0, 0};
    };
    clear();
    // the row blocks left of the run: its share, and one more as the remainders add up
    int run = r0, rest = r0 * p.more - p.over(r0) * p.runs, left;
    auto begin = [&] {
        rest += p.more;
        left = p.per + (rest >= p.runs);
        rest -= rest >= p.runs ? p.runs : 0;
    };
    begin();
    Rows<TERMS> rows;
    Sc sc[2][4 / GC][NB];
    auto load_w = [&](u32x4 (&o)[NB], int kb) {
#pragma unroll
        for (int i = 0; i < NB; i++) o[i] = W[i][(int64_t)(kb < k1 ? kb : k1 - 1) * 64];
    };
    auto load_s = [&](Sc (&o)[4 / GC][NB], int kb) {
#pragma unroll
        for (int g = 0; g < 4 / GC; g++) {
            // a group past the last row (its weights multiply zeros) takes the last scale
            const int at = kb * (4 / GC) + g;
#pragma unroll
            for (int i = 0; i < NB; i++)
                o[g][i] = Scales<SBF>::load(p.gscale, (int64_t)(at < ng ? at : ng - 1) * p.out + col[i]);
        }
    };
    bf16x8 off;
#pragma unroll
    for (int e = 0; e < 8; e++) off[e] = (__bf16)-24.0f;
    auto work = [&](const u32x4 (&wb)[NB], const Sc (&sb)[4 / GC][NB]) {
#pragma unroll
        for (int g = 0; g < 4 / GC; g++) {
            f32x4 acc[NB];
#pragma unroll
            for (int c = 0; c < GC; c++) {
                const int ck = g * GC + c;
                bf16x8 x[TERMS];
#pragma unroll
                for (int t = 0; t < TERMS; t++) x[t] = Rows<TERMS>::read(lds, t, tok, ck, sub);
                const f32x4 none = {0, 0, 0, 0};
                const f32x4 high = mfma(off, x[0], none);
                f32x4 rest = none;
#pragma unroll
                for (int t = 1; t < TERMS; t++) rest = mfma(off, x[t], rest);
#pragma unroll
                for (int i = 0; i < NB; i++) {
                    const bf16x8 q = weights(wb[i][ck]);
                    f32x4 sum = mfma(q, x[0], high);
                    if (TERMS > 1) {
                        f32x4 low = rest;
#pragma unroll
                        for (int t = 1; t < TERMS; t++) low = mfma(q, x[t], low);
                        sum += low;
                    }
                    acc[i] = c ? acc[i] + sum : sum;
                }
            }
#pragma unroll
            for (int i = 0; i < NB; i++) {
                const f32x4 s = Scales<SBF>::get(sb[g][i]);
#pragma unroll
                for (int r = 0; r < 4; r++) y[i][r] = fmaf(s[r], acc[i][r], y[i][r]);
            }
        }
    };
#pragma unroll
    for (int j = 0; j < kAhead; j++) load_w(w[j], k0 + j);
    rows.load(X, nt, p.in, k0 * kRows, lane);
    load_s(sc[0], k0);
    for (int kb = k0; kb < k1; kb += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            if (kb + j < k1) {
                const int next = kb + j + 1 < k1 ? kb + j + 1 : k1 - 1;
                // (the fences keep the order of a wave's own accesses to its piece of
                // shared memory, which needs no wait)
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                rows.store(lds, nt, lane);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                rows.load(X, nt, p.in, next * kRows, lane);
                load_s(sc[(j + 1) & 1], next);
                __builtin_amdgcn_sched_barrier(0);
                work(w[j], sc[j & 1]);
                load_w(w[j], kb + j + kAhead);
                __builtin_amdgcn_sched_barrier(0);
                if (--left == 0) {
                    done(run++, y);
                    clear();
                    begin();
                }
            }
        }
    }
}

// One workgroup: NB column blocks, 16 tokens, all rows, the rows' blocks
// dealt to the waves in runs, whose sums meet in shared memory and are added in
// their order.
template <int TERMS, bool SBF, int NB>
__global__ __launch_bounds__(64 * max_waves(TERMS, NB)) void q4_kernel(Q4Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];   // lds_bytes()
    constexpr int kLine = NB * kCols + 4;
    float *const red = (float *)(lds + a.waves * Rows<TERMS>::kBytes);   // [run][token][kLine]
    int pi = 0;
    while (pi + 1 < a.n && (int)blockIdx.x >= a.p[pi + 1].start) pi++;
    const Q4One p = a.p[pi];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tok0 = blockIdx.y * 16, sub = lane >> 4;
    const int nt = a.T - tok0 < 16 ? a.T - tok0 : 16;
    const char *X = (const char *)p.X + (int64_t)tok0 * p.in * Rows<TERMS>::ES;
    char *xs = lds + wave * Rows<TERMS>::kBytes;
    const int ncb = (p.out + kCols - 1) / kCols;
    const int cb0 = ((int)blockIdx.x - p.start) * NB;
    const int r0 = wave * p.wave_runs, r1 = r0 + p.wave_runs < p.runs ? r0 + p.wave_runs : p.runs;
    const int k0 = r0 * p.per + p.over(r0), k1 = r1 * p.per + p.over(r1);

    const u32x4 *W[NB];
    int col[NB];   // first of the 4 columns a lane accumulates
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const int cb = cb0 + b < ncb ? cb0 + b : ncb - 1;
        W[b] = (const u32x4 *)p.packed + ((int64_t)cb * p.nkb) * 64 + lane;
        const int c = cb * kCols + sub * 4;
        col[b] = c < p.out ? c : 0;   // the last block may be half full (out is a multiple of 8)
    }
    auto done = [&](int run, const f32x4 (&y)[NB]) {
        float *to = red + (run * a.rows + (lane & 15)) * kLine + sub * 4;
        if ((lane & 15) < a.rows)
#pragma unroll
            for (int b = 0; b < NB; b++) *(f32x4 *)(to + b * kCols) = y[b];
    };
    if (r0 < r1) {
        if (p.group_chunks == 1) run_blocks<TERMS, SBF, NB, 1>(p, X, nt, lane, xs, W, col, r0, k0, k1, done);
        else if (p.group_chunks == 2) run_blocks<TERMS, SBF, NB, 2>(p, X, nt, lane, xs, W, col, r0, k0, k1, done);
        else run_blocks<TERMS, SBF, NB, 4>(p, X, nt, lane, xs, W, col, r0, k0, k1, done);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * NB * kCols; i += a.waves * 64) {
        const int t = i / (NB * kCols), c = i % (NB * kCols);
        const float *from = red + t * kLine + c;
        float v = p.runs ? *from : 0.0f;
        for (int r = 1; r < p.runs; r++) v += *(from += a.rows * kLine);
        const int oc = cb0 * kCols + c;
        if (oc < p.out) {
            const int64_t o = (int64_t)(tok0 + t) * p.out + oc;
            if (a.y_bf16) ((__bf16 *)p.Y)[o] = (__bf16)v;
            else ((float *)p.Y)[o] = v;
        }
    }
}

template <int TERMS, int NB>
int lds_bytes(const Q4Args &a) {
    int runs = 1;
    for (int i = 0; i < a.n; i++) runs = std::max(runs, a.p[i].runs);
    return a.waves * Rows<TERMS>::kBytes + runs * a.rows * (NB * kCols + 4) * 4;
}

}  // namespace qdev

namespace {

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void *p) { return ((uintptr_t)p & 15u) != 0; }
size_t esize(int32_t dt) { return dt == TERN_BF16 ? 2 : 4; }
bool type_ok(int32_t dt) { return dt == TERN_F32 || dt == TERN_BF16; }
int64_t packed_bytes(int64_t in, int64_t out) {
    return cdiv(out, qdev::kCols) * cdiv(in, qdev::kRows) * qdev::kBlockWords * 4;
}
bool sizes_ok(int64_t in, int64_t out) {
    return in >= 0 && out >= 0 && in <= kMaxInOut && out <= kMaxInOut && in % 8 == 0 && out % 8 == 0;
}

template <int TERMS, bool SBF>
void launch_nb(int nb, dim3 g, dim3 b, hipStream_t st, const qdev::Q4Args &a) {
    if (nb == 1) hipLaunchKernelGGL((qdev::q4_kernel<TERMS, SBF, 1>), g, b, (qdev::lds_bytes<TERMS, 1>(a)), st, a);
    else hipLaunchKernelGGL((qdev::q4_kernel<TERMS, SBF, 2>), g, b, (qdev::lds_bytes<TERMS, 2>(a)), st, a);
}

}  // namespace
}  // namespace tern

using namespace tern;

extern "C" {

int64_t tern_q4_packed_bytes(int64_t in, int64_t out) {
    if (!sizes_ok(in, out)) return -1;
    return packed_bytes(in, out);
}

int tern_q4_pack(const int8_t *q, int64_t in, int64_t out, uint32_t *packed, void *stream) {
    if (!sizes_ok(in, out)) return TERN_ERR_SHAPE;
    const int64_t pb = packed_bytes(in, out);
    if (pb == 0) return TERN_OK;
    if (!q || !packed) return TERN_ERR_NULL;
    if (misaligned(packed)) return TERN_ERR_ALIGN;
    if (ranges_overlap(q, (size_t)in * out, packed, (size_t)pb)) return TERN_ERR_ALIAS;
    const int64_t words = pb / 4, blocks = cdiv(words, 256);
    if (blocks > INT64_C(0xFFFFFF)) return TERN_ERR_SHAPE;   // a launch counts its threads in 32 bits
    hipLaunchKernelGGL(qdev::q4_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, q, in, out,
                       cdiv(in, qdev::kRows), words, packed);
    return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP;
}

int tern_layer_q4_matvec(const tern_q4_proj_t *projs, int32_t n, int64_t T, int32_t act_dtype, int32_t scale_dtype,
                         int32_t y_dtype, void *stream) {
    if (n < 1 || n > kMaxGroup) return TERN_ERR_SHAPE;
    if (!projs) return TERN_ERR_NULL;
    if (T < 0 || T > INT64_C(16) * 65535) return TERN_ERR_SHAPE;
    for (int i = 0; i < n; i++) {
        if (!sizes_ok(projs[i].in, projs[i].out)) return TERN_ERR_SHAPE;
        if (projs[i].group != 32 && projs[i].group != 64 && projs[i].group != 128) return TERN_ERR_VALUE;
    }
    if (!type_ok(act_dtype) || !type_ok(scale_dtype)) return TERN_ERR_DTYPE;
    if (!(y_dtype == TERN_F32 || (y_dtype == TERN_BF16 && act_dtype == TERN_BF16))) return TERN_ERR_DTYPE;
    struct Span {
        const void *p;
        size_t n;
    } outs[kMaxGroup], ins[3 * kMaxGroup];
    for (int i = 0; i < n; i++) {
        const tern_q4_proj_t &p = projs[i];
        const size_t xb = (size_t)T * p.in * esize(act_dtype), yb = (size_t)T * p.out * esize(y_dtype);
        const size_t pb = (size_t)packed_bytes(p.in, p.out);
        const size_t sb = (size_t)cdiv(p.in, p.group) * p.out * esize(scale_dtype);
        if ((xb && !p.X) || (yb && !p.Y) || (pb && !p.packed) || (sb && !p.gscale)) return TERN_ERR_NULL;
        if (misaligned(p.X) || misaligned(p.Y) || misaligned(p.packed) || misaligned(p.gscale)) return TERN_ERR_ALIGN;
        outs[i] = {p.Y, yb};
        ins[3 * i] = {p.X, xb};
        ins[3 * i + 1] = {p.packed, pb};
        ins[3 * i + 2] = {p.gscale, sb};
    }
    for (int i = 0; i < n; i++) {
        for (int j = i + 1; j < n; j++)
            if (ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return TERN_ERR_ALIAS;
        for (int j = 0; j < 3 * n; j++)
            if (ranges_overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return TERN_ERR_ALIAS;
    }
    qdev::Q4Args a{};
    // Shape of the launch.  From 1024 column blocks on (4 a compute unit) a
    // wave takes two, which share its activations, and 4 waves share the rows:
    // 4096 x 16384, one bf16 token 13.8 us against 14.7 with single blocks, 16 fp32
    // tokens 22.5 against 38.4, the six matrices of d = 2048 14.9 against 20.8.  Fewer
    // blocks take one each (4096 x 4096 6.3 us against 8.4 with two, 16 tokens of
    // 16384 x 4096 17.5 against 30.5), and as many waves as the longest sums have runs.
    const int terms = act_dtype == TERN_F32 ? 3 : 1;
    int64_t ncb = 0, waves = 1;
    for (int i = 0; i < n; i++) ncb += cdiv(projs[i].out, qdev::kCols);
    const int nb = qdev::pair(ncb) ? 2 : 1;
    auto runs_of = [&](const tern_q4_proj_t &p) {
        return qdev::runs_of(cdiv(p.in, qdev::kRows), cdiv(p.out, qdev::kCols), terms);
    };
    for (int i = 0; i < n; i++) waves = std::max(waves, runs_of(projs[i]));
    a.waves = (int)(nb == 2 ? std::min<int64_t>(waves, 4) : waves);
    a.T = (int)T;
    a.rows = (int)std::min<int64_t>(T, 16);
    for (int i = 0; i < n; i++) {
        const tern_q4_proj_t &p = projs[i];
        if (p.out == 0) continue;
        qdev::Q4One &o = a.p[a.n++];
        o.X = p.X; o.packed = p.packed; o.gscale = p.gscale; o.Y = p.Y;
        o.in = (int)p.in; o.out = (int)p.out; o.nkb = (int)cdiv(p.in, qdev::kRows);
        o.group_chunks = (int)(p.group / 32);
        o.runs = (int)runs_of(p);
        o.per = o.runs ? o.nkb / o.runs : 0;
        o.more = o.runs ? o.nkb % o.runs : 0;
        o.inv = o.runs ? (65535 + o.runs) / o.runs : 0;
        o.wave_runs = (int)cdiv(o.runs, a.waves);
    }
    // the longest sums start first (each projection's results are its own)
    std::stable_sort(a.p, a.p + a.n, [](const qdev::Q4One &x, const qdev::Q4One &y) { return x.nkb > y.nkb; });
    int64_t wgs = 0;
    for (int i = 0; i < a.n; i++) {
        a.p[i].start = (int)wgs;
        wgs += cdiv(cdiv(a.p[i].out, qdev::kCols), nb);
    }
    if (wgs == 0 || T == 0) return TERN_OK;
    const dim3 g((unsigned)wgs, (unsigned)cdiv(T, 16)), b((unsigned)(a.waves * 64));
    hipStream_t st = (hipStream_t)stream;
    a.y_bf16 = y_dtype == TERN_BF16;
    const bool sbf = scale_dtype == TERN_BF16;
    if (act_dtype == TERN_F32) {
        if (sbf) launch_nb<3, true>(nb, g, b, st, a);
        else launch_nb<3, false>(nb, g, b, st, a);
    } else {
        if (sbf) launch_nb<1, true>(nb, g, b, st, a);
        else launch_nb<1, false>(nb, g, b, st, a);
    }
    return hipGetLastError() == hipSuccess ? TERN_OK : TERN_ERR_HIP;
}

int tern_q4_matvec(const void *X, int32_t act_dtype, const uint32_t *packed, const void *gscale, int32_t scale_dtype,
                   int64_t group, int64_t T, int64_t in, int64_t out, void *Y, int32_t y_dtype, void *stream) {
    const tern_q4_proj_t p = {in, out, group, packed, gscale, X, Y};
    return tern_layer_q4_matvec(&p, 1, T, act_dtype, scale_dtype, y_dtype, stream);
}

}  // extern "C"
