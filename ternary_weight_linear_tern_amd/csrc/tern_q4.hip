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
// the 24 sum_r X[t, r] too much is taken off by the accumulator's start, the
// same sum made by a matrix instruction with -24 in the place of every weight
// (one for all column blocks of a wave).  The sums then hold terms up to 31
// |x| where q x is meant: about 5 times the rounding of a sum of q x.
//
// fp32 activations are cut into three bf16 terms of 8 significant bits each,
// exactly, and multiplied term by term.
#include <hip/hip_runtime.h>
#include <stdint.h>
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
// waves of a workgroup: 16 where 128 registers a lane are enough
constexpr int max_waves(int terms, int nb) { return terms == 1 && nb == 1 ? 16 : 8; }

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
    int start;                        // first workgroup
};
struct Q4Args {
    Q4One p[kMaxGroup];
    int n, T, waves, y_bf16;
};

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
// The 16-byte pieces of a token's row are permuted by its number, so that
// equal pieces of the 16 tokens fall in different banks.
template <int TERMS>
struct Rows {
    static constexpr int ES = TERMS == 1 ? 2 : 4, kRowBytes = kRows * ES, kBytes = 16 * kRowBytes;
    static constexpr int kPieces = kRowBytes / 16, kPer = 64 / kPieces, kLoads = 16 / kPer;   // kPer: tokens a load
    u32x4 v[kLoads];
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
    __device__ void store(char *lds, int lane) const {
        const int t = lane / kPieces, piece = lane % kPieces;
#pragma unroll
        for (int j = 0; j < kLoads; j++)
            *(u32x4 *)(lds + (j * kPer + t) * kRowBytes + ((piece ^ (j * kPer + t)) * 16)) = v[j];
    }
};

// 8 activations of a lane's token: as loaded, and as bf16 terms (TERMS 1:
// bf16 activations; 3: fp32, cut into three terms of 8 significant bits)
template <int TERMS>
struct RawActs {
    static constexpr int kPieces = TERMS == 1 ? 1 : 2;
    u32x4 v[kPieces];
    __device__ void read(const char *lds, int tok, int ck, int sub) {
#pragma unroll
        for (int i = 0; i < kPieces; i++)
            v[i] = *(const u32x4 *)(lds + tok * Rows<TERMS>::kRowBytes + (((ck * 4 + sub) * kPieces + i) ^ tok) * 16);
    }
};
template <int TERMS>
struct Acts {
    bf16x8 t[TERMS];
};
template <int TERMS>
__device__ inline Acts<TERMS> terms(const RawActs<TERMS> &a) {
    Acts<TERMS> r;
    if constexpr (TERMS == 1) {
        r.t[0] = __builtin_bit_cast(bf16x8, a.v[0]);
    } else {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = a.v[i >> 2][i & 3];
#pragma unroll
        for (int t = 0; t < 3; t++) {
            u32x4 o;
#pragma unroll
            for (int d = 0; d < 4; d++) o[d] = __builtin_amdgcn_perm(v[2 * d + 1], v[2 * d], 0x07060302u);   // upper halves
            r.t[t] = __builtin_bit_cast(bf16x8, o);
#pragma unroll
            for (int i = 0; i < 8; i++)
                v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, v[i]) -
                                                        __builtin_bit_cast(float, v[i] & 0xFFFF0000u));
        }
    }
    return r;
}

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

// Blocks k0 .. k1 - 1 of a wave's NB column blocks (GC: 32-row chunks of a scale
// group).  The weights, which come from HBM, are loaded kAhead blocks ahead, the
// activations and scales, which mostly come from L2, one block ahead.
constexpr int kAhead = 2;
template <int TERMS, bool SBF, int NB, int GC>
__device__ inline void run_blocks(const Q4One &p, const char *X, int nt, int lane, char *lds, const u32x4 *const (&W)[NB],
                                  const int (&col)[NB], int k0, int k1, f32x4 (&y)[NB]) {
    using Sc = typename Scales<SBF>::Raw;
    const int ng = (p.in + GC * 32 - 1) / (GC * 32), tok = lane & 15, sub = lane >> 4;
    u32x4 w[kAhead][NB];
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
                RawActs<TERMS> raw;
                raw.read(lds, tok, ck, sub);
                const Acts<TERMS> x = terms<TERMS>(raw);
                f32x4 z = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < TERMS; t++) z = mfma(off, x.t[t], z);
#pragma unroll
                for (int i = 0; i < NB; i++) {
                    acc[i] = c ? acc[i] + z : z;
                    const bf16x8 q = weights(wb[i][ck]);
#pragma unroll
                    for (int t = 0; t < TERMS; t++) acc[i] = mfma(q, x.t[t], acc[i]);
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
                rows.store(lds, lane);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                rows.load(X, nt, p.in, next * kRows, lane);
                load_s(sc[(j + 1) & 1], next);
                __builtin_amdgcn_sched_barrier(0);
                work(w[j], sc[j & 1]);
                load_w(w[j], kb + j + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
}

// One workgroup: NB column blocks, 16 tokens, all rows, the rows' blocks
// dealt to the waves in runs; the waves' sums meet in shared memory in the
// order of the waves.
template <int TERMS, bool SBF, int NB>
__global__ __launch_bounds__(64 * max_waves(TERMS, NB)) void q4_kernel(Q4Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];   // lds_bytes()
    using Red = float[16][NB * kCols + 4];
    Red *const red = (Red *)(lds + a.waves * Rows<TERMS>::kBytes);
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
    const int per = (p.nkb + a.waves - 1) / a.waves;
    const int k0 = wave * per, k1 = k0 + per < p.nkb ? k0 + per : p.nkb;

    const u32x4 *W[NB];
    int col[NB];   // first of the 4 columns a lane accumulates
    f32x4 y[NB];
#pragma unroll
    for (int b = 0; b < NB; b++) {
        const int cb = cb0 + b < ncb ? cb0 + b : ncb - 1;
        W[b] = (const u32x4 *)p.packed + ((int64_t)cb * p.nkb) * 64 + lane;
        const int c = cb * kCols + sub * 4;
        col[b] = c < p.out ? c : 0;   // the last block may be half full (out is a multiple of 8)
        y[b] = f32x4{0, 0, 0, 0};
    }
    if (k0 < k1) {
        if (p.group_chunks == 1) run_blocks<TERMS, SBF, NB, 1>(p, X, nt, lane, xs, W, col, k0, k1, y);
        else if (p.group_chunks == 2) run_blocks<TERMS, SBF, NB, 2>(p, X, nt, lane, xs, W, col, k0, k1, y);
        else run_blocks<TERMS, SBF, NB, 4>(p, X, nt, lane, xs, W, col, k0, k1, y);
    }
#pragma unroll
    for (int b = 0; b < NB; b++) *(f32x4 *)&red[wave][lane & 15][b * kCols + sub * 4] = y[b];
    __syncthreads();
    for (int i = threadIdx.x; i < nt * NB * kCols; i += a.waves * 64) {
        const int t = i / (NB * kCols), c = i % (NB * kCols);
        float v = red[0][t][c];
        for (int w = 1; w < a.waves; w++) v += red[w][t][c];
        const int oc = cb0 * kCols + c;
        if (oc < p.out) {
            const int64_t o = (int64_t)(tok0 + t) * p.out + oc;
            if (a.y_bf16) ((__bf16 *)p.Y)[o] = (__bf16)v;
            else ((float *)p.Y)[o] = v;
        }
    }
}

template <int TERMS, int NB>
int lds_bytes(int waves) {
    return waves * (Rows<TERMS>::kBytes + 16 * (NB * kCols + 4) * 4);
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
    if (nb == 1) hipLaunchKernelGGL((qdev::q4_kernel<TERMS, SBF, 1>), g, b, (qdev::lds_bytes<TERMS, 1>(a.waves)), st, a);
    else hipLaunchKernelGGL((qdev::q4_kernel<TERMS, SBF, 2>), g, b, (qdev::lds_bytes<TERMS, 2>(a.waves)), st, a);
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
    // 4096 x 16384, one token 10.6 us against 11.8 with single blocks, 16 tokens
    // 14.1 against 20.7.  Fewer blocks take one each (4096 x 4096 5.3 us against
    // 6.1), and enough waves that each has about 4 row blocks, which is all it
    // needs to hide its loads (16384 x 2048: 16 waves 10.9 us, 8 13.1, 4 20.0;
    // three 2048 x 2048: 4 waves 5.2, 8 5.5, 16 7.7).
    int64_t maxk = 1, ncb = 0;
    for (int i = 0; i < n; i++) {
        maxk = projs[i].in > maxk ? projs[i].in : maxk;
        ncb += cdiv(projs[i].out, qdev::kCols);
    }
    const int nb = ncb >= 1024 ? 2 : 1;
    const int64_t nkb = cdiv(maxk, qdev::kRows);
    const int64_t most = qdev::max_waves(act_dtype == TERN_F32 ? 3 : 1, nb);
    int64_t waves = nb == 2 || nkb < 16 ? 4 : nkb / 4;
    if (waves > most) waves = most;
    if (waves > nkb) waves = nkb;
    a.waves = (int)waves;
    a.T = (int)T;
    int64_t wgs = 0;
    for (int i = 0; i < n; i++) {
        const tern_q4_proj_t &p = projs[i];
        if (p.out == 0) continue;
        qdev::Q4One &o = a.p[a.n++];
        o.X = p.X; o.packed = p.packed; o.gscale = p.gscale; o.Y = p.Y;
        o.in = (int)p.in; o.out = (int)p.out; o.nkb = (int)cdiv(p.in, qdev::kRows);
        o.group_chunks = (int)(p.group / 32);
        o.start = (int)wgs;
        wgs += cdiv(cdiv(p.out, qdev::kCols), nb);
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
