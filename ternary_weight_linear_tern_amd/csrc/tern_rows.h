// tern_rows.h -- device helpers of the kernels that reduce over a row (layer
// norm, softmax): eight elements at a time, sums and maxima over a wave and a
// workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/tern.h"

namespace tern {
namespace rows {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// (by value: __builtin_bit_cast of a vector's element reads its first one)
__device__ inline float as_f(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ inline uint32_t as_u(float x) { return __builtin_bit_cast(uint32_t, x); }

// Eight elements in memory: 16 bytes of bf16, 32 of fp32.
template <int DT>
struct Raw8 {
    static constexpr int N = DT == TERN_BF16 ? 1 : 2;
    u32x4 v[N];
};

template <int DT>
__device__ inline constexpr int esize() { return DT == TERN_BF16 ? 2 : 4; }

template <int DT>
__device__ inline Raw8<DT> load8(const void *p) {
    Raw8<DT> r;
#pragma unroll
    for (int i = 0; i < Raw8<DT>::N; i++) r.v[i] = ((const u32x4 *)p)[i];
    return r;
}
template <int DT>
__device__ inline void unpack8(const Raw8<DT> &r, float *f) {
    if constexpr (DT == TERN_BF16) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            f[2 * i] = as_f(r.v[0][i] << 16);
            f[2 * i + 1] = as_f(r.v[0][i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = as_f(r.v[i >> 2][i & 3]);
    }
}
// rounded to nearest even (NaN stays NaN)
template <int DT>
__device__ inline Raw8<DT> pack8(const float *f) {
    Raw8<DT> r;
    if constexpr (DT == TERN_BF16) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            r.v[0][i] = (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f[2 * i]) |
                        (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)f[2 * i + 1]) << 16;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) r.v[i >> 2][i & 3] = as_u(f[i]);
    }
    return r;
}
template <int DT>
__device__ inline void store8(void *p, const Raw8<DT> &r) {
#pragma unroll
    for (int i = 0; i < Raw8<DT>::N; i++) ((u32x4 *)p)[i] = r.v[i];
}

// one element
template <int DT>
__device__ inline float load1(const void *p) {
    if constexpr (DT == TERN_BF16) return __builtin_bit_cast(float, (uint32_t) * (const uint16_t *)p << 16);
    else return *(const float *)p;
}
template <int DT>
__device__ inline void store1(void *p, float f) {
    if constexpr (DT == TERN_BF16) *(uint16_t *)p = __builtin_bit_cast(unsigned short, (__bf16)f);
    else *(float *)p = f;
}

// Reductions over a wave; every lane gets the result, and the order of the
// operations is the same in all of them.  Four steps within 16 lanes, then the
// rows of 16 and the halves swapped.
struct Add {
    __device__ static float of(float a, float b) { return a + b; }
};
struct Max {   // NaN loses against a number
    __device__ static float of(float a, float b) { return fmaxf(a, b); }
};
template <int CTRL>
__device__ inline float dpp(float x) {
    return as_f((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u(x), CTRL, 0xF, 0xF, false));
}
// over groups of P = 8, 16, 32 or 64 neighbouring lanes
template <class Op>
__device__ inline float lanes_all(float x, int P) {
    x = Op::of(x, dpp<0xB1>(x));    // lane ^ 1
    x = Op::of(x, dpp<0x4E>(x));    // lane ^ 2
    x = Op::of(x, dpp<0x141>(x));   // mirrored in 8
    if (P > 8) x = Op::of(x, dpp<0x140>(x));   // mirrored in 16
    if (P > 16) {
        const auto a = __builtin_amdgcn_permlane16_swap(as_u(x), as_u(x), false, false);
        x = Op::of(as_f(a[0]), as_f(a[1]));
    }
    if (P > 32) {
        const auto b = __builtin_amdgcn_permlane32_swap(as_u(x), as_u(x), false, false);
        x = Op::of(as_f(b[0]), as_f(b[1]));
    }
    return x;
}
template <class Op>
__device__ inline float wave_all(float x) {
    return lanes_all<Op>(x, 64);
}

// Over the W waves of a workgroup; `sh` holds W floats and is free again after
// the next barrier.
template <class Op, int W>
__device__ inline float group_all(float x, float *sh) {
    x = wave_all<Op>(x);
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
        __syncthreads();
        x = sh[0];
#pragma unroll
        for (int i = 1; i < W; i++) x = Op::of(x, sh[i]);
    }
    return x;
}

}  // namespace rows
}  // namespace tern
