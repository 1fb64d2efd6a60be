// Device pieces that the 8-bit kernels share: vectors at any address that suits
// an element, and the element types.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp8.hpp"

namespace shampoo {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// A caller's pointer through the global address space.
template <typename T>
__device__ __forceinline__ T* gptr(uint64_t addr) {
    typedef __attribute__((address_space(1))) T gT;
    return (T*)reinterpret_cast<gT*>(addr);
}

template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

template <int DT> struct Elem { typedef unsigned short type; };
template <> struct Elem<DT_F32> { typedef float type; };

// Eight elements as they lie in memory.
template <int DT> struct Raw8 { u32x4 w; };
template <> struct Raw8<DT_F32> { f32x4 lo, hi; };

template <int DT>
__device__ __forceinline__ Raw8<DT> load8(uint64_t base, int64_t at) {
    typedef typename Elem<DT>::type T;
    const T* p = gptr<const T>(base) + at;
    Raw8<DT> r;
    if constexpr (DT == DT_F32) {
        r.lo = *reinterpret_cast<const f32x4u*>(p);
        r.hi = *reinterpret_cast<const f32x4u*>(p + 4);
    } else {
        r.w = *reinterpret_cast<const u32x4h*>(p);
    }
    return r;
}
// The first `left` of them, 1 to 7, and 0 for the others; without a branch, so
// that the eight loads are on their way together.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8_part(uint64_t base, int64_t at, int64_t left) {
    typedef typename Elem<DT>::type T;
    const T* p = gptr<const T>(base) + at;
    const int n = (int)left;
    T e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) e[k] = p[k < n ? k : n - 1];
    Raw8<DT> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == DT_F32) {
            r.lo[k] = k < n ? e[k] : 0.f;
            r.hi[k] = k + 4 < n ? e[k + 4] : 0.f;
        } else {
            r.w[k] = (2 * k < n ? (uint32_t)e[2 * k] : 0u) | (2 * k + 1 < n ? (uint32_t)e[2 * k + 1] : 0u) << 16;
        }
    }
    return r;
}
// As many of them as there are, none where `left` is not positive.
template <int DT>
__device__ __forceinline__ Raw8<DT> load8_upto(uint64_t base, int64_t at, int64_t left) {
    if (left >= 8) return load8<DT>(base, at);
    if (left > 0) return load8_part<DT>(base, at, left);
    return Raw8<DT>{};
}

__device__ __forceinline__ float half_value(uint32_t u) {
    const unsigned short s = (unsigned short)u;
    _Float16 h;
    __builtin_memcpy(&h, &s, 2);
    return (float)h;
}

template <int DT>
__device__ __forceinline__ void widen8(const Raw8<DT>& r, float* out) {
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            out[k] = r.lo[k];
            out[4 + k] = r.hi[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            out[2 * k] = DT == DT_BF16 ? __uint_as_float(r.w[k] << 16) : half_value(r.w[k]);
            out[2 * k + 1] = DT == DT_BF16 ? __uint_as_float(r.w[k] & 0xFFFF0000u) : half_value(r.w[k] >> 16);
        }
    }
}

// Two values in 16 bits each, rounded to nearest even.
template <int DT>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    uint32_t u;
    if constexpr (DT == DT_BF16) {
        const bf16x2 h = __builtin_convertvector(f32x2{a, b}, bf16x2);
        __builtin_memcpy(&u, &h, 4);
    } else {
        const f16x2 h = __builtin_convertvector(f32x2{a, b}, f16x2);
        __builtin_memcpy(&u, &h, 4);
    }
    return u;
}

// x as its type holds it.
template <int DT>
__device__ __forceinline__ float rounded(float x) {
    if constexpr (DT == DT_F32) return x;
    else if constexpr (DT == DT_BF16) return (float)(__bf16)x;
    else return (float)(_Float16)x;
}

template <int DT>
__device__ __forceinline__ void store8_upto(uint64_t base, int64_t at, int64_t left, const float* x) {
    typedef typename Elem<DT>::type T;
    T* p = gptr<T>(base) + at;
    if constexpr (DT == DT_F32) {
        if (left >= 8) {
            *reinterpret_cast<f32x4u*>(p) = f32x4{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4u*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) p[k] = x[k];
        }
    } else {
        const u32x4 w = {narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3]), narrow2<DT>(x[4], x[5]), narrow2<DT>(x[6], x[7])};
        if (left >= 8) {
            *reinterpret_cast<u32x4h*>(p) = w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < left) p[k] = (T)(w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

// Four codes as values.
template <int FMT>
__device__ __forceinline__ void values4(uint32_t u, float* out) {
    f32x2 a, b;
    if constexpr (FMT == F8_E4M3) {
        a = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, false);
        b = __builtin_amdgcn_cvt_pk_f32_fp8((int)u, true);
    } else {
        a = __builtin_amdgcn_cvt_pk_f32_bf8((int)u, false);
        b = __builtin_amdgcn_cvt_pk_f32_bf8((int)u, true);
    }
    out[0] = a.x;
    out[1] = a.y;
    out[2] = b.x;
    out[3] = b.y;
}

}  // namespace

}  // namespace shampoo
