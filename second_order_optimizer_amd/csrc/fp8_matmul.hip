// gfx950 kernels of the product of 8-bit matrices, C = A B^T (+ C), with a
// scale for each block of 128 of a row.
//
// Two ways to the sum, by the type of C.  bf16 and fp16: the matrix
// instructions that take 8-bit operands and a power of two for each 32 of them.
// They add products in eights, each cut off below 2^-13 of the largest, and
// those sums in fp32 (found by products of single powers of two): on normally
// distributed values 1.5e-5 of the result, with one column in a hundred
// twentyfold 4.4e-5, a fiftieth of what rounding to bf16 leaves.  fp32: the codes
// are widened to bf16 with their scale, exactly, and multiplied by the bf16
// instructions, whose sums are those of fp32 (6e-8 at K = 2048, 2e-7 at 16384),
// at half the rate: a weight's gradient that is added up over micro-batches
// keeps its small terms.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "fp8.hpp"
#include "fp8_device.hpp"

namespace shampoo {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Four neighbouring values of a row of C.
template <int DT>
__device__ __forceinline__ void store4(uint64_t base, int64_t at, int64_t left, f32x4 x, bool add) {
    typedef typename Elem<DT>::type T;
    T* p = gptr<T>(base) + at;
    if (left >= 4) {
        if constexpr (DT == DT_F32) {
            f32x4u* q = reinterpret_cast<f32x4u*>(p);
            *q = add ? *q + x : x;
        } else {
            u32x2h* q = reinterpret_cast<u32x2h*>(p);
            if (add) {
                const u32x2 o = *q;
                for (int k = 0; k < 4; ++k) {
                    const uint32_t u = o[k >> 1] >> (16 * (k & 1)) & 0xFFFF;
                    x[k] += DT == DT_BF16 ? __uint_as_float(u << 16) : half_value(u);
                }
            }
            *q = u32x2{narrow2<DT>(x[0], x[1]), narrow2<DT>(x[2], x[3])};
        }
    } else {
        for (int k = 0; k < 4; ++k)
            if (k < left) {
                if constexpr (DT == DT_F32) p[k] = add ? p[k] + x[k] : x[k];
                else {
                    if (add) x[k] += DT == DT_BF16 ? __uint_as_float((uint32_t)p[k] << 16) : half_value(p[k]);
                    p[k] = (T)narrow2<DT>(x[k], 0.f);
                }
            }
    }
}

__device__ __forceinline__ void store4(const Mul8Args& a, int64_t row, int64_t col, f32x4 x) {
    const int64_t at = row * a.c.pitch + col, left = a.n - col;
    if (a.c_type == DT_F32) store4<DT_F32>(a.c.ptr, at, left, x, a.accumulate);
    else if (a.c_type == DT_BF16) store4<DT_BF16>(a.c.ptr, at, left, x, a.accumulate);
    else store4<DT_F16>(a.c.ptr, at, left, x, a.accumulate);
}

// The exponent byte of a block of a row.
__device__ __forceinline__ int exponent(const Mat8& m, int64_t row, int64_t block) {
    return *gptr<const unsigned char>(m.scales + 4 * ((block >> 2) * m.spitch + row) + (block & 3));
}

// 32 bytes of a row: the k's from 32 (lane / 16) on of a block.
__device__ __forceinline__ i32x8 operand(const Mat8& m, int64_t row, int64_t block, int group) {
    return *gptr<const i32x8>(m.codes + row * m.pitch + block * kBlock8 + group * 32);
}

// Eight codes as bf16 values with their scale applied: exact, as bf16 has the
// exponents of fp32 and more digits than a code.
template <int FMT>
__device__ __forceinline__ bf16x8 widened(int lo, int hi, float scale) {
    bf16x2 q[4];
    if constexpr (FMT == F8_E4M3) {
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
        q[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
        q[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
        q[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    } else {
        q[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
        q[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
        q[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
        q[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
    }
    bf16x8 r;
    __builtin_memcpy(&r, q, 16);
    return r;
}

// One wave: 16 rows of A by 64 rows of B, operands straight from memory.  The
// rows of B stand as the instruction's rows, so that a lane holds four
// neighbouring columns of C.
template <int FA, int FB, bool EXACT>
__global__ __launch_bounds__(256) void k_mul8_plain(const Mul8Args a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = lane & 15, group = lane >> 4;
    const int64_t tiles_n = (a.n + 255) / 256;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * 16, n0 = (int64_t)(blockIdx.x % tiles_n) * 256 + wave * 64;
    const int64_t ra = m0 + col < a.m ? m0 + col : a.m - 1;
    int64_t rb[4];
    for (int j = 0; j < 4; ++j) rb[j] = n0 + 16 * j + col < a.n ? n0 + 16 * j + col : a.n - 1;
    f32x4 acc[4] = {};
    for (int64_t kb = 0; kb < (a.k + kBlock8 - 1) / kBlock8; ++kb) {
        const i32x8 x = operand(a.a, ra, kb, group);
        const int sx = exponent(a.a, ra, kb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const i32x8 y = operand(a.b, rb[j], kb, group);
            const int sy = exponent(a.b, rb[j], kb);
            if constexpr (EXACT) {
                const float fx = __int_as_float(sx << 23), fy = __int_as_float(sy << 23);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widened<FB>(y[2 * q], y[2 * q + 1], fy),
                                                                     widened<FA>(x[2 * q], x[2 * q + 1], fx), acc[j], 0, 0, 0);
            } else {
                acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y, x, acc[j], FB, FA, 0, sy, 0, sx);
            }
        }
    }
    if (m0 + col >= a.m) return;
    for (int j = 0; j < 4; ++j)
        if (n0 + 16 * j + group * 4 < a.n) store4(a, m0 + col, n0 + 16 * j + group * 4, acc[j]);
}

}  // namespace

Mul8Plan plan_mul8(int64_t m, int64_t n, int64_t k) { return {0, 1, (int32_t)((k + kBlock8 - 1) / kBlock8)}; }

size_t mul8_workspace(const Mul8Plan& p, int64_t m, int64_t n) { return 0; }

bool mul8_fits(const Mul8Plan& p, int64_t m, int64_t n) {
    return (double)((m + 15) / 16) * (double)((n + 255) / 256) < (double)(1 << 24);
}

hipError_t launch_mul8(const Mul8Plan& p, const Mul8Args& a, hipStream_t s) {
    const dim3 grid((uint32_t)((a.m + 15) / 16 * ((a.n + 255) / 256)));
    const bool exact = a.c_type == DT_F32;
#define M(FA, FB)                                                     \
    do {                                                              \
        if (exact) k_mul8_plain<FA, FB, true><<<grid, 256, 0, s>>>(a); \
        else k_mul8_plain<FA, FB, false><<<grid, 256, 0, s>>>(a);      \
    } while (0)
    if (a.fa == F8_E4M3 && a.fb == F8_E4M3) M(0, 0);
    else if (a.fa == F8_E4M3) M(0, 1);
    else if (a.fb == F8_E4M3) M(1, 0);
    else M(1, 1);
#undef M
    return hipGetLastError();
}

}  // namespace shampoo
