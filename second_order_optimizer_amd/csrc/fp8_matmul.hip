// gfx950 kernels of the product of 8-bit matrices, C = A B^T (+ C), with a
// scale for each block of 128 of a row.
//
// Two ways to the sum, by the type of C.  bf16 and fp16: the matrix
// instructions that take 8-bit operands and a power of two for each 32 of them.
// They add products in eights, each cut off below 2^-13 of the largest, and
// those sums in fp32 (found by products of single powers of two): on normally
// distributed values 1.5e-5 of the result, with one column in a hundred
// twentyfold 4.4e-5, a fiftieth of what rounding to bf16 leaves; where large
// products cancel it is more of what is left.  fp32: the codes are widened to
// bf16 with their scale, exactly between 2^-126 and 2^128, and multiplied by the
// bf16 instructions, whose sums are those of fp32 (6e-8 at K = 2048, 2e-7 at
// 16384), at half the rate: a weight's gradient that is added up over
// micro-batches keeps its small terms.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "fp8.hpp"
#include "fp8_device.hpp"

namespace shampoo {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum : int { MUL8_FEW = 0, MUL8_64 = 1, MUL8_128 = 2, MUL8_256 = 3 };
constexpr int64_t kFewRows = 64;

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
// exponents of fp32 and more digits than a code, but for values below 2^-126,
// which may become 0, and of 2^128 or more, which become infinite.  The
// instruction reads the scale's exponent alone: 0 is 2^-127.
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

// Few rows of A (a token, a small batch): 16 rows of B and up to 16 MT of A to a
// workgroup whose W waves share out the blocks of k, U neighbouring ones at a
// time, with operands straight from memory; the waves' sums are joined in LDS in
// their order.  Reading B bounds it, so what counts is how many of its bytes are
// on their way at once (1 x 8192 x 8192: 13.7 us, 4.9 TB/s, against 19.4 by tiles of
// 64 x 64; 1 x 4096 x 1024: 3.1 us, latency; 64 x 4096 x 1024: 5.7 us against 6.5, but
// 13.7 against 11.3 over 4096, where every workgroup reads all of A; each pair on
// one card, on another 12.2 us, 3.2 and 4.8, and 10.3 by tiles).  The rows of B
// stand as the instruction's rows, so that a lane holds four neighbouring columns
// of C.
template <int MT, int W, int U, int FA, int FB, bool EXACT>
__global__ __launch_bounds__(64 * W) void k_mul8_few(const Mul8Args a) {
    __shared__ f32x4 s_sum[W][MT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, group = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int nkb = (int)((a.k + kBlock8 - 1) / kBlock8);
    const int64_t rb = n0 + col < a.n ? n0 + col : a.n - 1;
    int64_t ra[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ra[i] = 16 * i + col < a.m ? 16 * i + col : a.m - 1;
    f32x4 acc[MT] = {};
    for (int kb = wave * U; kb < nkb; kb += W * U) {
        i32x8 y[U], x[U][MT];
        int ey[U], ex[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = kb + u < nkb ? kb + u : nkb - 1;    // behind the end the last one again, for nothing
            y[u] = operand(a.b, rb, k, group);
            ey[u] = exponent(a.b, rb, k);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                x[u][i] = operand(a.a, ra[i], k, group);
                ex[u][i] = exponent(a.a, ra[i], k);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb + u < nkb) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    if constexpr (EXACT) {
                        const float fx = __int_as_float(ex[u][i] << 23), fy = __int_as_float(ey[u] << 23);
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widened<FB>(y[u][2 * q], y[u][2 * q + 1], fy),
                                                                             widened<FA>(x[u][i][2 * q], x[u][i][2 * q + 1], fx), acc[i], 0, 0, 0);
                    } else {
                        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(y[u], x[u][i], acc[i], FB, FA, 0, ey[u], 0, ex[u][i]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) s_sum[wave][i][lane] = acc[i];
    __syncthreads();
    for (int i = wave; i < MT; i += W) {
        f32x4 sum = s_sum[0][i][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += s_sum[w][i][lane];
        if (16 * i + col < a.m && n0 + group * 4 < a.n) store4(a, 16 * i + col, n0 + group * 4, sum);
    }
}

// A value that all lanes share, in scalar registers.
__device__ __forceinline__ uint64_t uniform(uint64_t x) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x) | (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32;
}

// 16 bytes of each lane from memory into LDS, without registers between: to
// `lds` (the wave's, in bytes) + 16 lane, from `base` + `off`.  Written out so
// that the reads of one stage do not wait for the loads of the next; the wait
// is stage_ready's.  A memory instruction must not read a scalar register within
// five wait states of the vector instruction that wrote it (v_readfirstlane of
// `uniform`, v_readlane of a spill): the hardware does not wait, and the compiler
// does not look in here.  So the load reads a copy that a scalar instruction
// made, for which the hardware does; the copy is the wait that m0 needs as well
// (8192^3: 381 us, with s_nop 4 in its place 391).  m0 is a register that the
// compiler reserves and may be told of, with a warning: nothing that it writes
// itself in these kernels uses m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(uint32_t lds, uint64_t base, uint32_t off) {
    uint64_t from;
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0" : "=&s"(from) : "s"(lds), "v"(off), "s"(uniform(base)) : "memory", "m0");
}
__device__ __forceinline__ void dma4(uint32_t lds, uint64_t base, uint32_t off) {   // 4 bytes of each lane
    uint64_t from;
    asm volatile("s_mov_b32 m0, %1\n\ts_mov_b64 %0, %3\n\tglobal_load_lds_dword %2, %0" : "=&s"(from) : "s"(lds), "v"(off), "s"(uniform(base)) : "memory", "m0");
}
#pragma clang diagnostic pop
// Every load of this wave but the last N has arrived, its reads too, and so
// have those of the workgroup's other waves.
template <int N>
__device__ __forceinline__ void stage_ready() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroups of one XCD (every eighth) take neighbouring tiles, four rows
// of tiles deep, so that what they read together stays in its L2.
struct Tile {
    int64_t m, n;
    int32_t split;
};
__device__ __forceinline__ Tile tile_of(uint32_t id, uint32_t count, uint32_t tiles_m, uint32_t tiles_n) {
    const uint32_t xcd = id % 8, q = count / 8, r = count % 8;
    uint32_t t = xcd * q + (xcd < r ? xcd : r) + id / 8;
    const uint32_t split = t / (tiles_m * tiles_n);
    t -= split * tiles_m * tiles_n;
    const uint32_t deep = 4 * tiles_n, band = t / deep, in = t % deep;
    const uint32_t rows = tiles_m - band * 4 < 4 ? tiles_m - band * 4 : 4;
    return Tile{(int64_t)(band * 4 + in % rows), (int64_t)(in / rows), (int32_t)split};
}

// Rows of C from a wave's own piece of LDS, WIDTH values in fp32 each, WIDTH + 4
// apart: whole rows of eights of neighbouring lanes, where the accumulators'
// own order would give every row 32 bytes at a time (256 x 256 tiles: 26 us
// against 5 for the end of a tile).
template <int DT, int WIDTH, int ROWS>
__device__ __forceinline__ void store_rows(uint64_t base, int64_t pitch, int64_t m, int64_t n, bool add, const float* piece, int64_t r0, int64_t c0) {
    constexpr int kLanes = WIDTH / 8, kTurn = 64 / kLanes;
    const int lane = threadIdx.x & 63;
    const int64_t c = c0 + lane % kLanes * 8, left = n - c;
#pragma unroll
    for (int p = 0; p < ROWS; p += kTurn) {
        const int i = p + lane / kLanes;
        const float* v = piece + i * (WIDTH + 4) + lane % kLanes * 8;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(v), hi = *reinterpret_cast<const f32x4*>(v + 4);
        float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if (i < ROWS && r0 + i < m && left > 0) {
            const int64_t at = (r0 + i) * pitch + c;
            if (add) {
                float old[8];
                widen8<DT>(load8_upto<DT>(base, at, left), old);
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] += old[k];
            }
            store8_upto<DT>(base, at, left, x);
        }
    }
}
template <bool EXACT, int WIDTH, int ROWS>
__device__ __forceinline__ void store_rows(const Mul8Args& a, int split, const float* piece, int64_t r0, int64_t c0) {
    if (a.partials) {
        store_rows<DT_F32, WIDTH, ROWS>(reinterpret_cast<uint64_t>(a.partials + (int64_t)split * a.m * a.n), a.n, a.m, a.n, false, piece, r0, c0);
    } else if constexpr (EXACT) {
        store_rows<DT_F32, WIDTH, ROWS>(a.c.ptr, a.c.pitch, a.m, a.n, a.accumulate, piece, r0, c0);
    } else {
        if (a.c_type == DT_BF16) store_rows<DT_BF16, WIDTH, ROWS>(a.c.ptr, a.c.pitch, a.m, a.n, a.accumulate, piece, r0, c0);
        else store_rows<DT_F16, WIDTH, ROWS>(a.c.ptr, a.c.pitch, a.m, a.n, a.accumulate, piece, r0, c0);
    }
}

// f(0), f(1), ... with numbers that the compiler knows.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void for_each(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        for_each<N, I + 1>(f);
    }
}

// A tile of BM x BN of C by WM x WN waves.  Blocks of 128 k of both operands go
// through STAGES buffers in LDS, loaded past the registers while the blocks
// before them are multiplied.  A row's 128 bytes lie as eight chunks of 16 in an
// order that its number permutes (chunk c at c ^ (row / 2)), with which neither
// 16 nor 32 rows' reads meet a bank twice (4.3 cycles a wave, 8 in order of the
// row's number itself); the loads permute their source addresses, as LDS is
// filled in the order of the lanes.  Which k of a block a lane takes does not
// matter, as long as both operands agree: it has one scale.  128 x 128 by four
// waves (two workgroups on a CU), and 256 x 256 by eight for fp32 results: 773 us
// at 8192^3, 1.42 PFLOP/s, the library's bf16 product 765.
template <int BM, int BN, int WM, int WN, int FA, int FB, bool EXACT>
__global__ __launch_bounds__(64 * WM * WN) void k_mul8_tile(const Mul8Args a, const uint32_t tiles_m, const uint32_t tiles_n) {
    constexpr int kWaves = WM * WN, STAGES = 2;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;      // 32 x 32 pieces of a wave
    constexpr int LA = BM / 8 / kWaves, LB = BN / 8 / kWaves; // loads of a wave for a stage
    constexpr uint32_t kStage = (BM + BN) * kBlock8;
    static_assert(LA * 8 * kWaves == BM && LB * 8 * kWaves == BN && TM * 32 * WM == BM && TN * 32 * WN == BN, "whole loads");
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const Tile t = tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n);
    const int64_t m0 = t.m * BM, n0 = t.n * BN;
    const int64_t all = (a.k + kBlock8 - 1) / kBlock8;
    const int64_t kb0 = (int64_t)t.split * a.blocks_per_split;
    const int nkb = (int)(all - kb0 < a.blocks_per_split ? all - kb0 : a.blocks_per_split);

    // sources of this wave's loads: byte offsets from the tile's first row
    uint32_t offa[LA], offb[LB];
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = (wave * LA + i) * 8 + (lane >> 3);
        const int64_t row = m0 + r < a.m ? r : a.m - 1 - m0;
        offa[i] = (uint32_t)(row * a.a.pitch) + 16 * ((lane & 7) ^ (r >> 1 & 7));
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int r = (wave * LB + i) * 8 + (lane >> 3);
        const int64_t row = n0 + r < a.n ? r : a.n - 1 - n0;
        offb[i] = (uint32_t)(row * a.b.pitch) + 16 * ((lane & 7) ^ (r >> 1 & 7));
    }
    uint64_t basea = a.a.codes + (uint64_t)(m0 * a.a.pitch + kb0 * kBlock8), baseb = a.b.codes + (uint64_t)(n0 * a.b.pitch + kb0 * kBlock8);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    // block kb, or the last one again: without a condition the loop below is one
    // piece that is scheduled as a whole
    const auto load_one = [&](int stage, auto which) {
        constexpr int I = decltype(which)::value;
        if constexpr (I < LA) dma16(lds0 + stage * kStage + (wave * LA + I) * 1024, basea, offa[I]);
        else dma16(lds0 + stage * kStage + BM * kBlock8 + (wave * LB + I - LA) * 1024, baseb, offb[I - LA]);
    };
    const auto advance = [&](int kb) {    // behind the loads of block kb
        const uint32_t step = kb + 1 < nkb ? kBlock8 : 0;
        basea += step;
        baseb += step;
    };

    // this lane's rows, and its chunks in them: of half h of a block those at
    // 2 h + (lane / 32) and 4 further
    const int row = lane & 31, half = lane >> 5;
    const uint32_t turn = row >> 1 & 7;
    uint32_t chunk[2];
    for (int h = 0; h < 2; ++h) chunk[h] = 16 * ((2 * h + half) ^ turn);
    const uint32_t ra = (wm * TM * 32 + row) * kBlock8, rb = BM * kBlock8 + (wn * TN * 32 + row) * kBlock8;

    // scales: words of four blocks, of A's rows and then of B's, 64 rows to a
    // wave (some of them twice where there are more waves)
    constexpr int kWordLoads = (BM + BN) / 64, LW = (kWordLoads + kWaves - 1) / kWaves;
    uint32_t woff[LW];
    uint64_t wbase[LW];
    int64_t wpitch[LW];
    int wpart[LW];
#pragma unroll
    for (int i = 0; i < LW; ++i) {
        wpart[i] = (wave * LW + i) % kWordLoads;
        const bool of_a = wpart[i] < BM / 64;
        const int64_t first = of_a ? m0 : n0, last = (of_a ? a.m : a.n) - 1;
        const int64_t r = first + (of_a ? wpart[i] : wpart[i] - BM / 64) * 64 + lane;
        woff[i] = 4 * (uint32_t)((r < last ? r : last) - first);
        wpitch[i] = 4 * (of_a ? a.a.spitch : a.b.spitch);
        wbase[i] = (of_a ? a.a.scales : a.b.scales) + 4 * (uint64_t)first + (uint64_t)(kb0 / 4 * wpitch[i]);   // parts begin at whole groups
    }
    const auto words = [&](int group, bool on) {
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            dma4(lds0 + STAGES * kStage + ((group & 1) * (BM + BN) + wpart[i] * 64) * 4, wbase[i], woff[i]);
            wbase[i] += wpitch[i] & -(int64_t)(on & (4 * (group + 1) < nkb));
        }
    };
    int wa[TM], wb[TN];      // exponent bytes of this lane's rows in the block at hand

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;

    // a block is 2 TM steps, one for each half and each 32 rows of A; their
    // operands are read R - 1 steps ahead, B's a half ahead
    constexpr int kSteps = 2 * TM, R = TM < 4 ? 2 : 4;
    static_assert(kSteps % R == 0 && R <= TM + 1, "slots that the compiler knows; B's first half has been multiplied when the next block's is read");
    i32x8 x[R], y[2][TN];
    const auto operand_at = [&](const char* p, uint32_t rows, uint32_t c) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(p + rows + c);
        const i32x4 hi = *reinterpret_cast<const i32x4*>(p + rows + (c ^ 64));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    const auto read_x = [&](int stage, auto step) {
        constexpr int S = decltype(step)::value;
        x[S % R] = operand_at(lds + stage * kStage, ra + (S % TM) * 32 * kBlock8, chunk[S / TM]);
    };
    const auto read_y = [&](int stage, auto half_no) {
        constexpr int H = decltype(half_no)::value;
#pragma unroll
        for (int j = 0; j < TN; ++j) y[H][j] = operand_at(lds + stage * kStage, rb + j * 32 * kBlock8, chunk[H]);
    };
    const auto multiply = [&](auto step) {
        constexpr int S = decltype(step)::value, H = S / TM, i = S % TM;
        if constexpr (EXACT) {
            const float fx = __int_as_float(wa[i] << 23);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bf16x8 xw = widened<FA>(x[S % R][2 * u], x[S % R][2 * u + 1], fx);
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const float fy = __int_as_float(wb[j] << 23);
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widened<FB>(y[H][j][2 * u], y[H][j][2 * u + 1], fy), xw, acc[i][j], 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(y[H][j], x[S % R], acc[i][j], FB, FA, 0, wb[j], 0, wa[i]);
        }
    };
    const auto scales = [&](int kb, int (&va)[TM], int (&vb)[TN]) {
        const unsigned char* w = reinterpret_cast<const unsigned char*>(lds) + STAGES * kStage + (kb >> 2 & 1) * (BM + BN) * 4 + (kb & 3);
#pragma unroll
        for (int i = 0; i < TM; ++i) va[i] = w[4 * ((wm * TM + i) * 32 + row)];
#pragma unroll
        for (int j = 0; j < TN; ++j) vb[j] = w[4 * (BM + (wn * TN + j) * 32 + row)];
    };
    typedef std::integral_constant<int, 0> First;
    typedef std::integral_constant<int, 1> Second;

    if (nkb > 0) {
        words(0, true);
        for_each<STAGES>([&](auto n) {
            for_each<LA + LB>([&](auto which) { load_one(decltype(n)::value, which); });
            advance(decltype(n)::value);
        });
        stage_ready<(STAGES - 1) * (LA + LB)>();
        scales(0, wa, wb);
        read_y(0, First());
        for_each<R - 1>([&](auto step) { read_x(0, step); });
        int stage = 0;
        // In front of the step whose reads begin the next block, the waves agree
        // that this stage has been read and that the next has arrived; what is
        // left of this block is multiplied while the next one's first operands
        // come.  (Behind the last block they read what lies there.)
        for (int kb = 0; kb < nkb; ++kb) {
            int na[TM], nb[TN], free_stage = 0;
            for_each<kSteps>([&](auto step) {
                constexpr int S = decltype(step)::value;
                if constexpr (S == 0) read_y(stage, Second());
                if constexpr (S + R - 1 == kSteps) {
                    stage_ready<0>();
                    words(((kb + 1) >> 2) + 1, (kb + 1 & 3) == 3);
                    free_stage = stage;
                    stage = stage + 1 == STAGES ? 0 : stage + 1;
                    scales(kb + 1, na, nb);
                    read_y(stage, First());
                }
                if constexpr (S + R - 1 < kSteps) read_x(stage, std::integral_constant<int, S + R - 1>());
                else read_x(stage, std::integral_constant<int, S + R - 1 - kSteps>());
                multiply(step);
                if constexpr (S + R > kSteps) {     // the freed stage is filled, some loads behind each step
                    constexpr int kTurn = S + R - 1 - kSteps, kPer = (LA + LB + R - 2) / (R - 1);
                    for_each<kPer>([&](auto n) {
                        constexpr int I = kTurn * kPer + decltype(n)::value;
                        if constexpr (I < LA + LB) load_one(free_stage, std::integral_constant<int, I>());
                    });
                    if constexpr (S + 1 == kSteps) advance(kb + STAGES);
                }
                __builtin_amdgcn_sched_barrier(0);   // reads stay where they are: brought forward, they cost registers
            });
#pragma unroll
            for (int i = 0; i < TM; ++i) wa[i] = na[i];
#pragma unroll
            for (int j = 0; j < TN; ++j) wb[j] = nb[j];
        }
        stage_ready<0>();    // no load is left to a workgroup that comes after
    }

    // C, 32 rows of it at a time; a lane holds four times four neighbouring
    // columns of one row
    constexpr int kWidth = TN * 32, kPiece = 32 * (kWidth + 4);
    static_assert(kWaves * kPiece * 4 <= (int)(STAGES * kStage), "a piece of LDS for each wave");
    float* piece = reinterpret_cast<float*>(lds) + wave * kPiece;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(piece + row * (kWidth + 4) + j * 32 + 8 * q + 4 * half) =
                    f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        __builtin_amdgcn_wave_barrier();
        store_rows<EXACT, kWidth, 32>(a, t.split, piece, m0 + (wm * TM + i) * 32, n0 + wn * kWidth);
        __builtin_amdgcn_wave_barrier();
    }
}

// acc += P Q with their scales, acc staying in its accumulator registers: the
// builtin's result may be put elsewhere, and where every accumulator register is
// taken that means copies.  What reads acc after it waits for itself
// (products_done); operands come from LDS, whose reads the compiler waits for.
template <int FP, int FQ>
__device__ __forceinline__ void multiply_here(f32x4& acc, const i32x8& p, const i32x8& q, int sp, int sq) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:%5 blgp:%6"
                 : "+a"(acc)
                 : "v"(p), "v"(q), "v"(sp), "v"(sq), "n"(FP), "n"(FQ));
}
// Every product that was issued has been written (a 16 x 16 x 128 one takes
// eight passes of four cycles).
__device__ __forceinline__ void products_done() { asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" ::: "memory"); }

// The same for tiles of 256 x 256 by four waves, one to a SIMD, each with 128 x
// 128 of C in 256 accumulator registers: a third fewer bytes from LDS for a
// product than with eight waves.  Nothing else runs on the SIMD, so the wave
// itself keeps the matrix unit fed: a block is multiplied in four quarters, each
// half of A's rows by half of B's, and behind each product one piece of the next
// quarters' operands is read.  An even block goes through (A0, B0), (A0, B1),
// (A1, B1), (A1, B0), an odd one through (A0, B1), (A0, B0), (A1, B0), (A1, B1):
// so each half is free before its next values come, and the operands of one block
// are all that is held.  The halves that a block takes first and those that it
// takes later are freed and loaded half a block apart, so the loads are spread
// evenly and have a whole block's time (2048 cycles) to arrive at least.  8192^3:
// 380 to 400 us by the card, 2.8 PFLOP/s, the matrix unit busy 70 % of the 1.9 to
// 2.1 GHz that random codes leave.  On a card where it took 370, `k_mul8_tile`
// with eight waves took 428, and codes of 0, which take less power, 288.
template <int FA, int FB>
__global__ __launch_bounds__(256) void k_mul8_big(const Mul8Args a, const uint32_t tiles_m, const uint32_t tiles_n) {
    constexpr int BM = 256, BN = 256, L = 4;                 // loads of a wave for half a stage's A or B
    constexpr uint32_t kStage = (BM + BN) * kBlock8, kWords = 2 * kStage;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const Tile t = tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n);
    const int64_t m0 = t.m * BM, n0 = t.n * BN;
    const int64_t all = (a.k + kBlock8 - 1) / kBlock8;
    const int64_t kb0 = (int64_t)t.split * a.blocks_per_split;
    const int nkb = (int)(all - kb0 < a.blocks_per_split ? all - kb0 : a.blocks_per_split);

    // half h of an operand: rows 64 h to 64 h + 63 of either 128
    const auto tile_row = [&](int half, int i) { return (wave >> 1) * 128 + half * 64 + (wave & 1) * 32 + i * 8; };
    uint32_t offa[2][L], offb[2][L];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int r = tile_row(h, i) + (lane >> 3);
            const uint32_t chunk = 16 * ((lane & 7) ^ (r >> 1 & 7));
            offa[h][i] = (uint32_t)((m0 + r < a.m ? r : a.m - 1 - m0) * a.a.pitch) + chunk;
            offb[h][i] = (uint32_t)((n0 + r < a.n ? r : a.n - 1 - n0) * a.b.pitch) + chunk;
        }
    uint64_t basea = a.a.codes + (uint64_t)(m0 * a.a.pitch + kb0 * kBlock8), baseb = a.b.codes + (uint64_t)(n0 * a.b.pitch + kb0 * kBlock8);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    // loads 0 to 3 of half HA of A, 4 to 7 of half HB of B
    const auto load_one = [&](int stage, auto half_a, auto half_b, auto which) {
        constexpr int HA = decltype(half_a)::value, HB = decltype(half_b)::value, I = decltype(which)::value;
        if constexpr (I < L) dma16(lds0 + stage * kStage + tile_row(HA, I) * kBlock8, basea, offa[HA][I]);
        else dma16(lds0 + stage * kStage + (BM + tile_row(HB, I - L)) * kBlock8, baseb, offb[HB][I - L]);
    };
    const auto advance = [&](int kb) {    // behind the loads of block kb; the last one is loaded again behind the end
        const uint32_t step = kb + 1 < nkb ? kBlock8 : 0;
        basea += step;
        baseb += step;
    };
    // scale words: waves 0 and 1 those of A's rows, 2 and 3 of B's, 128 rows each
    const int64_t wfirst = wave < 2 ? m0 : n0, wlast = (wave < 2 ? a.m : a.n) - 1, wpitch = 4 * (wave < 2 ? a.a.spitch : a.b.spitch);
    uint64_t wbase = (wave < 2 ? a.a.scales : a.b.scales) + 4 * (uint64_t)wfirst + (uint64_t)(kb0 / 4 * wpitch);
    uint32_t woff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t r = wfirst + (wave & 1) * 128 + i * 64 + lane;
        woff[i] = 4 * (uint32_t)((r < wlast ? r : wlast) - wfirst);
    }
    const auto words = [&](int group, bool on) {
#pragma unroll
        for (int i = 0; i < 2; ++i) dma4(lds0 + kWords + ((group & 1) * (BM + BN) + wave * 128 + i * 64) * 4, wbase, woff[i]);
        wbase += wpitch & -(int64_t)(on & (4 * (group + 1) < nkb));
    };

    const int row = lane & 15, group = lane >> 4;
    const uint32_t c0 = 16 * (group ^ (row >> 1));           // chunks group and group + 4
    const uint32_t ra = (wm * 128 + row) * kBlock8 + c0, rb = BM * kBlock8 + (wn * 128 + row) * kBlock8 + c0;
    const uint32_t swa = kWords + 4 * (wm * 128 + row), swb = kWords + 4 * (BM + wn * 128 + row);

    i32x8 x[8], y[8];
    int ex[8], ey[8];
    f32x4 acc[8][8];
    for_each<64>([&](auto n) {
        f32x4& c = acc[decltype(n)::value / 8][decltype(n)::value % 8];
        c = f32x4{0.f, 0.f, 0.f, 0.f};
        asm volatile("" : "+a"(c));
    });

    const auto operand_at = [&](uint32_t at) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + at), hi = *reinterpret_cast<const i32x4*>(lds + (at ^ 64));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    // piece P of eight of the operands of half H: an operand, or a scale
    const auto read_a = [&](int kb, auto half_no, auto piece) {
        constexpr int P = decltype(piece)::value, I = 4 * decltype(half_no)::value + P / 2;
        if constexpr (P % 2 == 0) x[I] = operand_at((kb & 1) * kStage + ra + I * 16 * kBlock8);
        else ex[I] = *reinterpret_cast<const unsigned char*>(lds + (kb >> 2 & 1) * (BM + BN) * 4 + (kb & 3) + swa + I * 64);
    };
    const auto read_b = [&](int kb, auto half_no, auto piece) {
        constexpr int P = decltype(piece)::value, I = 4 * decltype(half_no)::value + P / 2;
        if constexpr (P % 2 == 0) y[I] = operand_at((kb & 1) * kStage + rb + I * 16 * kBlock8);
        else ey[I] = *reinterpret_cast<const unsigned char*>(lds + (kb >> 2 & 1) * (BM + BN) * 4 + (kb & 3) + swb + I * 64);
    };
    // a quarter: sixteen products, act(0) to act(15) between them
    const auto quarter = [&](auto half_a, auto half_b, auto&& act) {
        constexpr int HA = 4 * decltype(half_a)::value, HB = 4 * decltype(half_b)::value;
        for_each<16>([&](auto n) {
            constexpr int I = decltype(n)::value / 4, J = decltype(n)::value % 4;
            multiply_here<FB, FA>(acc[HA + I][HB + J], y[HB + J], x[HA + I], ey[HB + J], ex[HA + I]);
            act(n);
            __builtin_amdgcn_sched_barrier(0);   // in this order
        });
    };
    typedef std::integral_constant<int, 0> Zero;
    typedef std::integral_constant<int, 1> One;
    // act(n) of a quarter: eight pieces read, then loads FIRST to FIRST + 3
    const auto between = [](auto n, auto first, auto&& read, auto&& load) {
        constexpr int N = decltype(n)::value, F = decltype(first)::value;
        if constexpr (N < 8) read(n);
        else if constexpr (N % 2 == 0) load(std::integral_constant<int, F + (N - 8) / 2>());
    };
    typedef std::integral_constant<int, 4> Four;
    // block kb, with P and Q the halves of B in the order of this block
    const auto block = [&](int kb, auto P, auto Q) {
        const auto early = [&](auto which) { load_one(kb & 1, Zero(), P, which); };    // of block kb + 2
        const auto late = [&](auto which) { load_one(kb & 1, One(), Q, which); };
        // this block's later halves have arrived, its first ones have been read;
        // behind them 16 loads are on their way
        stage_ready<4 * L>();
        quarter(Zero(), P, [&](auto n) { between(n, Zero(), [&](auto piece) { read_b(kb, Q, piece); }, early); });
        quarter(Zero(), Q, [&](auto n) { between(n, Four(), [&](auto piece) { read_a(kb, One(), piece); }, early); });
        // the next block's first halves have arrived, this one's later ones have been read
        stage_ready<4 * L>();
        words(((kb + 1) >> 2) + 1, (kb + 1 & 3) == 3);
        quarter(One(), Q, [&](auto n) { between(n, Zero(), [&](auto piece) { read_a(kb + 1, Zero(), piece); }, late); });
        quarter(One(), P, [&](auto n) { between(n, Four(), [&](auto piece) { read_b(kb + 1, Q, piece); }, late); });
        advance(kb + 2);
    };

    if (nkb > 0) {
        words(0, true);
        const auto fill = [&](auto stage, auto half_b) {
            for_each<2 * L>([&](auto which) { load_one(decltype(stage)::value, Zero(), half_b, which); });
            for_each<2 * L>([&](auto which) { load_one(decltype(stage)::value, One(), std::integral_constant<int, 1 - decltype(half_b)::value>(), which); });
            advance(decltype(stage)::value);
        };
        fill(Zero(), Zero());
        fill(One(), One());
        stage_ready<6 * L>();
        for_each<8>([&](auto piece) {
            read_a(0, Zero(), piece);
            read_b(0, Zero(), piece);
        });
        int kb = 0;
        for (; kb + 1 < nkb; kb += 2) {
            block(kb, Zero(), One());
            block(kb + 1, One(), Zero());
        }
        if (kb < nkb) block(kb, Zero(), One());
        stage_ready<0>();    // no load is left to a workgroup that comes after
    }
    products_done();
    for_each<64>([&](auto n) {
        f32x4& c = acc[decltype(n)::value / 8][decltype(n)::value % 8];
        asm volatile("" : "+a"(c));
    });

    constexpr int kWidth = 128, kPiece = 16 * (kWidth + 4);
    float* piece = reinterpret_cast<float*>(lds) + wave * 2 * kPiece;
    for_each<8>([&](auto in) {
        constexpr int I = decltype(in)::value;
        float* p = piece + (I & 1) * kPiece;
        for_each<8>([&](auto jn) {
            constexpr int J = decltype(jn)::value;
            *reinterpret_cast<f32x4*>(p + row * (kWidth + 4) + J * 16 + 4 * group) = acc[I][J];
        });
        __builtin_amdgcn_wave_barrier();
        store_rows<false, kWidth, 16>(a, t.split, p, m0 + wm * 128 + I * 16, n0 + wn * 128);
        __builtin_amdgcn_wave_barrier();
    });
}

// Tiles of 64 x 64 by eight waves, for products of few tiles, where the time is
// that of one block after another: two waves share 32 x 32 of C, each taking one
// half of every block, and join their sums in LDS; four stages, three of them on
// their way.  777 x 1000 x 2048: 9.9 us in fp32, 7.3 in bf16, against 11.3 and 7.6
// where one wave took both halves; eight stages, or two blocks between barriers,
// made no difference.
template <int FA, int FB, bool EXACT>
__global__ __launch_bounds__(512) void k_mul8_small(const Mul8Args a, const uint32_t tiles_m, const uint32_t tiles_n) {
    constexpr int BM = 64, BN = 64, STAGES = 4;
    constexpr uint32_t kStage = (BM + BN) * kBlock8, kWords = STAGES * kStage;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1 & 1, mine = wave >> 2;      // mine: the half of a block
    const Tile t = tile_of(blockIdx.x, gridDim.x, tiles_m, tiles_n);
    const int64_t m0 = t.m * BM, n0 = t.n * BN;
    const int64_t all = (a.k + kBlock8 - 1) / kBlock8;
    const int64_t kb0 = (int64_t)t.split * a.blocks_per_split;
    const int nkb = (int)(all - kb0 < a.blocks_per_split ? all - kb0 : a.blocks_per_split);

    // each wave loads eight rows of A and eight of B
    const int lr = wave * 8 + (lane >> 3);
    const uint32_t lc = 16 * ((lane & 7) ^ (lr >> 1 & 7));
    const uint32_t offa = (uint32_t)((m0 + lr < a.m ? lr : a.m - 1 - m0) * a.a.pitch) + lc;
    const uint32_t offb = (uint32_t)((n0 + lr < a.n ? lr : a.n - 1 - n0) * a.b.pitch) + lc;
    uint64_t basea = a.a.codes + (uint64_t)(m0 * a.a.pitch + kb0 * kBlock8), baseb = a.b.codes + (uint64_t)(n0 * a.b.pitch + kb0 * kBlock8);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
    const auto load = [&](int stage, int kb) {     // block kb, or the last one again
        dma16(lds0 + stage * kStage + wave * 1024, basea, offa);
        dma16(lds0 + stage * kStage + BM * kBlock8 + wave * 1024, baseb, offb);
        const uint32_t step = kb + 1 < nkb ? kBlock8 : 0;
        basea += step;
        baseb += step;
    };
    // scale words: the even waves those of A's rows, the odd ones of B's
    const int of_b = wave & 1;
    const int64_t wfirst = of_b ? n0 : m0, wlast = (of_b ? a.n : a.m) - 1, wpitch = 4 * (of_b ? a.b.spitch : a.a.spitch);
    uint64_t wbase = (of_b ? a.b.scales : a.a.scales) + 4 * (uint64_t)wfirst + (uint64_t)(kb0 / 4 * wpitch);
    const uint32_t woff = 4 * (uint32_t)((wfirst + lane < wlast ? wfirst + lane : wlast) - wfirst);
    const auto words = [&](int group, bool on) {
        dma4(lds0 + kWords + ((group & 1) * (BM + BN) + of_b * 64) * 4, wbase, woff);
        wbase += wpitch & -(int64_t)(on & (4 * (group + 1) < nkb));
    };

    const int row = lane & 31, half = lane >> 5;
    const uint32_t chunk = 16 * ((2 * mine + half) ^ (row >> 1 & 7));
    const uint32_t ra = (wm * 32 + row) * kBlock8 + chunk, rb = (BM + wn * 32 + row) * kBlock8 + chunk;
    const auto operand_at = [&](uint32_t at) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + at), hi = *reinterpret_cast<const i32x4*>(lds + (at ^ 64));
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    f32x16 acc;
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;

    if (nkb > 0) {
        words(0, true);
        for (int s = 0; s < STAGES - 1; ++s) load(s, s);
        for (int kb = 0; kb < nkb; ++kb) {
            const int stage = kb % STAGES;
            // this block has arrived, the one before it has been read
            stage_ready<2 * (STAGES - 2)>();
            if ((kb & 3) == 0) words((kb >> 2) + 1, true);
            load((kb + STAGES - 1) % STAGES, kb + STAGES - 1);
            const unsigned char* w = reinterpret_cast<const unsigned char*>(lds) + kWords + (kb >> 2 & 1) * (BM + BN) * 4 + (kb & 3);
            const int ex = w[4 * (wm * 32 + row)], ey = w[4 * (BM + wn * 32 + row)];
            const i32x8 x = operand_at(stage * kStage + ra), y = operand_at(stage * kStage + rb);
            if constexpr (EXACT) {
                const float fx = __int_as_float(ex << 23), fy = __int_as_float(ey << 23);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widened<FB>(y[2 * u], y[2 * u + 1], fy), widened<FA>(x[2 * u], x[2 * u + 1], fx), acc, 0, 0, 0);
            } else {
                acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(y, x, acc, FB, FA, 0, ey, 0, ex);
            }
        }
        stage_ready<0>();    // no load is left, to these waves or to a workgroup that comes after
    }

    // the second halves' sums, then C by the waves of the first
    f32x4* joined = reinterpret_cast<f32x4*>(lds + 2 * kStage) + (wave & 3) * 256 + lane;
    if (mine) {
#pragma unroll
        for (int q = 0; q < 4; ++q) joined[q * 64] = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
    }
    __syncthreads();
    if (mine) return;
    constexpr int kPiece = 32 * 36;
    static_assert(4 * kPiece * 4 <= (int)(2 * kStage), "a piece of LDS for each wave in front of the sums");
    float* piece = reinterpret_cast<float*>(lds) + wave * kPiece;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(piece + row * 36 + 8 * q + 4 * half) = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]} + joined[q * 64];
    __builtin_amdgcn_wave_barrier();
    store_rows<EXACT, 32, 32>(a, t.split, piece, m0 + wm * 32, n0 + wn * 32);
}

// C from the parts' sums, in the order of the parts.
__global__ __launch_bounds__(256) void k_mul8_join(const Mul8Args a) {
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, per = (a.n + 3) / 4 * 4;
    const int64_t r = at / per, c = at % per;
    if (r >= a.m) return;
    f32x4 sum = {};
    for (int s = 0; s < a.splits; ++s) {
        const float* p = a.partials + ((int64_t)s * a.m + r) * a.n + c;
        if (c + 4 <= a.n) sum += *reinterpret_cast<const f32x4u*>(p);
        else
            for (int k = 0; k < 4; ++k) sum[k] += c + k < a.n ? p[k] : 0.f;
    }
    store4(a, r, c, sum);
}

template <int BM, int BN, int WM, int WN, int FA, int FB, bool EXACT>
hipError_t launch_tile(const Mul8Args& a, hipStream_t s) {
    const uint32_t tm = (uint32_t)((a.m + BM - 1) / BM), tn = (uint32_t)((a.n + BN - 1) / BN);
    constexpr int bytes = 2 * (BM + BN) * kBlock8 + 2 * (BM + BN) * 4;
    const auto k = k_mul8_tile<BM, BN, WM, WN, FA, FB, EXACT>;
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    k<<<tm * tn * a.splits, 64 * WM * WN, bytes, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <int FA, int FB>
hipError_t launch_big(const Mul8Args& a, hipStream_t s) {
    const uint32_t tm = (uint32_t)((a.m + 255) / 256), tn = (uint32_t)((a.n + 255) / 256);
    constexpr int bytes = 2 * 512 * kBlock8 + 2 * 512 * 4;
    const auto k = k_mul8_big<FA, FB>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    k<<<tm * tn * a.splits, 256, bytes, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <int FA, int FB, bool EXACT>
hipError_t launch_small(const Mul8Args& a, hipStream_t s) {
    const uint32_t tm = (uint32_t)((a.m + 63) / 64), tn = (uint32_t)((a.n + 63) / 64);
    constexpr int bytes = 4 * 128 * kBlock8 + 2 * 128 * 4;
    const auto k = k_mul8_small<FA, FB, EXACT>;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    k<<<tm * tn * a.splits, 512, bytes, s>>>(a, tm, tn);
    return hipGetLastError();
}

template <int MT, int FA, int FB, bool EXACT>
hipError_t launch_few(const Mul8Args& a, hipStream_t s) {
    const uint32_t grid = (uint32_t)((a.n + 15) / 16);
    const int64_t nkb = (a.k + kBlock8 - 1) / kBlock8;
    if constexpr (MT > 1) {      // short sums only (plan_mul8)
        k_mul8_few<MT, 4, 2, FA, FB, EXACT><<<grid, 256, 0, s>>>(a);
    } else {
        if (nkb <= 8) k_mul8_few<1, 4, 2, FA, FB, EXACT><<<grid, 256, 0, s>>>(a);
        else if (nkb <= 32) k_mul8_few<1, 8, 2, FA, FB, EXACT><<<grid, 512, 0, s>>>(a);
        else k_mul8_few<1, 8, 4, FA, FB, EXACT><<<grid, 512, 0, s>>>(a);
    }
    return hipGetLastError();
}

template <int FA, int FB, bool EXACT>
hipError_t launch_kind(int kind, const Mul8Args& a, hipStream_t s) {
    switch (kind) {
    case MUL8_FEW:
        if (a.m <= 16) return launch_few<1, FA, FB, EXACT>(a, s);
        if (a.m <= 32) return launch_few<2, FA, FB, EXACT>(a, s);
        return launch_few<4, FA, FB, EXACT>(a, s);
    case MUL8_64: return launch_small<FA, FB, EXACT>(a, s);
    case MUL8_128: return launch_tile<128, 128, 2, 2, FA, FB, EXACT>(a, s);
    default:
        if constexpr (EXACT) return launch_tile<256, 256, 2, 4, FA, FB, EXACT>(a, s);
        else return launch_big<FA, FB>(a, s);
    }
}

}  // namespace

// What one block of k costs a tile, in us, by the way of the sum: with one
// workgroup on a CU, and with as many as fit (two of the smaller tiles); and what
// a tile costs besides (first loads, storing).  From 8192^3 (370 us with 256 x
// 256, 539 with 128 x 128, 921 with 64 x 64; fp32: 759, 842, 1380) and from tiles
// that are alone: 777 x 1000 x 2048 in 7.5 and 14 us with 64 and 128 (fp32: 11, 18),
// 1024 x 1024 x 8192 in fp32 in 33, 56 and 133, and with 128 in four parts in 29.
// In between the table is short: 10.5 us for 2048^3 (16.6 measured), 15.8 for
// 4096 x 4096 x 1024 (24.8), 6.9 for 64 x 4096 x 4096 (10.3), all in bf16.
struct TileCost {
    int size, resident;
    double alone[2], full[2], fixed;   // [0]: bf16 and fp16, [1]: fp32
};
constexpr TileCost kTileCosts[] = {
    {64, 2, {0.17, 0.40}, {0.45, 0.70}, 1.5},
    {128, 2, {0.50, 0.92}, {1.02, 1.60}, 2.5},
    {256, 1, {1.22, 2.75}, {1.22, 2.75}, 6.0},
};

Mul8Plan plan_mul8(int64_t m, int64_t n, int64_t k, int type) {
    const int64_t nkb = (k + kBlock8 - 1) / kBlock8;
    const int exact = type == DT_F32;
    Mul8Plan best{MUL8_FEW, 1, (int32_t)nkb};
    if (m <= 16 || (m <= kFewRows && nkb <= 8)) return best;
    double least = 1e300;
    for (int kind = MUL8_64; kind <= MUL8_256; ++kind) {
        const TileCost& c = kTileCosts[kind - MUL8_64];
        const double tiles = std::ceil((double)m / c.size) * std::ceil((double)n / c.size);
        for (int64_t want = 1; want <= 32 && (want == 1 || 8 * want <= nkb); want *= 2) {
            const int64_t per = want == 1 ? nkb : ((nkb + want - 1) / want + 3) / 4 * 4;    // whole groups of scales
            const int64_t parts = nkb ? (nkb + per - 1) / per : 1;
            const double groups = tiles * (double)parts;
            const bool alone = groups <= 256;
            const double rounds = alone ? 1.0 : std::ceil(groups / (256.0 * c.resident));
            double us = rounds * (c.fixed + (double)per * (alone ? c.alone : c.full)[exact]);
            if (parts > 1) us += 4.0 + (double)m * (double)n * (8.0 * (double)parts) / 8e6;   // its launch; the parts written and read
            if (us < least) {
                least = us;
                best = Mul8Plan{kind, (int32_t)parts, (int32_t)per};
            }
        }
    }
    return best;
}

size_t mul8_workspace(const Mul8Plan& p, int64_t m, int64_t n) {
    return p.splits > 1 ? (size_t)p.splits * (size_t)m * (size_t)n * 4 : 0;
}

bool mul8_fits(const Mul8Plan& p, int64_t m, int64_t n) {
    const int64_t t = p.kind == MUL8_FEW ? 16 : kTileCosts[p.kind - MUL8_64].size, tm = p.kind == MUL8_FEW ? 1 : (m + t - 1) / t;
    return (double)tm * (double)((n + t - 1) / t) * p.splits < (double)(1 << 22);
}

hipError_t launch_mul8(const Mul8Plan& p, const Mul8Args& in, hipStream_t s) {
    Mul8Args a = in;
    if (p.splits <= 1) a.partials = nullptr;
    const bool exact = a.c_type == DT_F32;
    hipError_t e;
#define M(FA, FB) e = exact ? launch_kind<FA, FB, true>(p.kind, a, s) : launch_kind<FA, FB, false>(p.kind, a, s)
    if (a.fa == F8_E4M3 && a.fb == F8_E4M3) M(F8_E4M3, F8_E4M3);
    else if (a.fa == F8_E4M3) M(F8_E4M3, F8_E5M2);
    else if (a.fb == F8_E4M3) M(F8_E5M2, F8_E4M3);
    else M(F8_E5M2, F8_E5M2);
#undef M
    if (e != hipSuccess || !a.partials) return e;
    k_mul8_join<<<(uint32_t)((a.m * ((a.n + 3) / 4) + 255) / 256), 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace shampoo
