// gfx950 kernels that make and feed 8-bit matrices: quantisation of a matrix
// by its rows and by its columns, 8-bit copies of many weights, and the
// root-mean-square norm with the residual's addition and its gradient.
//
// An 8-bit matrix holds e4m3 or e5m2 codes and one power of two 2^e for each
// block of 128 values along a row: the least e >= -127 with which the block's
// largest finite value fits the format (448 = 1.75 2^8, or 57344 = 1.75 2^15).
// A power of two scales without rounding, so a value is rounded once, by the
// code (half a step: 2^-4 of the value for e4m3, 2^-3 for e5m2, unless it is
// below 2^-6 or 2^-14 of the scale); it is what the matrix instructions of
// gfx950 apply to their operands themselves; and taking it costs the block at
// most one of the format's binary orders, against a scale that maps the
// largest value to the format's end.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fp8.hpp"
#include "fp8_device.hpp"

namespace shampoo {

namespace {

// ------------------------------------------------------------ quantisation
// The byte e + 127 for a block whose largest finite magnitude has the bits
// `amax`, in a format whose largest value is 1.75 2^top: a significand above
// 1.75 carries into the exponent.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, int top) {
    const int e = (int)((amax + 0x1FFFFFu) >> 23) - top;
    return e > 0 ? (uint32_t)e : 0u;
}
// 2^-e as fp32 (e from -127 to 120).
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^e as fp32 (2^-127 is a denormal number).
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

// The bits of |x|, 0 where x is not finite.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    return u < 0x7F800000u ? u : 0u;
}

template <int FMT> constexpr int top_of() { return FMT == F8_E4M3 ? 8 : 15; }

// Four values as codes, rounded to nearest even; e4m3 has no infinity, so a
// value that is not finite becomes NaN there.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    int u = 0;
    if constexpr (FMT == F8_E4M3) {
        u = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, u, false);
        u = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, u, true);
    } else {
        u = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, u, false);
        u = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, u, true);
    }
    return (uint32_t)u;
}

// The largest of 16 neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = umax(v, moved<0xB1>(v));     // quad_perm [1,0,3,2]
    v = umax(v, moved<0x4E>(v));     // quad_perm [2,3,0,1]
    v = umax(v, moved<0x141>(v));    // the other quad of eight
    return umax(v, moved<0x140>(v)); // the other eight
}

// One 128 x 128 tile by one workgroup of 256 threads: a thread holds 8 x 8
// neighbouring values, so that both the row's codes and the column's are whole
// 8-byte words of it.  Row maxima come from the 16 lanes of a row, column
// maxima from the wave's four groups of rows and then from the four waves; the
// transpose is turned in LDS (16 KB, chunks of 8 bytes exchanged by the
// column's number so that neither side meets a bank twice) and leaves in rows
// of 128 bytes.  Values are read once whatever is written.
template <int SRC, int FR, int FC, bool ROWS, bool COLS, bool SHARED>
__device__ __forceinline__ void quantize_tile(const QuantJob& j, int64_t tr, int64_t tc) {
    __shared__ uint32_t s_max[4][128];
    __shared__ u32x2 s_turn[COLS ? 128 * 16 : 1];
    const int tid = threadIdx.x, wave = tid >> 6;
    const int cg = tid & 15, rg = tid >> 4;
    const int64_t r0 = tr * kBlock8 + rg * 8, c0 = tc * kBlock8 + cg * 8;
    const bool full = (tr + 1) * kBlock8 <= j.nrows && (tc + 1) * kBlock8 <= j.ncols;

    float v[8][8];
    if constexpr (SRC < SRC_E4M3) {
        Raw8<SRC> raw[8];
        if (full) {
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[i] = load8<SRC>(j.x.ptr, (r0 + i) * j.x.pitch + c0);
        } else {
            // one branch around all the loads of a kind, so that they are on
            // their way together; rows behind the last are that one, for nothing
            const int64_t left = j.ncols - c0;
            const auto at = [&](int i) { return (r0 + i < j.nrows ? r0 + i : j.nrows - 1) * j.x.pitch + c0; };
            if (left >= 8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) raw[i] = load8<SRC>(j.x.ptr, at(i));
            } else if (left > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) raw[i] = load8_part<SRC>(j.x.ptr, at(i), left);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) raw[i] = Raw8<SRC>{};
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) widen8<SRC>(raw[i], v[i]);
        if (!full) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i >= j.nrows) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[i][k] = 0.f;
                }
        }
    } else {
        // rows of an 8-bit matrix are whole blocks
        u32x2 raw[8];
        uint32_t byte[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = r0 + i < j.nrows;
            raw[i] = in ? *gptr<const u32x2>(j.src.codes + (r0 + i) * j.src.pitch + c0) : u32x2{0, 0};
            byte[i] = in ? *gptr<const unsigned char>(j.src.scales + 4 * ((tc >> 2) * j.src.spitch + r0 + i) + (tc & 3)) : 127u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float sc = scale_value(byte[i]);
            values4<SRC - SRC_E4M3>(raw[i].x, v[i]);
            values4<SRC - SRC_E4M3>(raw[i].y, v[i] + 4);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] *= sc;
        }
        if (!full) {   // what lies behind the last column says nothing
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c0 + k >= j.ncols) v[i][k] = 0.f;
        }
    }

    // Largest magnitudes as bits, in which whatever is not finite is larger than
    // all that is: only where one turns up are they taken again without it.
    uint32_t rmax[8], cmax[8];
    const auto largest = [&](auto finite) {
#pragma unroll
        for (int k = 0; k < 8; ++k) rmax[k] = cmax[k] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t u = decltype(finite)::value ? finite_bits(v[i][k]) : __float_as_uint(v[i][k]) & 0x7FFFFFFFu;
                if (ROWS || SHARED) rmax[i] = umax(rmax[i], u);
                if (COLS && !SHARED) cmax[k] = umax(cmax[k], u);
            }
    };
    largest(std::integral_constant<bool, false>());
    {
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) all = umax(all, ROWS || SHARED ? rmax[i] : cmax[i]);
        if (__any(all >= 0x7F800000u)) largest(std::integral_constant<bool, true>());
    }
    if constexpr (SHARED) {
        uint32_t all = rmax[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) all = umax(all, rmax[i]);
        all = max16(all);
        all = umax(all, (uint32_t)__shfl_xor((int)all, 16));
        all = umax(all, (uint32_t)__shfl_xor((int)all, 32));
        if ((tid & 63) == 0) s_max[0][wave] = all;
        __syncthreads();
        all = umax(umax(s_max[0][0], s_max[0][1]), umax(s_max[0][2], s_max[0][3]));
#pragma unroll
        for (int i = 0; i < 8; ++i) rmax[i] = cmax[i] = all;
    } else {
        if constexpr (ROWS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) rmax[i] = max16(rmax[i]);
        }
        if constexpr (COLS) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                cmax[k] = umax(cmax[k], (uint32_t)__shfl_xor((int)cmax[k], 16));
                cmax[k] = umax(cmax[k], (uint32_t)__shfl_xor((int)cmax[k], 32));
            }
            if ((tid & 63) < 16) {
#pragma unroll
                for (int k = 0; k < 8; ++k) s_max[wave][cg * 8 + k] = cmax[k];
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 8; ++k)
                cmax[k] = umax(umax(s_max[0][cg * 8 + k], s_max[1][cg * 8 + k]),
                               umax(s_max[2][cg * 8 + k], s_max[3][cg * 8 + k]));
        }
    }

    if constexpr (ROWS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t byte = scale_byte(rmax[i], top_of<FR>());
            const float inv = scale_inverse(byte);
            if (r0 + i < j.nrows) {
                u32x2 q;
                q.x = codes4<FR>(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv);
                q.y = codes4<FR>(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv);
                *gptr<u32x2>(j.rows.codes + (r0 + i) * j.rows.pitch + c0) = q;
                if (cg == 0) *gptr<unsigned char>(j.rows.scales + 4 * ((tc >> 2) * j.rows.spitch + r0 + i) + (tc & 3)) = (unsigned char)byte;
            }
        }
    }
    if constexpr (COLS) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t byte = scale_byte(cmax[k], top_of<FC>());
            const float inv = scale_inverse(byte);
            u32x2 q;
            q.x = codes4<FC>(v[0][k] * inv, v[1][k] * inv, v[2][k] * inv, v[3][k] * inv);
            q.y = codes4<FC>(v[4][k] * inv, v[5][k] * inv, v[6][k] * inv, v[7][k] * inv);
            s_turn[(cg * 8 + k) * 16 + (rg ^ cg)] = q;
            if (rg == 0 && c0 + k < j.ncols)
                *gptr<unsigned char>(j.cols.scales + 4 * ((tr >> 2) * j.cols.spitch + c0 + k) + (tr & 3)) = (unsigned char)byte;
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int c = p * 32 + (tid >> 3), k = tid & 7, turn = c >> 3;
            const u32x2 a = s_turn[c * 16 + ((2 * k) ^ turn)], b = s_turn[c * 16 + ((2 * k + 1) ^ turn)];
            if (tc * kBlock8 + c < j.ncols)
                *gptr<u32x4>(j.cols.codes + (tc * kBlock8 + c) * j.cols.pitch + tr * kBlock8 + k * 16) = u32x4{a.x, a.y, b.x, b.y};
        }
    }
}

template <int SRC, int FR, int FC, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_quantize(const QuantJob j, const uint32_t tiles_c) {
    quantize_tile<SRC, FR, FC, ROWS, COLS, false>(j, blockIdx.x / tiles_c, blockIdx.x % tiles_c);
}

// 8-bit copies of many weights and of their transposes, one scale for each
// 128 x 128 values: every tile of every matrix is one workgroup of one launch.
template <int SRC>
__global__ __launch_bounds__(256) void k_weights8(const QuantJob* __restrict__ jobs, const QuantTile* __restrict__ tiles) {
    const QuantTile t = tiles[blockIdx.x];
    const QuantJob j = jobs[t.job];
    quantize_tile<SRC, F8_E4M3, F8_E4M3, true, true, true>(j, t.row, t.col);
}

__global__ void k_weights8_bind(QuantJob* jobs, int first, int n, const AddrBatch b) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) jobs[first + i].x.ptr = b.a[i];
}

// ------------------------------------------------------------ norm
// W waves share a row; each thread holds 8 V of its values, in chunks of 8
// neighbouring ones.  V = 0: any length, the row is read a second time.
template <int W, typename T>
__device__ __forceinline__ T row_sum(T x, T (*s)[16], int wave) {
#pragma unroll
    for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
    if constexpr (W > 1) {
        const int group = wave / W;
        if ((threadIdx.x & 63) == 0) s[group][wave % W] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) x += s[group][k];
    }
    return x;
}

__device__ __forceinline__ void weight8(const void* w, int type, int64_t at, int64_t left, float (&out)[8]) {
    const uint64_t p = reinterpret_cast<uint64_t>(w);
    if (type == DT_F32) widen8<DT_F32>(load8_upto<DT_F32>(p, at, left), out);
    else if (type == DT_BF16) widen8<DT_BF16>(load8_upto<DT_BF16>(p, at, left), out);
    else widen8<DT_F16>(load8_upto<DT_F16>(p, at, left), out);
}

// h = z r w of eight values, formed in 64 bits, in 8 bits and wide; the sixteen
// lanes that hold a block of 128 are neighbours.
__device__ __forceinline__ void norm_out(const NormFwdArgs& a, int64_t row, int64_t c, const float (&z)[8], double r) {
    const int64_t left = a.dim - c;
    float h[8];
    weight8(a.w, a.w_type, c, left, h);
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = (float)((double)z[k] * r * (double)h[k]);
    if (left < 8) {   // behind the end: 0, also in a row that is not finite
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k >= left) h[k] = 0.f;
    }
    if (a.out.ptr) {
        if (a.out_type == DT_F32) store8_upto<DT_F32>(a.out.ptr, row * a.out.pitch + c, left, h);
        else if (a.out_type == DT_BF16) store8_upto<DT_BF16>(a.out.ptr, row * a.out.pitch + c, left, h);
        else store8_upto<DT_F16>(a.out.ptr, row * a.out.pitch + c, left, h);
    }
    if (a.out8.codes) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = umax(m, finite_bits(h[k]));
        m = max16(m);
        const uint32_t byte = scale_byte(m, top_of<F8_E4M3>());
        const float inv = scale_inverse(byte);
        if (c < (a.dim + kBlock8 - 1) / kBlock8 * kBlock8) {
            u32x2 q;
            q.x = codes4<F8_E4M3>(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
            q.y = codes4<F8_E4M3>(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv);
            *gptr<u32x2>(a.out8.codes + row * a.out8.pitch + c) = q;
            const int64_t b = c / kBlock8;
            if ((threadIdx.x & 15) == 0)
                *gptr<unsigned char>(a.out8.scales + 4 * ((b >> 2) * a.out8.spitch + row) + (b & 3)) = (unsigned char)byte;
        }
    }
}

// Memory bounds it: x and residual are read and z, h and r written once.  Sum,
// root and products are taken in 64 bits, which costs no time beside that (16384 x
// 1024 of bf16 with a residual in fp32: 38 us either way, 4.9 TB/s), so that a
// code is the one that the exact h has but for h itself rounded to fp32.
template <int XT, int RT, int V, int W>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void k_norm_fwd(const NormFwdArgs a) {
    constexpr int kGroups = W < 4 ? 4 / W : 1;
    constexpr bool kRes = RT >= 0;
    constexpr int ZT = kRes ? RT : XT;     // the type in which z is held
    __shared__ double s_sum[kGroups][16];
    const int wave = threadIdx.x >> 6, lane = (wave % W) * 64 + (threadIdx.x & 63);
    const int64_t want = (int64_t)blockIdx.x * kGroups + wave / W;
    const bool live = want < a.rows;
    const int64_t row = live ? want : a.rows - 1;   // every wave meets the barriers
    const int64_t xat = row * a.x.pitch, rat = row * a.res.pitch, tat = row * a.total.pitch;
    double sum = 0.0;

    auto z_of = [&](int64_t c, float (&z)[8]) {
        const int64_t left = a.dim - c;
        const auto x = load8_upto<XT>(a.x.ptr, xat + c, left);
        if constexpr (kRes) {
            const auto q = load8_upto<RT>(a.res.ptr, rat + c, left);
            float b[8];
            widen8<XT>(x, z);
            widen8<RT>(q, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] = rounded<RT>(z[k] + b[k]);
        } else {
            widen8<XT>(x, z);
        }
    };

    if constexpr (V > 0) {
        float z[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) z_of((int64_t)(v * W * 64 + lane) * 8, z[v]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t c = (int64_t)(v * W * 64 + lane) * 8;
            if (kRes && live) store8_upto<ZT>(a.total.ptr, tat + c, a.dim - c, z[v]);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fma((double)z[v][k], (double)z[v][k], sum);
        }
        sum = row_sum<W>(sum, s_sum, wave);
        const double r = 1.0 / sqrt(sum / (double)a.dim + a.eps);
        if (!live) return;
        if (lane == 0 && a.rstd) a.rstd[row] = (float)r;
#pragma unroll
        for (int v = 0; v < V; ++v) norm_out(a, row, (int64_t)(v * W * 64 + lane) * 8, z[v], r);
    } else {
        for (int64_t c = lane * 8; c < a.dim; c += W * 64 * 8) {
            float z[8];
            z_of(c, z);
            if (kRes) store8_upto<ZT>(a.total.ptr, tat + c, a.dim - c, z);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fma((double)z[k], (double)z[k], sum);
        }
        sum = row_sum<W>(sum, s_sum, wave);
        const double r = 1.0 / sqrt(sum / (double)a.dim + a.eps);
        if (lane == 0 && a.rstd) a.rstd[row] = (float)r;
        const int64_t end = (a.dim + kBlock8 - 1) / kBlock8 * kBlock8;
        for (int64_t c = lane * 8; c < end; c += W * 64 * 8) {
            float z[8];
            if constexpr (kRes) widen8<ZT>(load8_upto<ZT>(a.total.ptr, tat + c, a.dim - c), z);
            else z_of(c, z);
            norm_out(a, row, c, z, r);
        }
    }
}

// dz = r (a - x mean(a x)) + add with a = w g, x = z r, and this workgroup's
// part of dw = sum over the rows of g x.  Memory bounds it.  Groups of W waves
// take rows in turn; each thread's part of dw stays in registers over them, the
// groups' are added up in LDS in their order, and what remains, a row for each
// of at most 512 workgroups, is a sixteenth of what 8192 rows of 4096 read
// (V = 0: dw grows in that row, in memory).
constexpr int bwd_groups(int waves) { return waves < 8 ? 8 / waves : 1; }

template <int GT, int ZT, int V, int W>
__global__ __launch_bounds__(64 * W * bwd_groups(W)) void k_norm_bwd(const NormBwdArgs a) {
    constexpr int kGroups = bwd_groups(W);
    __shared__ float s_sum[2][kGroups][16];
    __shared__ float s_dw[V > 0 && kGroups > 1 ? V * W * 512 : 1];
    const int wave = threadIdx.x >> 6, lane = (wave % W) * 64 + (threadIdx.x & 63), mine = wave / W;
    const int64_t group = (int64_t)blockIdx.x * kGroups + mine, groups = (int64_t)a.slots * kGroups;
    const int64_t turns = (a.rows + groups - 1) / groups;
    const uint64_t partial = reinterpret_cast<uint64_t>(a.partials) + (uint64_t)blockIdx.x * (uint64_t)a.dim * 4;
    const float inv_dim = 1.f / (float)a.dim;
    float dw[V > 0 ? V : 1][8] = {};
    int phase = 0;
    for (int64_t t = 0; t < turns; ++t, phase ^= 1) {
        const int64_t want = t * groups + group;
        const bool live = want < a.rows;
        const int64_t row = live ? want : a.rows - 1;
        const int64_t gat = row * a.g.pitch, zat = row * a.z.pitch, aat = row * a.add.pitch, dat = row * a.dz.pitch;
        const float r = live ? a.rstd[row] : 0.f;   // a row that is not there adds 0 to dw
        float dot = 0.f;
        if constexpr (V > 0) {
            float g[V][8], x[V][8], add[V][8] = {};
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = (int64_t)(v * W * 64 + lane) * 8, left = live ? a.dim - c : 0;
                widen8<GT>(load8_upto<GT>(a.g.ptr, gat + c, left), g[v]);
                widen8<ZT>(load8_upto<ZT>(a.z.ptr, zat + c, left), x[v]);
                if (a.add.ptr) widen8<ZT>(load8_upto<ZT>(a.add.ptr, aat + c, left), add[v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int64_t c = (int64_t)(v * W * 64 + lane) * 8;
                float w[8];
                weight8(a.w, a.w_type, c, a.dim - c, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[v][k] *= r;
                    dw[v][k] = fmaf(g[v][k], x[v][k], dw[v][k]);
                    g[v][k] *= w[k];
                    dot = fmaf(g[v][k], x[v][k], dot);
                }
            }
            dot = row_sum<W>(dot, s_sum[phase], wave) * inv_dim;
            if (live) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int64_t c = (int64_t)(v * W * 64 + lane) * 8;
#pragma unroll
                    for (int k = 0; k < 8; ++k) add[v][k] += r * (g[v][k] - x[v][k] * dot);
                    store8_upto<ZT>(a.dz.ptr, dat + c, a.dim - c, add[v]);
                }
            }
        } else {
            for (int64_t c = lane * 8; c < a.dim; c += W * 64 * 8) {
                const int64_t left = live ? a.dim - c : 0;
                float g[8], x[8], w[8];
                widen8<GT>(load8_upto<GT>(a.g.ptr, gat + c, left), g);
                widen8<ZT>(load8_upto<ZT>(a.z.ptr, zat + c, left), x);
                weight8(a.w, a.w_type, c, a.dim - c, w);
                float part[8] = {};
                if (t && a.dw) widen8<DT_F32>(load8_upto<DT_F32>(partial, c, a.dim - c), part);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[k] *= r;
                    part[k] = fmaf(g[k], x[k], part[k]);
                    dot = fmaf(g[k] * w[k], x[k], dot);
                }
                if (a.dw) store8_upto<DT_F32>(partial, c, a.dim - c, part);
            }
            dot = row_sum<W>(dot, s_sum[phase], wave) * inv_dim;
            if (live) {
                for (int64_t c = lane * 8; c < a.dim; c += W * 64 * 8) {
                    const int64_t left = a.dim - c;
                    float g[8], x[8], w[8], add[8] = {};
                    widen8<GT>(load8_upto<GT>(a.g.ptr, gat + c, left), g);
                    widen8<ZT>(load8_upto<ZT>(a.z.ptr, zat + c, left), x);
                    weight8(a.w, a.w_type, c, left, w);
                    if (a.add.ptr) widen8<ZT>(load8_upto<ZT>(a.add.ptr, aat + c, left), add);
#pragma unroll
                    for (int k = 0; k < 8; ++k) add[k] += r * (g[k] * w[k] - (x[k] * r) * dot);
                    store8_upto<ZT>(a.dz.ptr, dat + c, left, add);
                }
            }
        }
    }
    if constexpr (V > 0) {
        if (a.dw) {
            for (int q = 0; q < kGroups; ++q) {
                if (mine == q) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int c = (v * W * 64 + lane) * 8;
                        if constexpr (kGroups > 1) {
                            float* p = s_dw + c;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                if (q) dw[v][k] += p[k];
                                if (q + 1 < kGroups) p[k] = dw[v][k];
                            }
                        }
                        if (q + 1 == kGroups) store8_upto<DT_F32>(partial, c, a.dim - c, dw[v]);
                    }
                }
                if constexpr (kGroups > 1) __syncthreads();
            }
        }
    }
}

// dw: the slots' sums, in the order of the slots; 32 columns and 32 runs of
// slots to a workgroup, which takes further columns where a row has more than
// kDwGroups of them (a launch of 2^32 threads or more would wrap).
constexpr int64_t kDwGroups = 1 << 20;
__global__ __launch_bounds__(1024) void k_norm_dw(const NormBwdArgs a) {
    __shared__ float s[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int per = (a.slots + 31) / 32, from = y * per, to = from + per < a.slots ? from + per : a.slots;
    for (int64_t first = (int64_t)blockIdx.x * 32; first < a.dim; first += kDwGroups * 32) {
        const int64_t c = first + x;
        float sum = 0.f;
        if (c < a.dim) {
            const float* p = a.partials + c;
            int i = from;
            for (; i + 8 <= to; i += 8) {       // eight loads on their way together
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = p[(int64_t)(i + k) * a.dim];
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += v[k];
            }
            for (; i < to; ++i) sum += p[(int64_t)i * a.dim];
        }
        s[y][x] = sum;
        __syncthreads();
        if (y == 0 && c < a.dim) {
#pragma unroll
            for (int k = 1; k < 32; ++k) sum += s[k][x];
            a.dw[c] = a.accumulate ? a.dw[c] + sum : sum;
        }
        if (first + kDwGroups * 32 < a.dim) __syncthreads();     // s has been read
    }
}

// How many waves share a row, and the eights of each thread: for rows up to
// 16384 long every value stays in a register.
struct RowShape {
    int waves, chunks;
};
RowShape row_shape(int64_t dim) {
    if (dim <= 512) return {1, 1};
    if (dim <= 1024) return {1, 2};
    if (dim <= 2048) return {2, 2};
    if (dim <= 4096) return {4, 2};
    if (dim <= 8192) return {8, 2};
    if (dim <= 16384) return {16, 2};
    return {16, 0};
}
int groups_of(const RowShape& s) { return s.waves < 4 ? 4 / s.waves : 1; }

}  // namespace

hipError_t launch_quantize(int src, int fr, int fc, const QuantJob& j, hipStream_t s) {
    const uint32_t tc = (uint32_t)((j.ncols + kBlock8 - 1) / kBlock8);
    const uint32_t tr = (uint32_t)((j.nrows + kBlock8 - 1) / kBlock8);
    const dim3 grid(tc * tr);
    const bool rows = j.rows.codes != 0, cols = j.cols.codes != 0;
#define Q(SRC, FR, FC, R, C) k_quantize<SRC, FR, FC, R, C><<<grid, 256, 0, s>>>(j, tc)
#define Q_SIDES(SRC)                                                     \
    do {                                                                 \
        if (rows && cols) {                                              \
            if (fr == F8_E4M3) {                                         \
                if (fc == F8_E4M3) Q(SRC, F8_E4M3, F8_E4M3, true, true); \
                else Q(SRC, F8_E4M3, F8_E5M2, true, true);               \
            } else {                                                     \
                if (fc == F8_E4M3) Q(SRC, F8_E5M2, F8_E4M3, true, true); \
                else Q(SRC, F8_E5M2, F8_E5M2, true, true);               \
            }                                                            \
        } else if (rows) {                                               \
            if (fr == F8_E4M3) Q(SRC, F8_E4M3, F8_E4M3, true, false);    \
            else Q(SRC, F8_E5M2, F8_E5M2, true, false);                  \
        } else {                                                         \
            if (fc == F8_E4M3) Q(SRC, F8_E4M3, F8_E4M3, false, true);    \
            else Q(SRC, F8_E5M2, F8_E5M2, false, true);                  \
        }                                                                \
    } while (0)
#define Q_TURN(SRC)                                                      \
    do {                                                                 \
        if (fc == F8_E4M3) Q(SRC, F8_E4M3, F8_E4M3, false, true);        \
        else Q(SRC, F8_E5M2, F8_E5M2, false, true);                      \
    } while (0)
    switch (src) {
    case DT_F32: Q_SIDES(DT_F32); break;
    case DT_BF16: Q_SIDES(DT_BF16); break;
    case DT_F16: Q_SIDES(DT_F16); break;
    case SRC_E4M3: Q_TURN(SRC_E4M3); break;
    default: Q_TURN(SRC_E5M2); break;
    }
#undef Q_TURN
#undef Q_SIDES
#undef Q
    return hipGetLastError();
}

hipError_t launch_weights8(int src, const QuantJob* jobs, const QuantTile* tiles, int ntiles, hipStream_t s) {
    if (src == DT_F32) k_weights8<DT_F32><<<ntiles, 256, 0, s>>>(jobs, tiles);
    else if (src == DT_BF16) k_weights8<DT_BF16><<<ntiles, 256, 0, s>>>(jobs, tiles);
    else k_weights8<DT_F16><<<ntiles, 256, 0, s>>>(jobs, tiles);
    return hipGetLastError();
}

hipError_t launch_weights8_bind(QuantJob* jobs, int first, int n, const AddrBatch& b, hipStream_t s) {
    k_weights8_bind<<<(n + 63) / 64, 64, 0, s>>>(jobs, first, n, b);
    return hipGetLastError();
}

namespace {

template <int XT, int RT>
void norm_fwd(const NormFwdArgs& a, hipStream_t s) {
    const RowShape sh = row_shape(a.dim);
    const int64_t g = groups_of(sh);
    const dim3 grid((uint32_t)((a.rows + g - 1) / g));
#define N(V, W) k_norm_fwd<XT, RT, V, W><<<grid, W < 4 ? 256 : 64 * W, 0, s>>>(a)
    if (sh.chunks == 0) N(0, 16);
    else if (sh.waves == 1 && sh.chunks == 1) N(1, 1);
    else if (sh.waves == 1) N(2, 1);
    else if (sh.waves == 2) N(2, 2);
    else if (sh.waves == 4) N(2, 4);
    else if (sh.waves == 8) N(2, 8);
    else N(2, 16);
#undef N
}
template <int XT>
void norm_fwd(int rt, const NormFwdArgs& a, hipStream_t s) {
    if (rt < 0) norm_fwd<XT, -1>(a, s);
    else if (rt == DT_F32) norm_fwd<XT, DT_F32>(a, s);
    else if (rt == DT_BF16) norm_fwd<XT, DT_BF16>(a, s);
    else norm_fwd<XT, DT_F16>(a, s);
}

template <int GT, int ZT>
void norm_bwd(const NormBwdArgs& a, hipStream_t s) {
    const RowShape sh = row_shape(a.dim);
    const dim3 grid(a.slots);
#define N(V, W) k_norm_bwd<GT, ZT, V, W><<<grid, 64 * W * bwd_groups(W), 0, s>>>(a)
    if (sh.chunks == 0) N(0, 16);
    else if (sh.waves == 1 && sh.chunks == 1) N(1, 1);
    else if (sh.waves == 1) N(2, 1);
    else if (sh.waves == 2) N(2, 2);
    else if (sh.waves == 4) N(2, 4);
    else if (sh.waves == 8) N(2, 8);
    else N(2, 16);
#undef N
}
template <int GT>
void norm_bwd(int zt, const NormBwdArgs& a, hipStream_t s) {
    if (zt == DT_F32) norm_bwd<GT, DT_F32>(a, s);
    else if (zt == DT_BF16) norm_bwd<GT, DT_BF16>(a, s);
    else norm_bwd<GT, DT_F16>(a, s);
}

}  // namespace

bool norm_fwd_fits(int64_t rows, int64_t dim) {
    const RowShape sh = row_shape(dim);
    const int64_t g = groups_of(sh), threads = 64 * sh.waves * g;
    return (rows + g - 1) / g < ((int64_t)1 << 32) / threads;
}

hipError_t launch_norm_fwd(int xt, int rt, const NormFwdArgs& a, hipStream_t s) {
    if (xt == DT_F32) norm_fwd<DT_F32>(rt, a, s);
    else if (xt == DT_BF16) norm_fwd<DT_BF16>(rt, a, s);
    else norm_fwd<DT_F16>(rt, a, s);
    return hipGetLastError();
}

// Workgroups of the gradient, each of which leaves a row of partial sums.
int norm_bwd_slots(int64_t rows, int64_t dim) {
    const int g = bwd_groups(row_shape(dim).waves);
    const int64_t want = (rows + g - 1) / g;
    return (int)(want < 512 ? want : 512);
}

hipError_t launch_norm_bwd(int gt, int zt, const NormBwdArgs& a, hipStream_t s) {
    if (a.rows) {
        if (gt == DT_F32) norm_bwd<DT_F32>(zt, a, s);
        else if (gt == DT_BF16) norm_bwd<DT_BF16>(zt, a, s);
        else norm_bwd<DT_F16>(zt, a, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.dw) return e;
    const int64_t groups = (a.dim + 31) / 32;
    k_norm_dw<<<(uint32_t)(groups < kDwGroups ? groups : kDwGroups), 1024, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace shampoo
