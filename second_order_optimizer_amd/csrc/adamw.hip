// gfx950 kernels of the first-order operators: one AdamW step over many
// tensors (moments in fp32 or in 8 bits) and the global gradient norm.
//
// Per element, in fp32, every operation rounded on its own (no contraction,
// IEEE division and root), so that a result does not depend on which wave,
// vector or tail handled its element:
//   x = coef g;  m = b1 m + (1 - b1) x;  v = b2 v + (1 - b2) x^2
//   p = p - (a p + b m / (sqrt(v) c + eps))
// with a = lr lr_scale weight_decay, b = lr lr_scale / (1 - b1^t) and
// c = 1 / sqrt(1 - b2^t) formed in fp64 and rounded once.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "adamw.hpp"

#pragma clang fp contract(off)

namespace shampoo {

namespace {

// Vectors that are aligned like their elements: a caller's tensor may start
// anywhere (gfx950 loads and stores 16 bytes at any address).
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned short u16x8u __attribute__((ext_vector_type(8), aligned(2)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

// A caller's pointer through the global address space (global, not flat,
// memory instructions).
template <typename T>
__device__ __forceinline__ T* gptr(uint64_t addr) {
    typedef __attribute__((address_space(1))) T gT;
    return (T*)reinterpret_cast<gT*>(addr);
}

template <int DT> struct Store { typedef unsigned short type; typedef u16x4u vec; };
template <> struct Store<DT_F32> { typedef float type; typedef f32x4u vec; };

__device__ __forceinline__ float widen(unsigned short u, int dt) {
    if (dt == DT_BF16) return __uint_as_float((uint32_t)u << 16);
    _Float16 h;
    __builtin_memcpy(&h, &u, 2);
    return (float)h;
}

// Four consecutive elements from `first` of a tensor of `numel`, as fp32;
// past the end 0.
template <int DT>
__device__ __forceinline__ f32x4 load4(uint64_t base, int64_t first, int64_t numel) {
    typedef typename Store<DT>::type T;
    typedef typename Store<DT>::vec V;
    const T* q = gptr<const T>(base) + first;
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (first + 4 <= numel) {
        const V u = *gptr<const V>((uint64_t)q);
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == DT_F32) r[k] = u[k];
            else r[k] = widen(u[k], DT);
        }
    } else {
        for (int k = 0; k < 4; ++k)
            if (first + k < numel) {
                if constexpr (DT == DT_F32) r[k] = q[k];
                else r[k] = widen(q[k], DT);
            }
    }
    return r;
}

template <typename T, typename V, typename W>
__device__ __forceinline__ void store4(uint64_t base, int64_t first, int64_t numel, const W& w) {
    T* q = gptr<T>(base) + first;
    if (first + 4 <= numel) {
        V u;
        for (int k = 0; k < 4; ++k) u[k] = (T)w[k];
        *gptr<V>((uint64_t)q) = u;
    } else {
        for (int k = 0; k < 4; ++k)
            if (first + k < numel) q[k] = (T)w[k];
    }
}

// The largest of the 32 lanes of a half wave, in each of them.
__device__ __forceinline__ uint32_t half_max(uint32_t v) {
    for (int o = 16; o > 0; o >>= 1) {
        const uint32_t w = (uint32_t)__shfl_xor((int)v, o, 64);
        v = v > w ? v : w;
    }
    return v;
}

// Scale of a run from the largest magnitude among its finite values, and the
// factor that takes values to e4m3's range (up to 448).  The floor keeps the
// factor finite; values below it are kept as they fall under that scale.
__device__ __forceinline__ void run_scale(uint32_t amax_bits, float& scale, float& inv) {
    scale = fmaxf(__uint_as_float(amax_bits), 0x1p-110f) * (1.0f / 448);
    inv = 1.0f / scale;
}

constexpr uint32_t kFinite = 0x7F7FFFFFu;

// One value as an e4m3 code (without sign): y = |x| inv in [0, 448].  Rounded
// up with the probability of the fraction that e4m3 drops (r: 16 random bits
// shifted to the top of the 20 mantissa bits that it drops), so that moving
// averages whose change in one step is less than half a code still move.
// Below 2^-6 e4m3 steps evenly, as it does in [2^-6, 2^-5): adding 2^-6 puts
// those values there.  A value that is not finite becomes NaN.
template <bool POSITIVE>
__device__ __forceinline__ uint32_t encode(float x, float inv, uint32_t r) {
    const float y = fabsf(x) * inv;
    const bool small = y < 0x1p-6f;
    const uint32_t b = __float_as_uint(small ? y + 0x1p-6f : y);
    uint32_t c = ((b + r) >> 20) - (small ? 968u : 960u);
    c = c < 126u ? c : 126u;
    // a positive root never becomes 0, whose division would be by eps alone
    if (POSITIVE) {
        if (x > 0.f && c == 0u) c = 1u;
    }
    if ((__float_as_uint(x) & 0x7FFFFFFFu) > kFinite) c = 127u;
    if (!POSITIVE) c |= (__float_as_uint(x) >> 24) & 128u;
    return c;
}

__device__ __forceinline__ f32x4 decode4(uint32_t w) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return f32x4{lo.x, lo.y, hi.x, hi.y};
}

// One step of the elements of this wave's tiles.  Half a wave takes a run of
// 256 elements: lane l the elements 4l.. and 128 + 4l.., so that every load
// and store of the half covers whole 128-byte lines.
template <int P, int G, bool S8>
__global__ __launch_bounds__(256) void k_adamw(AdamwArgs a) {
    const AdamwClock clk = a.clocks[blockIdx.x];
    float coef = 1.f;
    if (a.clip) {
        if (a.clip->nonfinite) return;   // the same for every workgroup: nothing changes
        coef = a.clip->coef;
    }
    __syncthreads();   // every wave has read the clock
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    const int lane = threadIdx.x & 63, l = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const uint32_t key0 = mix32(a.seed_mixed + (uint32_t)(clk.t + 1));
    for (int i = wave; i < a.ntiles; i += gridDim.x * 4) {
        const AdamwTile tl = a.tiles[i];
        const AdamwTensor ts = a.tensors[tl.tensor];
        if (!ts.g_ptr) continue;
        const float fa = (float)(lr * ts.lr_scale * ts.weight_decay);
        const float fb = (float)(lr * ts.lr_scale * clk.inv1);
        const uint32_t key1 = mix32(key0 + (uint32_t)ts.id);
        for (int k = lane >> 5; k < tl.nruns; k += 2) {
            const int64_t run = tl.run0 + k;
            const int64_t st = (ts.state_run + run) * kRun;
            f32x4 p[2], m[2], v[2], g[2];
            i16x4 rem[2];
            float ms = 0.f, ss = 0.f;
            if constexpr (S8) {
                ms = a.m_scale[ts.state_run + run];
                ss = a.s_scale[ts.state_run + run];
            }
            for (int j = 0; j < 2; ++j) {
                const int o = 128 * j + 4 * l;
                const int64_t e = run * kRun + o;
                g[j] = load4<G>(ts.g_ptr, e, ts.numel);
                p[j] = load4<P>(ts.p_ptr, e, ts.numel);
                if constexpr (P == DT_BF16)
                    rem[j] = *reinterpret_cast<const i16x4*>(a.rem + (ts.rem_run + run) * kRun + o);
                if constexpr (S8) {
                    m[j] = decode4(*reinterpret_cast<const uint32_t*>(a.m8 + st + o));
                    v[j] = decode4(*reinterpret_cast<const uint32_t*>(a.s8 + st + o));
                } else {
                    m[j] = *reinterpret_cast<const f32x4*>(a.m + st + o);
                    v[j] = *reinterpret_cast<const f32x4*>(a.v + st + o);
                }
            }
            uint32_t mmax = 0, smax = 0;
            for (int j = 0; j < 2; ++j)
                for (int q = 0; q < 4; ++q) {
                    const float x = g[j][q] * coef;
                    float m0 = m[j][q], v0 = v[j][q];
                    if constexpr (S8) {
                        m0 = m0 * ms;
                        v0 = v0 * ss;
                        v0 = v0 * v0;
                    }
                    const float m1 = m0 * a.b1 + x * a.c1;
                    const float v1 = v0 * a.b2 + (x * x) * a.c2;
                    const float root = sqrtf(v1);
                    const float d = root * clk.inv_root2 + a.eps;
                    float w = p[j][q];
                    if constexpr (P == DT_BF16)
                        w = __uint_as_float(__float_as_uint(w) + (uint32_t)(int)rem[j][q]);
                    w = w - (w * fa + (m1 / d) * fb);
                    p[j][q] = w;
                    m[j][q] = m1;
                    v[j][q] = S8 ? root : v1;
                    if constexpr (S8) {
                        const uint32_t mb = __float_as_uint(m1) & 0x7FFFFFFFu;
                        const uint32_t sb = __float_as_uint(root) & 0x7FFFFFFFu;
                        if (mb <= kFinite) mmax = mmax > mb ? mmax : mb;
                        if (sb <= kFinite) smax = smax > sb ? smax : sb;
                    }
                }
            float mi = 0.f, si = 0.f;
            if constexpr (S8) {
                run_scale(half_max(mmax), ms, mi);
                run_scale(half_max(smax), ss, si);
                if (l == 0) {
                    a.m_scale[ts.state_run + run] = ms;
                    a.s_scale[ts.state_run + run] = ss;
                }
            }
            for (int j = 0; j < 2; ++j) {
                const int o = 128 * j + 4 * l;
                const int64_t e = run * kRun + o;
                if constexpr (P == DT_BF16) {
                    u16x4 hi;
                    for (int q = 0; q < 4; ++q) {
                        // nearest bf16 (ties away from zero); what is left fits 16 bits
                        const uint32_t b = __float_as_uint(p[j][q]);
                        const uint32_t h = (b + 0x8000u) >> 16;
                        const bool nan = (b & 0x7FFFFFFFu) > 0x7F800000u;
                        hi[q] = nan ? (unsigned short)0x7FC0 : (unsigned short)h;
                        rem[j][q] = nan ? (short)0 : (short)(b - (h << 16));
                    }
                    store4<unsigned short, u16x4u>(ts.p_ptr, e, ts.numel, hi);
                    *reinterpret_cast<i16x4*>(a.rem + (ts.rem_run + run) * kRun + o) = rem[j];
                } else {
                    store4<float, f32x4u>(ts.p_ptr, e, ts.numel, p[j]);
                }
                if constexpr (S8) {
                    uint32_t mw = 0, sw = 0;
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t key = key1 + (uint32_t)((uint64_t)e >> 32) * 0x85157AF5u;
                        const uint32_t h = mix32(key ^ ((uint32_t)e + q));
                        mw |= encode<false>(m[j][q], mi, (h & 0xFFFFu) << 4) << (8 * q);
                        sw |= encode<true>(v[j][q], si, (h >> 16) << 4) << (8 * q);
                    }
                    *reinterpret_cast<uint32_t*>(a.m8 + st + o) = mw;
                    *reinterpret_cast<uint32_t*>(a.s8 + st + o) = sw;
                } else {
                    *reinterpret_cast<f32x4*>(a.m + st + o) = m[j];
                    *reinterpret_cast<f32x4*>(a.v + st + o) = v[j];
                }
            }
        }
    }
    if (threadIdx.x == 0) {
        AdamwClock n = clk;
        n.t += 1;
        n.b1t *= a.beta1;
        n.b2t *= a.beta2;
        n.inv1 = 1.0 / (1.0 - n.b1t);
        n.inv_root2 = (float)(1.0 / sqrt(1.0 - n.b2t));
        a.clocks[blockIdx.x] = n;
    }
}

__global__ __launch_bounds__(256) void k_adamw_clock(AdamwClock* clocks, int n, AdamwClock c) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) clocks[i] = c;
}

// The pointers travel as kernel arguments, so that a captured graph holds
// them and nothing on the host has to outlive the call.
__global__ __launch_bounds__(256) void k_adamw_bind(AdamwTensor* tensors, int n, PtrBatch b,
                                                   int which) {
    const int i = threadIdx.x;
    if (i >= n) return;
    if (which & 1) tensors[i].p_ptr = b.a[i];
    if (which & 2) tensors[i].g_ptr = b.b[i];
}

__global__ __launch_bounds__(256) void k_norm_bind(NormTensor* tensors, int n, PtrBatch b) {
    const int i = threadIdx.x;
    if (i >= n) return;
    tensors[i].g_ptr = b.a[i];
    tensors[i].out_ptr = b.b[i];
}

// ------------------------------------------------------------ gradient norm
__device__ __forceinline__ double wave_sum_d(double v) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ double group_sum(double v, double* red) {
    v = wave_sum_d(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

template <int DT>
__device__ __forceinline__ double tile_squares(uint64_t g, int64_t first, int64_t numel, int lane) {
    double s[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < kNormTile / 256; ++k) {
        const f32x4 x = load4<DT>(g, first + k * 256 + lane * 4, numel);
        for (int q = 0; q < 4; ++q) s[q] += (double)x[q] * (double)x[q];
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum of the squares of every gradient in fp64 (the squares of fp32 values
// are exact in it, none overflows), in an order that the plan fixes: each
// wave over its tiles, each workgroup over its waves, the last workgroup to
// finish over the workgroups' sums.
__global__ __launch_bounds__(256) void k_norm(NormArgs a) {
    __shared__ double red[4];
    __shared__ int last;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    double acc = 0.0;
    for (int i = wave; i < a.ntiles; i += gridDim.x * 4) {
        const NormTile tl = a.tiles[i];
        const NormTensor ts = a.tensors[tl.tensor];
        if (!ts.g_ptr) continue;
        if (ts.dtype == DT_F32) acc += tile_squares<DT_F32>(ts.g_ptr, tl.first, ts.numel, lane);
        else if (ts.dtype == DT_BF16) acc += tile_squares<DT_BF16>(ts.g_ptr, tl.first, ts.numel, lane);
        else acc += tile_squares<DT_F16>(ts.g_ptr, tl.first, ts.numel, lane);
    }
    const double sum = group_sum(acc, red);
    if (threadIdx.x == 0) {
        __hip_atomic_store(a.partials + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(a.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    double t = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 256)
        t += __hip_atomic_load(a.partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    t = group_sum(t, red);
    if (threadIdx.x == 0) {
        const double n = sqrt(t) * a.grad_scale;
        const bool finite = n <= 1.7976931348623157e308;   // not infinite, not NaN
        const double c = n > a.max_norm ? a.max_norm / n : 1.0;
        ClipRecord r;
        r.norm = (float)n;
        r.coef = finite ? (float)(c * a.grad_scale) : 0.f;
        r.nonfinite = finite ? 0 : 1;
        r.pad_ = 0;
        *a.record = r;
        *a.ticket = 0;   // for the next launch
    }
}

template <int DT>
__device__ __forceinline__ void tile_clip(const NormTensor& ts, int64_t first, int lane, float coef,
                                          bool zero) {
#pragma unroll
    for (int k = 0; k < kNormTile / 256; ++k) {
        const int64_t e = first + k * 256 + lane * 4;
        f32x4 x = load4<DT>(ts.g_ptr, e, ts.numel);
        for (int q = 0; q < 4; ++q) x[q] = zero ? 0.f : x[q] * coef;
        store4<float, f32x4u>(ts.out_ptr, e, ts.numel, x);
    }
}

// The clipped gradients in fp32; zeros when the norm is not finite, so that a
// step that takes them adds nothing to its statistics.
__global__ __launch_bounds__(256) void k_clip(NormArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    const ClipRecord r = *a.record;
    for (int i = wave; i < a.ntiles; i += gridDim.x * 4) {
        const NormTile tl = a.tiles[i];
        const NormTensor ts = a.tensors[tl.tensor];
        if (!ts.g_ptr || !ts.out_ptr) continue;
        // in place and nothing to clip: the gradient stands
        if (ts.out_ptr == ts.g_ptr && r.coef == 1.f) continue;
        const bool zero = r.nonfinite != 0;
        if (ts.dtype == DT_F32) tile_clip<DT_F32>(ts, tl.first, lane, r.coef, zero);
        else if (ts.dtype == DT_BF16) tile_clip<DT_BF16>(ts, tl.first, lane, r.coef, zero);
        else tile_clip<DT_F16>(ts, tl.first, lane, r.coef, zero);
    }
}

template <int P, int G>
hipError_t go(bool bits8, const AdamwArgs& a, hipStream_t s) {
    const dim3 grid(adamw_grid(a.ntiles)), block(256);
    if (bits8) hipLaunchKernelGGL((k_adamw<P, G, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_adamw<P, G, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int P>
hipError_t go_grad(int grad, bool bits8, const AdamwArgs& a, hipStream_t s) {
    if (grad == DT_F32) return go<P, DT_F32>(bits8, a, s);
    if (grad == DT_BF16) return go<P, DT_BF16>(bits8, a, s);
    return go<P, DT_F16>(bits8, a, s);
}

}  // namespace

// Eight workgroups on each of the 256 CUs at most, four tiles (one per wave)
// to a workgroup.
int adamw_grid(int64_t ntiles) { return (int)(ntiles < 8192 ? (ntiles + 3) / 4 : 2048); }
int norm_grid(int64_t ntiles) { return (int)(ntiles < 4096 ? (ntiles + 3) / 4 + (ntiles == 0) : 1024); }

hipError_t launch_adamw(int param, int grad, bool bits8, const AdamwArgs& a, hipStream_t s) {
    return param == DT_F32 ? go_grad<DT_F32>(grad, bits8, a, s)
                           : go_grad<DT_BF16>(grad, bits8, a, s);
}

hipError_t launch_adamw_clock(AdamwClock* clocks, int n, const AdamwClock& c, hipStream_t s) {
    hipLaunchKernelGGL(k_adamw_clock, dim3((n + 255) / 256), dim3(256), 0, s, clocks, n, c);
    return hipGetLastError();
}

hipError_t launch_adamw_bind(AdamwTensor* tensors, int first, int n, const PtrBatch& b, int which,
                             hipStream_t s) {
    hipLaunchKernelGGL(k_adamw_bind, dim3(1), dim3(256), 0, s, tensors + first, n, b, which);
    return hipGetLastError();
}

hipError_t launch_norm_bind(NormTensor* tensors, int first, int n, const PtrBatch& b,
                            hipStream_t s) {
    hipLaunchKernelGGL(k_norm_bind, dim3(1), dim3(256), 0, s, tensors + first, n, b);
    return hipGetLastError();
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_norm, dim3(norm_grid(a.ntiles)), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_clip(const NormArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_clip, dim3(norm_grid(a.ntiles)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace shampoo
