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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2h __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4h __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// A caller's pointer through the global address space (global, not flat,
// memory instructions).
template <typename T>
__device__ __forceinline__ T* gptr(uint64_t addr) {
    typedef __attribute__((address_space(1))) T gT;
    return (T*)reinterpret_cast<gT*>(addr);
}

// One load or store, past the caches' retention (NT) or not.
template <bool NT, typename T>
__device__ __forceinline__ T ld(const T* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, typename T>
__device__ __forceinline__ void st(T* p, T x) {
    if constexpr (NT) __builtin_nontemporal_store(x, p);
    else *p = x;
}

// The same at any address that suits an element (a template argument would
// lose the vector's alignment, so each type has its own).
#define SHAMPOO_LOOSE(V)                                                  \
    template <bool NT>                                                    \
    __device__ __forceinline__ V ld_loose(const V* p) {                   \
        if constexpr (NT) return __builtin_nontemporal_load(p);           \
        else return *p;                                                   \
    }                                                                     \
    template <bool NT>                                                    \
    __device__ __forceinline__ void st_loose(V* p, V x) {                 \
        if constexpr (NT) __builtin_nontemporal_store(x, p);              \
        else *p = x;                                                      \
    }
SHAMPOO_LOOSE(f32x4u)
SHAMPOO_LOOSE(u32x2h)
SHAMPOO_LOOSE(u32x4h)
#undef SHAMPOO_LOOSE

template <int DT> struct Elem { typedef unsigned short type; };
template <> struct Elem<DT_F32> { typedef float type; };

template <int DT>
__device__ __forceinline__ float widen(typename Elem<DT>::type u) {
    if constexpr (DT == DT_F32) return u;
    else if constexpr (DT == DT_BF16) return __uint_as_float((uint32_t)u << 16);
    else {
        _Float16 h;
        __builtin_memcpy(&h, &u, 2);
        return (float)h;
    }
}

// Four elements as they lie in memory: 16 or 8 bytes.
template <int DT> struct Raw { u32x2 w; };
template <> struct Raw<DT_F32> { f32x4 w; };

template <int DT>
__device__ __forceinline__ f32x4 widen4(const Raw<DT>& r) {
    if constexpr (DT == DT_F32) return r.w;
    else if constexpr (DT == DT_BF16)
        return f32x4{__uint_as_float(r.w.x << 16), __uint_as_float(r.w.x & 0xFFFF0000u),
                     __uint_as_float(r.w.y << 16), __uint_as_float(r.w.y & 0xFFFF0000u)};
    else {
        f32x4 x;
        for (int k = 0; k < 4; ++k) x[k] = widen<DT>((unsigned short)(r.w[k >> 1] >> (16 * (k & 1))));
        return x;
    }
}

// A lane's address: a base that the whole wave shares (in scalar registers),
// the lane's own 32-bit byte offset, and a constant.
template <typename T>
__device__ __forceinline__ T* lane_at(uint64_t base, uint32_t bytes, int add) {
    typedef typename std::conditional<std::is_const<T>::value, const char, char>::type C;
    return reinterpret_cast<T*>(gptr<C>(base) + bytes + add);
}

// Four consecutive elements, from element lane + add of what starts at `base`
// and has `rest` elements; FULL: all four exist, else those past the end read
// as 0.
template <int DT, bool FULL, bool NT = false>
__device__ __forceinline__ Raw<DT> load4(uint64_t base, uint32_t lane, int add, int64_t rest) {
    typedef typename Elem<DT>::type T;
    constexpr int kSize = (int)sizeof(T);
    const T* p = lane_at<const T>(base, lane * kSize, add * kSize);
    const int64_t left = rest - ((int64_t)lane + add);
    Raw<DT> r;
    if constexpr (DT == DT_F32) {
        if (FULL || left >= 4) {
            r.w = ld_loose<NT>(reinterpret_cast<const f32x4u*>(p));
        } else {
            for (int k = 0; k < 4; ++k) r.w[k] = k < left ? p[k] : 0.f;
        }
    } else {
        if (FULL || left >= 4) {
            r.w = ld_loose<NT>(reinterpret_cast<const u32x2h*>(p));
        } else {
            uint32_t u[4];
            for (int k = 0; k < 4; ++k) u[k] = k < left ? p[k] : 0u;
            r.w = u32x2{u[0] | u[1] << 16, u[2] | u[3] << 16};
        }
    }
    return r;
}

template <int DT, bool FULL, bool NT = false>
__device__ __forceinline__ void store4(uint64_t base, uint32_t lane, int add, int64_t rest, const Raw<DT>& r) {
    typedef typename Elem<DT>::type T;
    constexpr int kSize = (int)sizeof(T);
    T* p = lane_at<T>(base, lane * kSize, add * kSize);
    const int64_t left = rest - ((int64_t)lane + add);
    if constexpr (DT == DT_F32) {
        if (FULL || left >= 4) {
            st_loose<NT>(reinterpret_cast<f32x4u*>(p), r.w);
        } else {
            for (int k = 0; k < 4; ++k)
                if (k < left) p[k] = r.w[k];
        }
    } else {
        if (FULL || left >= 4) {
            st_loose<NT>(reinterpret_cast<u32x2h*>(p), r.w);
        } else {
            for (int k = 0; k < 4; ++k)
                if (k < left) p[k] = (T)(r.w[k >> 1] >> (16 * (k & 1)));
        }
    }
}

// Lane permutations inside the ALU.  A half wave is two rows of 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
// The largest `a` of the half in the lanes of its first row, the largest `b`
// in those of its second: the rows' halves are exchanged first, so that one
// reduction does for both.  The lanes of a half are active together.
__device__ __forceinline__ uint32_t half_max2(uint32_t a, uint32_t b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    uint32_t v = umax(r[0], r[1]);
    v = umax(v, moved<0xB1>(v));    // quad_perm [1,0,3,2]
    v = umax(v, moved<0x4E>(v));    // quad_perm [2,3,0,1]
    v = umax(v, moved<0x141>(v));   // the other quad of eight
    return umax(v, moved<0x140>(v));   // the other eight of the row
}
// What the first and the second row hold (each the same in its 16 lanes), to
// all lanes of the half.
__device__ __forceinline__ void half_both(float v, float& first, float& second) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    first = __uint_as_float(r[0]);
    second = __uint_as_float(r[1]);
}

// 1/d rounded to nearest, for normal d and 1/d: one Newton step on the
// hardware's reciprocal (equal to 1/d for every significand and every
// exponent from -125 to 125; the tests count those of the divisors that second
// moments from 2^-96 on give).
__device__ __forceinline__ float reciprocal(float d) {
    const float y = __builtin_amdgcn_rcpf(d);
    return __builtin_fmaf(__builtin_fmaf(-d, y, 1.f), y, y);
}
// m/d rounded to nearest: the quotient by the rounded reciprocal is within
// one unit, and its remainder, exact in one fma, decides (Markstein 1990).
// d: positive, normal, below 2^126.  m: 0, or at least 2^-100 in magnitude, so
// that the remainder's last place (2^-47 of m) is one of fp32, with a quotient
// that is normal and finite: of smaller ones one in ten at m = 2^-125 would be
// off by its last place.
__device__ __forceinline__ float quotient(float m, float d) {
    const float y = reciprocal(d);
    const float q = m * y;
    return __builtin_fmaf(__builtin_fmaf(-d, q, m), y, q);
}
// sqrt(v) rounded to nearest for v = 0 and 2^-96 <= v < infinity: one
// correction of v / sqrt(v) (equal to the rounded root for every significand
// and every exponent of that range, which the tests count).  NaN for v that is
// not finite.
constexpr uint32_t kRootLow = 0x0F800000u;   // 2^-96
constexpr float kQuoLow = 0x1p-100f;         // the least |m| of `quotient`
constexpr uint32_t kQuoHigh = 0x67000000u;   // 2^79, which the root of kRootLow takes to 2^127
__device__ __forceinline__ float near_root(float v) {
    const float y = __builtin_amdgcn_rsqf(__uint_as_float(umax(__float_as_uint(v), kRootLow)));
    const float r = v * y;
    return __builtin_fmaf(__builtin_fmaf(-r, r, v), 0.5f * y, r);
}

// Scale of a run from the largest magnitude among its finite values, and the
// factor that takes values to e4m3's range (up to 448, and up to 3 units in
// the last place past it).  The floor keeps the factor finite; values below
// it are kept as they fall under that scale.
__device__ __forceinline__ void run_scale(uint32_t amax_bits, float& scale, float& inv) {
    scale = fmaxf(__uint_as_float(amax_bits), 0x1p-110f) * (1.0f / 448);
    inv = reciprocal(scale);
}

constexpr uint32_t kFinite = 0x7F7FFFFFu;

// A value x becomes an e4m3 code of y = x inv, |y| <= 448, rounded to the code
// above in magnitude with the probability of the fraction that e4m3 drops, so
// that moving averages whose change in one step is less than half a code still
// move: 16 random bits are added at the top of the 20 mantissa bits that are
// dropped.  Their sum does not carry past code 126: the random part is at most
// 2^20 - 16 of 2^20.  The hardware's conversion does this for |y| >= 2^-6.
//
// Below 2^-6 e4m3 steps evenly, as fp32 rounded to three bits does in [2^-6,
// 2^-5): there y counts as y + 2^-6 in fp32.  In integers, with the code in
// the top byte and bit 31 clear: (y + 2^-6) / 2 has the code 8 less that
// belongs there, is larger than y below 2^-6 and smaller above; r holds the
// random bits in bits 8 to 23 and 0x40 = -(120 << 3) mod 256, the difference
// in bias, in the top byte.  A value that is not finite becomes NaN, code 127.
__device__ __forceinline__ uint32_t encode_any(float x, float inv, uint32_t r) {
    const bool finite = (__float_as_uint(x) & 0x7FFFFFFFu) <= kFinite;
    const float y = finite ? fabsf(x) * inv : 0.f;
    const float z = fmaxf(y, __builtin_fmaf(y, 0.5f, 0x1p-7f));
    return finite ? (__float_as_uint(z) << 4) + r : 0x7F000000u;
}
// The top bytes of four words, as one word.
__device__ __forceinline__ uint32_t top_bytes(const uint32_t* w) {
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w[3], w[2], 0x07030c0cu),
                                 __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0703u), 0x07060100u);
}

__device__ __forceinline__ f32x4 decode4(uint32_t w) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    return f32x4{lo.x, lo.y, hi.x, hi.y};
}

// The codes of this lane's eight elements.  `start`: the hash's input of the
// first one after the first shift-xor; those of the others differ by their
// offset, in bits that the shift does not reach.  ANY: the run holds values
// below 2^-6 of e4m3's range or not finite.
template <bool ANY, bool NT>
__device__ __forceinline__ void encode_run(const f32x4* m, const f32x4* root, float mi, float si,
                                           uint32_t start, uint64_t m8, uint64_t s8, uint32_t lo) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t h[4], mw = 0, sw = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) h[q] = mix32_rest(start ^ (uint32_t)(128 * j + q));
        if constexpr (ANY) {
            uint32_t mc[4], sc[4];
            for (int q = 0; q < 4; ++q) {
                const float x = m[j][q], y = root[j][q];
                // from the top byte down: 0x40, half of the hash, 0
                mc[q] = encode_any(x, mi, __builtin_amdgcn_perm(0x40000000u, h[q], 0x0701000cu));
                sc[q] = encode_any(y, si, __builtin_amdgcn_perm(0x40000000u, h[q], 0x0703020cu));
                mc[q] = (mc[q] & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u);
                // a positive root never becomes 0, whose division would be by
                // eps alone: code 1 at least, unless the root is 0
                const uint32_t yb = __float_as_uint(y);
                sc[q] = umax(sc[q], yb < 0x01000000u ? yb : 0x01000000u);
            }
            mw = top_bytes(mc);
            sw = top_bytes(sc);
        } else {
            mw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(m[j][0] * mi, h[0] << 16, (int)mw, 0);
            mw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(m[j][1] * mi, h[1] << 16, (int)mw, 1);
            mw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(m[j][2] * mi, h[2] << 16, (int)mw, 2);
            mw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(m[j][3] * mi, h[3] << 16, (int)mw, 3);
            sw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(root[j][0] * si, h[0] & 0xFFFF0000u, (int)sw, 0);
            sw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(root[j][1] * si, h[1] & 0xFFFF0000u, (int)sw, 1);
            sw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(root[j][2] * si, h[2] & 0xFFFF0000u, (int)sw, 2);
            sw = (uint32_t)__builtin_amdgcn_cvt_sr_fp8_f32(root[j][3] * si, h[3] & 0xFFFF0000u, (int)sw, 3);
        }
        st<NT>(lane_at<uint32_t>(m8, lo, 128 * j), mw);
        st<NT>(lane_at<uint32_t>(s8, lo, 128 * j), sw);
    }
}

// Two runs of 256 elements from `run`, one to each half of the wave: lane l
// (of 32) takes the elements 4l.. and 128 + 4l.. of its run, so that every
// load and store of a half covers whole 128-byte lines.  Without FULL the runs
// are those that the tensor ends in, and the second half may be idle.
template <int P, int G, bool S8, bool FULL, bool NT>
__device__ __forceinline__ void step_runs(const AdamwArgs& a, const AdamwTensor& ts, int64_t run, float coef,
                                          float fa, float fb, float root_c, uint32_t key) {
    const int l = threadIdx.x & 31;
    const uint32_t half = (threadIdx.x >> 5) & 1;
    const uint32_t lo = half * kRun + 4 * l;                  // the lane's first element
    const int64_t sr = ts.state_run + run;
    const int64_t rest = ts.numel - run * kRun;               // elements from the first run on
    const uint64_t gb = ts.g_ptr + (uint64_t)run * kRun * sizeof(typename Elem<G>::type);
    const uint64_t pb = ts.p_ptr + (uint64_t)run * kRun * sizeof(typename Elem<P>::type);
    const uint64_t rb = reinterpret_cast<uint64_t>(a.rem + (ts.rem_run + run) * kRun);
    const uint64_t mb = S8 ? reinterpret_cast<uint64_t>(a.m8 + sr * kRun) : reinterpret_cast<uint64_t>(a.m + sr * kRun);
    const uint64_t vb = S8 ? reinterpret_cast<uint64_t>(a.s8 + sr * kRun) : reinterpret_cast<uint64_t>(a.v + sr * kRun);
    const uint64_t msb = reinterpret_cast<uint64_t>(a.m_scale + sr);
    const uint64_t ssb = reinterpret_cast<uint64_t>(a.s_scale + sr);
    Raw<G> graw[2];
    Raw<P> praw[2];
    u32x2 rem[2];
    uint32_t mw[2], sw[2];
    f32x4 m[2], v[2];
    float ms = 0.f, ss = 0.f;
    if constexpr (S8) {
        ms = *lane_at<const float>(msb, 4 * half, 0);
        ss = *lane_at<const float>(ssb, 4 * half, 0);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        graw[j] = load4<G, FULL, NT>(gb, lo, 128 * j, rest);
        praw[j] = load4<P, FULL, NT>(pb, lo, 128 * j, rest);
        if constexpr (P == DT_BF16) rem[j] = ld<NT>(lane_at<const u32x2>(rb, 2 * lo, 256 * j));
        if constexpr (S8) {
            mw[j] = ld<NT>(lane_at<const uint32_t>(mb, lo, 128 * j));
            sw[j] = ld<NT>(lane_at<const uint32_t>(vb, lo, 128 * j));
        } else {
            m[j] = ld<NT>(lane_at<const f32x4>(mb, 4 * lo, 512 * j));
            v[j] = ld<NT>(lane_at<const f32x4>(vb, 4 * lo, 512 * j));
        }
    }
    // the largest magnitude of m as the largest signed and the largest unsigned
    // of its bits: positive and negative values, NaN above all; the least that
    // is not 0 as the least of twice its bits - 1
    int mpos = 0;
    uint32_t mneg = 0, mlow = 0xFFFFFFFFu, vmin = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        f32x4 x = widen4<G>(graw[j]);
        if (coef != 1.f)
            for (int q = 0; q < 4; ++q) x[q] = x[q] * coef;
        if constexpr (S8) {
            m[j] = decode4(mw[j]);
            v[j] = decode4(sw[j]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (S8) {
                m[j][q] = m[j][q] * ms;
                v[j][q] = v[j][q] * ss;
                v[j][q] = v[j][q] * v[j][q];
            }
            m[j][q] = m[j][q] * a.b1 + x[q] * a.c1;
            v[j][q] = v[j][q] * a.b2 + (x[q] * x[q]) * a.c2;
            vmin = umin(vmin, __float_as_uint(v[j][q]));
            const uint32_t b = __float_as_uint(m[j][q]);
            mpos = mpos > (int)b ? mpos : (int)b;
            mneg = umax(mneg, b);
            mlow = umin(mlow, (b << 1) - 1u);
        }
    }
    f32x4 root[2], quo[2];
    uint32_t smax = 0, mmax = umax((uint32_t)mpos, mneg & 0x7FFFFFFFu);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            root[j][q] = near_root(v[j][q]);
            smax = umax(smax, __float_as_uint(root[j][q]));
        }
    // the least m whose quotient by the lane's largest divisor is normal
    const float least = fmaxf((__uint_as_float(smax) * root_c + a.eps) * 0x1p-125f, kQuoLow);
    if (__any(vmin < kRootLow || smax > kFinite || mlow < (__float_as_uint(least) << 1) - 1u || mmax >= kQuoHigh)) {
        // second moments that are 0, tiny or not finite, and tiny or huge m
        smax = 0;
        for (int j = 0; j < 2; ++j)
            for (int q = 0; q < 4; ++q) {
                root[j][q] = sqrtf(v[j][q]);
                smax = umax(smax, __float_as_uint(root[j][q]));
                quo[j][q] = m[j][q] / (root[j][q] * root_c + a.eps);
            }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) quo[j][q] = quotient(m[j][q], root[j][q] * root_c + a.eps);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        Raw<P> out;
        u32x2 left;
        f32x4 w;
        if constexpr (P == DT_BF16) {
            // bits = (hi << 16) + the signed remainder
            for (int q = 0; q < 4; ++q) {
                const uint32_t hi = q & 1 ? praw[j].w[q >> 1] & 0xFFFF0000u : praw[j].w[q >> 1] << 16;
                const uint32_t r = q & 1 ? (uint32_t)((int)rem[j][q >> 1] >> 16)
                                         : (uint32_t)(int)(short)rem[j][q >> 1];
                w[q] = __uint_as_float(hi + r);
            }
        } else {
            w = praw[j].w;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = w[q] - (w[q] * fa + quo[j][q] * fb);
        if constexpr (P == DT_BF16) {
            // the nearest bf16 (ties away from zero) is the upper half of bits +
            // 2^15, and what is left, as a signed number, is the lower half of
            // bits; a NaN becomes the quiet NaN without remainder
            uint32_t b[4];
            for (int q = 0; q < 4; ++q) b[q] = __float_as_uint(w[q]);
            if (__any(__builtin_isunordered(w[0], w[1]) || __builtin_isunordered(w[2], w[3])))
                for (int q = 0; q < 4; ++q) b[q] = w[q] != w[q] ? 0x7FC00000u : b[q];
            for (int k = 0; k < 2; ++k) {
                out.w[k] = __builtin_amdgcn_perm(b[2 * k + 1] + 0x8000u, b[2 * k] + 0x8000u, 0x07060302u);
                left[k] = __builtin_amdgcn_perm(b[2 * k + 1], b[2 * k], 0x05040100u);
            }
            st<NT>(lane_at<u32x2>(rb, 2 * lo, 256 * j), left);
        } else {
            out.w = w;
        }
        store4<P, FULL, NT>(pb, lo, 128 * j, rest, out);
        if constexpr (!S8) {
            st<NT>(lane_at<f32x4>(mb, 4 * lo, 512 * j), m[j]);
            st<NT>(lane_at<f32x4>(vb, 4 * lo, 512 * j), v[j]);
        }
    }
    if constexpr (S8) {
        float mleast = __builtin_inff(), sleast = __builtin_inff();
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mleast = fminf(mleast, fabsf(m[j][q]));
                sleast = fminf(sleast, root[j][q]);
            }
        uint32_t top = half_max2(mmax, smax);
        const bool odd = __any(top > kFinite);
        if (odd) {   // the scales are those of the finite values
            mmax = smax = 0;
            for (int j = 0; j < 2; ++j)
                for (int q = 0; q < 4; ++q) {
                    const uint32_t mb = __float_as_uint(m[j][q]) & 0x7FFFFFFFu;
                    const uint32_t sb = __float_as_uint(root[j][q]) & 0x7FFFFFFFu;
                    mmax = umax(mmax, mb <= kFinite ? mb : 0u);
                    smax = umax(smax, sb <= kFinite ? sb : 0u);
                }
            top = half_max2(mmax, smax);
        }
        // the first row works on m, the second on the root
        float scale, inv, mi, si;
        run_scale(top, scale, inv);
        half_both(inv, mi, si);
        if (l == 0) *lane_at<float>(msb, 4 * half, 0) = scale;
        if (l == 16) *lane_at<float>(ssb, 4 * half, 0) = scale;
        // the element's index: two runs from an even one share its upper half
        const uint64_t e0 = (uint64_t)run * kRun;
        uint32_t start = (key + (uint32_t)(e0 >> 32) * 0x85157AF5u) ^ ((uint32_t)e0 | lo);
        start ^= start >> 16;
        if (__any(mleast * mi < 0x1p-6f || sleast * si < 0x1p-6f) || odd)
            encode_run<true, NT>(m, root, mi, si, start, mb, vb, lo);
        else
            encode_run<false, NT>(m, root, mi, si, start, mb, vb, lo);
    }
}

// One step of the elements of this workgroup's tile.
//
// Waves per SIMD are held below what the registers would allow: more of them
// spread the accesses over more of the memory's pages at once.  fp32 moments,
// 302M fp32 elements: 1367 us with 4, 1385 with 6, 1434 (up to 1520) with 8.
// 8-bit moments need more for the arithmetic, 302M / 60M bf16 elements: 805 /
// 192 us with 3, 730 / 177 with 4, 695 / 161 with 5, 745 / 158 with 6, 755 /
// 157 with 7.
template <int P, int G, bool S8, bool NT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, S8 ? 5 : 4))) void k_adamw(AdamwArgs a) {
    // field by field: a copy of the whole struct, its padding included, went
    // through LDS and cost 14 us at 256 workgroups
    AdamwClock* clock = a.clocks + blockIdx.x;
    const int64_t t = clock->t, k = clock->k;
    const double b1k = clock->b1k, b2k = clock->b2k, inv1 = clock->inv1;
    const float root_c = clock->inv_root2;
    float coef = 1.f;
    if (a.clip) {
        if (a.clip->nonfinite) return;   // the same for every workgroup: nothing changes
        coef = a.clip->coef;
    }
    const double lr = a.lr_dev ? (double)*a.lr_dev : a.lr;
    const uint32_t key0 = mix32(a.seed_mixed + (uint32_t)(t + 1));
    const AdamwTile tl = a.tiles[blockIdx.x];
    const AdamwTensor ts = a.tensors[tl.tensor];
    const float fa = (float)(lr * ts.lr_scale * ts.weight_decay);
    const float fb = (float)(lr * ts.lr_scale * inv1);
    const uint32_t key = mix32(key0 + (uint32_t)ts.id);
    // two runs to each of the four waves
    const int64_t run = tl.run0 + 2 * __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (ts.g_ptr) {
        if ((run + 2) * kRun <= ts.numel)
            step_runs<P, G, S8, true, NT>(a, ts, run, coef, fa, fb, root_c, key);
        else if ((run + ((threadIdx.x >> 5) & 1)) * kRun < ts.numel)
            step_runs<P, G, S8, false, false>(a, ts, run, coef, fa, fb, root_c, key);
    }
    __syncthreads();   // every wave has read the clock
    if (threadIdx.x == 0) {
        clock->t = t + 1;
        if (a.per_tensor && !ts.g_ptr) return;   // no step of this tensor
        const double n1 = b1k * a.beta1, n2 = b2k * a.beta2;
        clock->k = k + 1;
        clock->b1k = n1;
        clock->b2k = n2;
        clock->inv1 = 1.0 / (1.0 - n1);
        clock->inv_root2 = (float)(1.0 / sqrt(1.0 - n2));
    }
}

__global__ __launch_bounds__(256) void k_adamw_clock(AdamwClock* clocks, int n, AdamwClock c, int which) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    if (which & 1) clocks[i].t = c.t;
    if (which & 2) {
        clocks[i].k = c.k;
        clocks[i].b1k = c.b1k;
        clocks[i].b2k = c.b2k;
        clocks[i].inv1 = c.inv1;
        clocks[i].inv_root2 = c.inv_root2;
    }
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
// Sum over the 64 lanes of a wave by lane permutations inside the ALU: pairs,
// quads, rows of 16, then rows 0 and 2 into 1 and 3, and row 1 into row 3,
// whose last lane is read out.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved_d(double v) {
    const int lo = __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xf, false);
    return __hiloint2double(hi, lo);
}
__device__ __forceinline__ double wave_total(double v) {
    v += moved_d<0xB1, 0xf>(v);    // quad_perm [1,0,3,2]
    v += moved_d<0x4E, 0xf>(v);    // quad_perm [2,3,0,1]
    v += moved_d<0x141, 0xf>(v);   // the other quad of eight
    v += moved_d<0x140, 0xf>(v);   // the other eight of a row
    v += moved_d<0x142, 0xa>(v);   // row_bcast:15 into rows 1 and 3
    v += moved_d<0x143, 0xc>(v);   // row_bcast:31 into rows 2 and 3
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), 63),
                            __builtin_amdgcn_readlane(__double2loint(v), 63));
}
// The sum over a workgroup of kNormWaves waves, to every lane.
__device__ __forceinline__ double group_sum(double v, double* red) {
    v = wave_total(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kNormWaves; ++w) t += red[w];
    return t;
}

// 16 bytes of a gradient per lane and load: a wave reads a piece of kNormPiece
// elements with all its loads in flight.
template <int DT> struct Piece {
    static constexpr int kPer = DT == DT_F32 ? 4 : 8;          // elements of a load
    static constexpr int kLoads = kNormPiece / 64 / kPer;
    u32x4 w[kLoads];
};

template <int DT, bool NT>
__device__ __forceinline__ void load_piece(Piece<DT>& r, uint64_t g, int64_t first, int64_t numel, int lane) {
    typedef typename Elem<DT>::type T;
    constexpr int kPer = Piece<DT>::kPer;
    if (first + kNormPiece <= numel) {
#pragma unroll
        for (int k = 0; k < Piece<DT>::kLoads; ++k)
            r.w[k] = ld_loose<NT>(gptr<const u32x4h>(g + (uint64_t)(first + (k * 64 + lane) * kPer) * sizeof(T)));
        return;
    }
    for (int k = 0; k < Piece<DT>::kLoads; ++k) {
        const int64_t e = first + (k * 64 + lane) * kPer;
        const uint64_t at = g + (uint64_t)e * sizeof(T);
        if (e + kPer <= numel) {
            r.w[k] = *gptr<const u32x4h>(at);
        } else {
            r.w[k] = u32x4{0, 0, 0, 0};
            for (int q = 0; q < kPer; ++q)
                if (e + q < numel) {
                    if constexpr (DT == DT_F32) r.w[k][q] = gptr<const uint32_t>(at)[q];
                    else r.w[k][q >> 1] |= (uint32_t)gptr<const unsigned short>(at)[q] << (16 * (q & 1));
                }
        }
    }
}

template <int DT>
__device__ __forceinline__ double piece_squares(const Piece<DT>& r) {
    double s[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < Piece<DT>::kLoads; ++k)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (DT == DT_F32) {
                const double x = (double)__uint_as_float(r.w[k][q]);
                s[q] = __builtin_fma(x, x, s[q]);
            } else {
                const Raw<DT> two{u32x2{r.w[k][q], 0u}};
                const f32x4 f = widen4<DT>(two);
                const double x = (double)f[0], y = (double)f[1];
                s[q] = __builtin_fma(x, x, s[q]);
                s[q] = __builtin_fma(y, y, s[q]);
            }
        }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

template <int DT, bool NT>
__device__ __forceinline__ double tile_squares(const NormTensor& ts, int64_t first, int pieces, int lane) {
    double acc = 0.0;
    for (int p = 0; p < pieces; ++p) {
        const int64_t e = first + (int64_t)p * kNormPiece;
        if (e >= ts.numel) break;
        Piece<DT> r;
        load_piece<DT, NT>(r, ts.g_ptr, e, ts.numel, lane);
        acc += piece_squares<DT>(r);
    }
    return acc;
}

// Sum of the squares of every gradient in fp64 (the squares of fp32 values
// are exact in it, none overflows), in an order that the plan fixes: each
// wave over its tiles, each workgroup over its waves, the last workgroup to
// finish over the workgroups' sums.
template <bool NT>
__global__ __launch_bounds__(64 * kNormWaves) void k_norm(NormArgs a) {
    __shared__ double red[kNormWaves];
    __shared__ int last;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * kNormWaves + (threadIdx.x >> 6));
    double acc = 0.0;
    // the tables are read ahead: the tile after next and the next one's tensor
    // while a tile's gradients arrive
    const int stride = gridDim.x * kNormWaves, end = a.ntiles - 1;
    if (wave <= end) {
        NormTile tl = a.tiles[wave];
        NormTile next = a.tiles[wave + stride < end ? wave + stride : end];
        NormTensor ts = a.tensors[tl.tensor];
        for (int i = wave; i <= end; i += stride) {
            const NormTile later = a.tiles[i + 2 * stride < end ? i + 2 * stride : end];
            const NormTensor tn = a.tensors[next.tensor];
            if (ts.g_ptr) {
                if (ts.dtype == DT_F32) acc += tile_squares<DT_F32, NT>(ts, tl.first, a.pieces, lane);
                else if (ts.dtype == DT_BF16) acc += tile_squares<DT_BF16, NT>(ts, tl.first, a.pieces, lane);
                else acc += tile_squares<DT_F16, NT>(ts, tl.first, a.pieces, lane);
            }
            tl = next;
            next = later;
            ts = tn;
        }
    }
    const double sum = group_sum(acc, red);
    if (threadIdx.x == 0) {
        // The sum is written through to where every XCD reads it, and is there
        // before this workgroup counts itself as done.  A release at agent
        // scope would also write the whole L2 back, 60 ns a workgroup one
        // after another.
        __hip_atomic_store(a.partials + blockIdx.x, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        // counts of one address are 12 ns one after another: a large grid
        // counts in groups, and the last of each group among the groups
        const int n = (int)gridDim.x, groups = n > 2 * kNormGroups ? kNormGroups : 1;
        const int g = (int)blockIdx.x % groups;
        int32_t* ticket = a.tickets + 32 * g;
        last = __hip_atomic_fetch_add(ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
               (n - g + groups - 1) / groups - 1;
        if (last) {
            *ticket = 0;   // for the next launch
            if (groups > 1)
                last = __hip_atomic_fetch_add(a.tickets + 32 * kNormGroups, 1, __ATOMIC_RELAXED,
                                              __HIP_MEMORY_SCOPE_AGENT) == groups - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    double t = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += 64 * kNormWaves)
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
        a.tickets[32 * kNormGroups] = 0;
    }
}

template <int DT, bool FULL>
__device__ __forceinline__ void piece_clip(const NormTensor& ts, int64_t first, int lane, float coef, bool zero) {
    const int64_t rest = ts.numel - first;
    const uint64_t gb = ts.g_ptr + (uint64_t)first * sizeof(typename Elem<DT>::type);
    const uint64_t ob = ts.out_ptr + (uint64_t)first * 4;
    Raw<DT> raw[kNormPiece / 256];
#pragma unroll
    for (int k = 0; k < kNormPiece / 256; ++k)
        raw[k] = load4<DT, FULL>(gb, 4 * lane, 256 * k, rest);
#pragma unroll
    for (int k = 0; k < kNormPiece / 256; ++k) {
        const f32x4 x = widen4<DT>(raw[k]);
        Raw<DT_F32> y;
        for (int q = 0; q < 4; ++q) y.w[q] = zero ? 0.f : x[q] * coef;
        store4<DT_F32, FULL>(ob, 4 * lane, 256 * k, rest, y);
    }
}
template <int DT>
__device__ __forceinline__ void tile_clip(const NormTensor& ts, int64_t first, int pieces, int lane, float coef,
                                          bool zero) {
    for (int p = 0; p < pieces; ++p) {
        const int64_t e = first + (int64_t)p * kNormPiece;
        if (e >= ts.numel) break;
        if (e + kNormPiece <= ts.numel) piece_clip<DT, true>(ts, e, lane, coef, zero);
        else piece_clip<DT, false>(ts, e, lane, coef, zero);
    }
}

// The clipped gradients in fp32; zeros when the norm is not finite, so that
// nothing else reaches the statistics of a step that takes them.
__global__ __launch_bounds__(256) void k_clip(NormArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    if (wave >= a.ntiles) return;
    const float coef = a.record->coef;
    const bool zero = a.record->nonfinite != 0;
    const NormTile tl = a.tiles[wave];
    const NormTensor ts = a.tensors[tl.tensor];
    // nothing asked for, or in place and nothing to clip
    if (!ts.g_ptr || !ts.out_ptr || (ts.out_ptr == ts.g_ptr && coef == 1.f)) return;
    if (ts.dtype == DT_F32) tile_clip<DT_F32>(ts, tl.first, a.pieces, lane, coef, zero);
    else if (ts.dtype == DT_BF16) tile_clip<DT_BF16>(ts, tl.first, a.pieces, lane, coef, zero);
    else tile_clip<DT_F16>(ts, tl.first, a.pieces, lane, coef, zero);
}

template <int P, int G>
hipError_t go(bool bits8, const AdamwArgs& a, hipStream_t s) {
    const dim3 grid(a.ntiles), block(256);
    if (bits8) {
        if (a.stream_past) hipLaunchKernelGGL((k_adamw<P, G, true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_adamw<P, G, true, false>), grid, block, 0, s, a);
    } else {
        if (a.stream_past) hipLaunchKernelGGL((k_adamw<P, G, false, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((k_adamw<P, G, false, false>), grid, block, 0, s, a);
    }
    return hipGetLastError();
}

template <int P>
hipError_t go_grad(int grad, bool bits8, const AdamwArgs& a, hipStream_t s) {
    if (grad == DT_F32) return go<P, DT_F32>(bits8, a, s);
    if (grad == DT_BF16) return go<P, DT_BF16>(bits8, a, s);
    return go<P, DT_F16>(bits8, a, s);
}

}  // namespace

// At most two workgroups of eight waves on each of the 256 CUs (302M bf16
// elements: 92 us; 98 with workgroups of 16 waves, 104 with four workgroups).
int norm_grid(int64_t ntiles) {
    return (int)(ntiles < 512 * kNormWaves ? (ntiles + kNormWaves - 1) / kNormWaves + (ntiles == 0) : 512);
}

hipError_t launch_adamw(int param, int grad, bool bits8, const AdamwArgs& a, hipStream_t s) {
    return param == DT_F32 ? go_grad<DT_F32>(grad, bits8, a, s)
                           : go_grad<DT_BF16>(grad, bits8, a, s);
}

hipError_t launch_adamw_clock(AdamwClock* clocks, int n, const AdamwClock& c, int which, hipStream_t s) {
    hipLaunchKernelGGL(k_adamw_clock, dim3((n + 255) / 256), dim3(256), 0, s, clocks, n, c, which);
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
    const dim3 grid(norm_grid(a.ntiles)), block(64 * kNormWaves);
    if (a.stream_past) hipLaunchKernelGGL(k_norm<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(k_norm<false>, grid, block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_clip(const NormArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(k_clip, dim3((a.ntiles + 3) / 4), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace shampoo
