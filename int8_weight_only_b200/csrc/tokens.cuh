// Per-token int8 quantization of activations: for every row m of X [M, K]
//   s_m = max_k |X[m,k]| / 127,  q[m,k] = clamp(rne(X[m,k] / s_m), -127, 127),
//   sum_m = sum_k q[m,k]
// in IEEE fp32 (s_m = 0 gives q = 0), and the same for the SwiGLU of a gated
// MLP's first product, h = g / (1 + exp(-g)) * u.  The row sums let the
// int8 linear undo the offset of the weight codes.
//
// What is not finite stays visible behind the linear.  A row with a NaN has a
// NaN for its scale (and codes of 0): every output of the row is NaN.  A row
// with infinities has an infinite scale, their codes at the last level of
// their sign and the others 0: every output is infinite or NaN.
//
// One pass over X: a row is spread over TPR threads, each of which holds its
// values in registers between the row maximum and the rounding, so the plain
// quantizer is bound by HBM for many rows (4096 x 4096 fp32: 13.6 us, 6.2 TB/s)
// and by latency for few (1 x 4096: 1.6 us).  The SwiGLU (2048 x 13696: 40.9 us,
// 3.4 TB/s) saturates nothing: 28 instructions a value keep the schedulers busy
// in 56 % of the cycles, and three blocks an SM, each of loads, arithmetic,
// barrier and codes, do not cover one another's phases.
#pragma once

#include "i8.cuh"

namespace w8 {
namespace tokens {

constexpr int kF32 = 0;
constexpr int kF16 = 1;
constexpr int kSwiglu = 2;   // fp16 [M, 2K]: gate half, then up half

struct Params {
    const void *X;
    int64_t ldx;      // elements between rows
    int64_t M, K;
    int8_t *q;
    int64_t ldq;
    float *scales;
    int32_t *sums;
};

// Values travel as pairs of fp32 (f32x2): most steps below are IEEE operations
// on two values at once, half the instructions of this kernel's bound.
__device__ __forceinline__ void widen8(const uint4 &v, uint64_t (&f)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[i] = f32x2(p.x, p.y);
    }
}

// g / (1 + exp(-g)) by CUDA's exponential, an IEEE sum and an IEEE quotient: the
// values of an elementwise formula in fp32.
__device__ __forceinline__ float silu_ieee(float g) { return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g))); }

// Minus the same, for two values with |g| <= kSiluFast (the sign spares the
// negations on the way; the codes undo it).  The quotient by Markstein's method
// (IBM J. Res. Dev. 34(1), 1990): q = g r with an approximate reciprocal r of
// d, its exact remainder, q + (g - d q) r.  It gives the correctly rounded
// quotient for every one of the fp16 gates, which tests/test_tokens_gpu.py
// checks one by one.
constexpr float kSiluFast = 80.0f;
__device__ __forceinline__ float rcp_approx(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}
__device__ __forceinline__ uint64_t minus_silu2(uint64_t g) {
    const uint64_t ng = f32x2_mul(g, f32x2(-1.0f, -1.0f));
    const float2 v = f32x2_parts(ng);
    const uint64_t d = f32x2_add(f32x2(1.0f, 1.0f), f32x2(expf(v.x), expf(v.y)));
    const float2 dv = f32x2_parts(d);
    const uint64_t r = f32x2(rcp_approx(dv.x), rcp_approx(dv.y));
    const uint64_t minus_rem = f32x2_fma(d, f32x2_mul(g, r), ng);
    return f32x2_fma(minus_rem, r, f32x2_mul(ng, r));
}

// The largest magnitude of the even and of the odd ones of eight fp16 values.
__device__ __forceinline__ __half2 max_abs8(const uint4 &g) {
    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
    __half2 m = __habs2(*reinterpret_cast<const __half2 *>(&w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __half2 *>(&w[i])));
    return m;
}

// Minus silu(g) u of eight pairs.
__device__ __forceinline__ void swiglu8(const uint4 &g, const uint4 &u, uint64_t (&f)[4]) {
    uint64_t up[4];
    widen8(g, f);
    widen8(u, up);
    // (false for NaN: those take the plain formula)
    if (__hble2(max_abs8(g), __float2half2_rn(kSiluFast))) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f32x2_mul(minus_silu2(f[i]), up[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = f32x2_parts(f[i]);
            f[i] = f32x2_mul(f32x2(-silu_ieee(v.x), -silu_ieee(v.y)), up[i]);
        }
    }
}

// Eight consecutive values of a row, from element k (of the SwiGLU with the
// sign turned).  By ordinary loads: the kernel before, which may still run when
// this one begins, writes X, and the read-only path (ld.global.nc) is for memory
// that nobody writes in the meantime.
template <int kSrc>
__device__ __forceinline__ void load8(const Params &p, int64_t row, int64_t k, uint64_t (&f)[4]) {
    if constexpr (kSrc == kF32) {
        const ulonglong2 *src = reinterpret_cast<const ulonglong2 *>(static_cast<const float *>(p.X) + row * p.ldx + k);
        const ulonglong2 a = src[0], b = src[1];
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    } else if constexpr (kSrc == kF16) {
        widen8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.X) + row * p.ldx + k), f);
    } else {
        const uint16_t *src = static_cast<const uint16_t *>(p.X) + row * p.ldx + k;
        const uint4 g = *reinterpret_cast<const uint4 *>(src), u = *reinterpret_cast<const uint4 *>(src + p.K);
        swiglu8(g, u, f);
    }
}

// What the codes of a row need: its scale and the reciprocal, with the sign
// that the values carry.  A scale below fp32's normal range has no usable
// reciprocal: NaN sends every value to the IEEE quotient.
template <int kSrc>
struct RowScale {
    static constexpr float kSign = kSrc == kSwiglu ? -1.0f : 1.0f;
    float s, inv;
    __device__ explicit RowScale(float amax) {
        s = __fdiv_rn(amax, 127.0f);
        inv = s >= 1.17549435e-38f ? __fdiv_rn(kSign, s) : __int_as_float(0x7fffffff);
    }
};

// The IEEE quotient v / (kSign s), clamped to the levels.  Of an infinity, whose
// row has an infinite scale, the quotient is NaN, which fminf turns into the
// last level.
template <int kSrc>
__device__ __forceinline__ float level(float v, float s) {
    return copysignf(fminf(__fdiv_rn(fabsf(v), s), 127.0f), RowScale<kSrc>::kSign * v);
}

// The codes of eight values, as two words.  x / s is formed as x fl(1/s),
// within 2^-15 of the quotient for |x / s| <= 128, and rounded by adding
// 1.5 2^23; where the product lies within 2^-13 of a half-integer (or is not
// finite) the IEEE quotient decides.  (Elsewhere no code passes 127: the
// largest value over a normal s is within 2^-16 of 127.)
template <int kSrc>
__device__ __forceinline__ uint2 codes8(const uint64_t (&f)[4], const RowScale<kSrc> &rs) {
    constexpr float kMagic = 12582912.0f;
    if (!(rs.s > 0.0f)) return make_uint2(0u, 0u);   // a row of zeros, or with a NaN
    const uint64_t magic = f32x2(kMagic, kMagic), inv = f32x2(rs.inv, rs.inv);
    uint32_t b[8];
    bool safe = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t r = f32x2_mul(f[i], inv), t = f32x2_add(r, magic);
        const float2 off = f32x2_parts(f32x2_sub(r, f32x2_sub(t, magic)));
        safe = safe && fabsf(off.x) < 0.5f - 0x1p-13f && fabsf(off.y) < 0.5f - 0x1p-13f;
        const float2 tv = f32x2_parts(t);
        b[2 * i] = __float_as_uint(tv.x);
        b[2 * i + 1] = __float_as_uint(tv.y);
    }
    if (!safe) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = f32x2_parts(f[i]);
            b[2 * i] = __float_as_uint(__fadd_rn(level<kSrc>(v.x, rs.s), kMagic));
            b[2 * i + 1] = __float_as_uint(__fadd_rn(level<kSrc>(v.y, rs.s), kMagic));
        }
    }
    uint2 out;
    out.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    out.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return out;
}

// The largest of m, |a| and |b|; a NaN among them gives NaN (fmaxf would drop it).
__device__ __forceinline__ float max_abs_nan(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_abs(const uint64_t (&f)[4], float m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = f32x2_parts(f[i]);
        m = max_abs_nan(m, v.x, v.y);
    }
    return m;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int TPR>
__device__ __forceinline__ float row_max(float v, float *sh) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, d));
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v = max_nan(v, sh[i]);
    }
    return v;
}

template <int TPR>
__device__ __forceinline__ int row_sum(int v, int *sh) {
    v = __reduce_add_sync(0xffffffffu, v);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v += sh[i];
    }
    return v;
}

// Threads of a block: one row of TPR threads, or eight rows of a warp each.
template <int TPR>
constexpr int kBlock = TPR == 32 ? 256 : TPR;

// V > 0: the row's K <= 8 TPR V values stay in registers.  V == 0: any K,
// the row is read twice (the second time from the caches).  kFirst: all of a
// thread's loads are issued before any arithmetic, which pays for the SwiGLU's
// long arithmetic with few rows or very many (128 x 13696: 6.2 -> 4.4 us, 2048
// x 13696: 47.2 -> 40.8) and not where its registers cost a wave of blocks (512
// x 13696: 12.6 -> 15.1; the plain quantizer, 4096 x 13696 fp16: 35.8 -> 45.7).
// Rows brought ahead into shared memory by a producer thread were no faster
// (2048 x 13696: 44.6).  Of kFirst with 256 threads three blocks share an SM up to
// V = 7, where the compiler by itself takes registers for two (2048 rows of 10240:
// 26.7 us with the bound, 33.1 without; 12288: 31.3, 38.6; 13696, with 24 bytes of
// spills: 40.8, 42.9); V = 8 would spill more than that gives (16384: 50.4, 50.1).
template <int kSrc, int TPR, int V, bool kFirst>
__global__ void __launch_bounds__(kBlock<TPR>, kFirst && TPR == 256 && V >= 5 && V <= 7 ? 3 : 0) quantize_tokens_kernel(const __grid_constant__ Params p) {
    __shared__ float sh_max[TPR / 32];
    __shared__ int sh_sum[TPR / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = TPR == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (row >= p.M) return;   // whole warps
    const int64_t k0 = 8 * (TPR == 32 ? (int)(threadIdx.x & 31) : (int)threadIdx.x);
    constexpr int kStep = 8 * TPR;
    float amax = 0.0f;
    int8_t *dst = p.q + row * p.ldq;
    int sum = 0;
    if constexpr (V > 0) {
        uint64_t f[V][4];
        if constexpr (kFirst) {
            static_assert(kSrc == kSwiglu, "long arithmetic");
            const uint16_t *src = static_cast<const uint16_t *>(p.X) + row * p.ldx + k0;
            uint4 g[V], u[V];
#pragma unroll
            for (int c = 0; c < V; ++c) {
                if (k0 + c * kStep < p.K) {
                    g[c] = *reinterpret_cast<const uint4 *>(src + c * kStep);
                    u[c] = *reinterpret_cast<const uint4 *>(src + p.K + c * kStep);
                }
            }
#pragma unroll
            for (int c = 0; c < V; ++c) {
                if (k0 + c * kStep < p.K) {
                    swiglu8(g[c], u[c], f[c]);
                    amax = max_abs(f[c], amax);
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c) {
                if (k0 + c * kStep < p.K) {
                    load8<kSrc>(p, row, k0 + c * kStep, f[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[c][i] = 0;
                }
            }
#pragma unroll
            for (int c = 0; c < V; ++c) amax = max_abs(f[c], amax);
        }
        const RowScale<kSrc> rs(row_max<TPR>(amax, sh_max));
#pragma unroll
        for (int c = 0; c < V; ++c) {
            if (k0 + c * kStep < p.K) {
                const uint2 w = codes8<kSrc>(f[c], rs);
                *reinterpret_cast<uint2 *>(dst + k0 + c * kStep) = w;
                sum = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, sum));
            }
        }
        sum = row_sum<TPR>(sum, sh_sum);
        if (k0 == 0) {
            p.scales[row] = rs.s;
            p.sums[row] = sum;
        }
    } else {
        uint64_t f[4];
        for (int64_t k = k0; k < p.K; k += kStep) {
            load8<kSrc>(p, row, k, f);
            amax = max_abs(f, amax);
        }
        const RowScale<kSrc> rs(row_max<TPR>(amax, sh_max));
        for (int64_t k = k0; k < p.K; k += kStep) {
            load8<kSrc>(p, row, k, f);
            const uint2 w = codes8<kSrc>(f, rs);
            *reinterpret_cast<uint2 *>(dst + k) = w;
            sum = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, sum));
        }
        sum = row_sum<TPR>(sum, sh_sum);
        if (k0 == 0) {
            p.scales[row] = rs.s;
            p.sums[row] = sum;
        }
    }
}

}  // namespace tokens
}  // namespace w8
