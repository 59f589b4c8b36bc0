// Per-token int8 quantization of activations: for every row m of X [M, K]
//   s_m = max_k |X[m,k]| / 127,  q[m,k] = clamp(rne(X[m,k] / s_m), -127, 127),
//   sum_m = sum_k q[m,k]
// in IEEE fp32 (s_m = 0 gives q = 0), and the same for the SwiGLU of a gated
// MLP's first product, h = g / (1 + exp(-g)) * u.  The row sums let the
// int8 linear undo the offset of the weight codes.
//
// One pass over X: a row is spread over TPR threads, each of which holds its
// values in registers between the row maximum and the rounding.  Bound by
// HBM for many rows and by latency for few.
#pragma once

#include "common.cuh"

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

__device__ __forceinline__ void widen8(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// Eight consecutive values of a row, from element k.
template <int kSrc>
__device__ __forceinline__ void load8(const Params &p, int64_t row, int64_t k, float (&f)[8]) {
    if constexpr (kSrc == kF32) {
        const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.X) + row * p.ldx + k);
        const float4 a = __ldg(src), b = __ldg(src + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        const uint16_t *src = static_cast<const uint16_t *>(p.X) + row * p.ldx + k;
        widen8(__ldg(reinterpret_cast<const uint4 *>(src)), f);
        if constexpr (kSrc == kSwiglu) {
            float u[8];
            widen8(__ldg(reinterpret_cast<const uint4 *>(src + p.K)), u);
            // every step one IEEE operation: the same values as an
            // elementwise formula in fp32
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fdiv_rn(f[i], 1.0f + expf(-f[i])), u[i]);
        }
    }
}

// The codes of eight values, as two words.  x / s is formed as x fl(1/s),
// within 2^-15 of the quotient for |x / s| <= 128, and rounded by adding
// 1.5 2^23; where the product lies within 2^-13 of a half-integer (or is not
// finite) the IEEE quotient decides.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s, float inv) {
    constexpr float kMagic = 12582912.0f;
    float t[8];
    bool near_half = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = __fmul_rn(f[i], inv);
        t[i] = __fadd_rn(r, kMagic);
        near_half |= !(fabsf(__fsub_rn(r, __fsub_rn(t[i], kMagic))) < 0.5f - 0x1p-13f);
    }
    if (near_half) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __fadd_rn(fminf(fmaxf(__fdiv_rn(f[i], s), -127.0f), 127.0f), kMagic);
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fminf(fmaxf(t[i], kMagic - 127.0f), kMagic + 127.0f));
    uint2 out;
    out.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    out.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return out;
}

template <int TPR>
__device__ __forceinline__ float row_max(float v, float *sh) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TPR / 32; ++i) v = fmaxf(v, sh[i]);
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
// the row is read twice (the second time from the caches).
template <int kSrc, int TPR, int V>
__global__ void __launch_bounds__(kBlock<TPR>) quantize_tokens_kernel(const __grid_constant__ Params p) {
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
        float f[V][8];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            if (k0 + c * kStep < p.K) {
                load8<kSrc>(p, row, k0 + c * kStep, f[c]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[c][i] = 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[c][i]));
        amax = row_max<TPR>(amax, sh_max);
        const float s = __fdiv_rn(amax, 127.0f);
        const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            if (k0 + c * kStep < p.K) {
                const uint2 w = s > 0.0f ? codes8(f[c], s, inv) : make_uint2(0u, 0u);
                *reinterpret_cast<uint2 *>(dst + k0 + c * kStep) = w;
                sum = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, sum));
            }
        }
        sum = row_sum<TPR>(sum, sh_sum);
        if (k0 == 0) {
            p.scales[row] = s;
            p.sums[row] = sum;
        }
    } else {
        float f[8];
        for (int64_t k = k0; k < p.K; k += kStep) {
            load8<kSrc>(p, row, k, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
        }
        amax = row_max<TPR>(amax, sh_max);
        const float s = __fdiv_rn(amax, 127.0f);
        const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
        for (int64_t k = k0; k < p.K; k += kStep) {
            load8<kSrc>(p, row, k, f);
            const uint2 w = s > 0.0f ? codes8(f, s, inv) : make_uint2(0u, 0u);
            *reinterpret_cast<uint2 *>(dst + k) = w;
            sum = __dp4a((int)w.x, 0x01010101, __dp4a((int)w.y, 0x01010101, sum));
        }
        sum = row_sum<TPR>(sum, sh_sum);
        if (k0 == 0) {
            p.scales[row] = s;
            p.sums[row] = sum;
        }
    }
}

}  // namespace tokens
}  // namespace w8
