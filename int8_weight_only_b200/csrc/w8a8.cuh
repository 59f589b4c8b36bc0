// W8A8 linear: Y[m,n] = s_m s_n sum_k x[m,k] (w[k,n] - z_n) + bias_n with int8
// activations x (scale s_m per token) and int8 weights w (scale s_n and zero
// point z_n per channel), one weight or one for each group of tokens (experts).
//
// The packed weight tile holds the bytes u = w + 128 of 128 channels x 64
// features as rows of 64 bytes in the 64-byte-swizzle order, so a tile copied
// to shared memory is an operand of the 8-bit integer tensor-core product as
// it stands: A (unsigned, the 128 channels), B (signed, the tokens), exact
// sums in 32-bit integers in tensor memory.  No weight is ever converted:
//   sum_k x (w - z) = sum_k x u - (128 + z) sum_k x
// and sum_k x, one integer per token, comes with the activations.
//
// This kernel: whole output tiles of 128 channels x TN tokens dealt round robin
// to the thread blocks, for few tokens and for products of about one wave of
// tiles (512 x 4096 x 4096: 10.4 us, on pairs of SMs 14.4).  With few tokens it
// is bound by the weight stream (1 x 4096 x 27392: 18.3 us, 6.1 TB/s, 94 % of the
// measured copy rate), which 94 of 148 SMs already draw at 5.7 TB/s, so sharing
// output tiles to occupy all SMs does not pay: an even split over K, the parts
// added through a workspace, took 21.7 us for 1 x 4096 x 27392 (107 blocks with
// two tiles each), and against a first form of whole tiles 14.7 to 12.0 for 1 x
// 4096 x 13696 and 31.4 to 29.0 for 1 x 13696 x 12000.  Few output tiles with a
// long K go to clusters (w8a8_cluster.cuh).  Groups of few tokens (kGrouped) run
// here too, their tiles counted on the device (8 groups of 2 x 4096 x 4096: 22 us).
//
// Roles: warp 0 producer (weight tiles by one bulk copy, tokens by TMA),
// warp 1 issues the products, warp 2 owns the tensor memory, warps 4 and up
// scale and store.
#pragma once

#include <type_traits>

#include "i8.cuh"

namespace w8 {
namespace w8a8 {

constexpr int kBN = 128;                 // channels of an output tile
constexpr int kTile = 8192;              // packed weight tile, 128 x 64
constexpr int kStep = 4;                 // weight tiles per stage (256 features)
constexpr int kWBytes = kStep * kTile;
// Weight tiles that a block brings into L2 ahead of the previous kernel's end
// (1 x 4096 x 27392: 18.7 us with 1, 18.5 with 16, 19.3 with 32).
constexpr int kPrefetch = 16;

template <int TN>
struct Cfg {
    static constexpr int kXBox = TN * 128;                   // TN tokens x 128 features
    static constexpr int kXBytes = (kStep / 2) * kXBox;
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = TN <= 64 ? 4 : 3;
    static constexpr int kSmemBytes = kStages * kStageBytes + 1024;
    static constexpr uint32_t kTmemCols = 2 * TN < 32 ? 32 : 2 * TN;
    // four warps read the 128 channels; from 64 tokens on two sets of them
    // share the tokens
    static constexpr int kEpiWarps = TN >= 64 ? 8 : 4;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    static constexpr int kEpiTokens = TN / (kEpiWarps / 4);
    static constexpr int kChunk = TN >= 32 ? 32 : 16;        // tokens scaled at a time
    static_assert(kXBox % 1024 == 0, "swizzle alignment");
    static_assert(kSmemBytes <= 217 * 1024, "shared memory budget");
};

struct Params {
    const uint8_t *packed;     // [groups] packed weights
    const uint16_t *scales;    // [groups][N]
    const int8_t *zeros;       // [groups][N] or null
    const uint16_t *bias;      // [groups][N] or null
    const float *x_scales;     // [rows]
    const int32_t *x_sums;     // [rows]
    const int32_t *offsets;    // [groups + 1] first rows of the groups, or null: one group of all rows
    uint16_t *Y;               // [rows][N]
    int64_t rows;
    int64_t N;
    int groups;
    int NB;                    // ceil(N / 128)
    int KB;                    // ceil(K / 64)
};

constexpr int kMaxGroups = 1024;
// The groups' rows and token tiles, in shared memory.
struct Groups {
    int first[kMaxGroups + 1];    // first row, within [0, rows]
    int tiles[kMaxGroups + 1];    // token tiles of all groups before
};
struct OneGroup {};

// All kThreads_ threads of the block; a block barrier has to follow.  The
// first rows are clamped to [0, rows], so no offset can lead out of bounds.
template <int TN, int kThreads_>
__device__ __forceinline__ void load_groups(const Params &p, Groups &g) {
    for (int e = threadIdx.x; e <= p.groups; e += kThreads_) g.first[e] = (int)max64(0, min64(p.rows, p.offsets[e]));
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int before = 0;
        if (lane == 0) g.tiles[0] = 0;
        for (int e0 = 0; e0 < p.groups; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.groups) n = (max(0, g.first[e + 1] - g.first[e]) + TN - 1) / TN;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, n, d);
                if (lane >= d) n += o;
            }
            if (e < p.groups) g.tiles[e + 1] = before + n;
            before += __shfl_sync(0xffffffffu, n, 31);
        }
    }
}

// Output tiles dealt round robin to as few blocks as keep the longest run of
// tiles short: equally many each draw the weights evenly.  One group: tile u is
// channel block u / tt_n, token tile u % tt_n.  Several: those of a group
// follow one another.
struct Tile {
    int group, nb;
    int64_t row0;
    int rows;
};
template <int TN, bool kGrouped>
struct Deal {
    const Params &p;
    const Groups *g;
    int u, units, step, group;
    __device__ Deal(const Params &p_, const Groups *groups) : p(p_), g(groups), u(blockIdx.x), group(0) {
        // the host keeps the tiles of a call below 2^31, whatever overlapping
        // groups would add up to
        const int64_t all = kGrouped ? (int64_t)groups->tiles[p.groups] * p.NB : (p.rows + TN - 1) / TN * p.NB;
        units = (int)min64(all, INT32_MAX / 2);
        step = gridDim.x;
        if constexpr (kGrouped) {
            // (the host has sized the grid so where it knows the tiles)
            const unsigned each = ((unsigned)units + gridDim.x - 1) / gridDim.x;
            if (each > 0) step = (int)(((unsigned)units + each - 1) / each);
            if (u >= step) u = units;
        }
    }
    __device__ bool next(Tile &t) {
        if (u >= units) return false;
        int local = u, tt_n;
        int64_t first = 0, end = p.rows;
        if constexpr (kGrouped) {
            while ((int64_t)u >= (int64_t)p.NB * g->tiles[group + 1]) ++group;
            local -= p.NB * g->tiles[group];
            tt_n = g->tiles[group + 1] - g->tiles[group];
            first = g->first[group];
            end = g->first[group + 1];
        } else {
            tt_n = (int)((p.rows + TN - 1) / TN);
        }
        t.group = group;
        t.nb = local / tt_n;
        t.row0 = first + (int64_t)(local - t.nb * tt_n) * TN;
        t.rows = (int)min64(TN, end - t.row0);
        u += step;
        return true;
    }
};

// The outputs of C tokens (columns) of this thread's channel, as pairs of
// tokens: y = s_m s_n (sum - off sum_m) + bias, rounded once to fp16.  sums
// and x_scales (shared memory, 16-byte aligned) belong to the tokens.
template <int C>
__device__ __forceinline__ void scale_tokens(const uint32_t (&v)[C], const int *sums, const float *x_scales, int off,
                                             float sc, float bi, uint32_t (&h)[C / 2]) {
    const uint64_t sc2 = f32x2(sc, sc), bi2 = f32x2(bi, bi);
#pragma unroll
    for (int i = 0; i < C; i += 4) {
        const int4 s4 = *reinterpret_cast<const int4 *>(sums + i);
        const ulonglong2 x4 = *reinterpret_cast<const ulonglong2 *>(x_scales + i);
        const uint64_t ab = f32x2((float)((int)v[i] - off * s4.x), (float)((int)v[i + 1] - off * s4.y));
        const uint64_t cd = f32x2((float)((int)v[i + 2] - off * s4.z), (float)((int)v[i + 3] - off * s4.w));
        const float2 y0 = f32x2_parts(f32x2_fma(f32x2_mul(ab, x4.x), sc2, bi2));
        const float2 y1 = f32x2_parts(f32x2_fma(f32x2_mul(cd, x4.y), sc2, bi2));
        const __half2 h0 = __float22half2_rn(y0), h1 = __float22half2_rn(y1);
        h[i / 2] = *reinterpret_cast<const uint32_t *>(&h0);
        h[i / 2 + 1] = *reinterpret_cast<const uint32_t *>(&h1);
    }
}

// Scale and store: y points at the first token's output of this channel,
// rows of N apart; the first `left` tokens exist.  Whole runs of C tokens go
// in a straight line: with a test at every store the scaling took longer than
// the products of a short K.
template <int C>
__device__ __forceinline__ void store_tokens(const uint32_t (&v)[C], const int *sums, const float *x_scales, int off,
                                             float sc, float bi, uint16_t *y, int64_t N, int left) {
    uint32_t h[C / 2];
    scale_tokens(v, sums, x_scales, off, sc, bi, h);
    if (left >= C) {
#pragma unroll
        for (int i = 0; i < C; ++i) y[i * N] = (uint16_t)(i & 1 ? h[i / 2] >> 16 : h[i / 2]);
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < left) y[i * N] = (uint16_t)(i & 1 ? h[i / 2] >> 16 : h[i / 2]);
    }
}

template <int TN, bool kGrouped>
__global__ void __launch_bounds__(Cfg<TN>::kThreads, 1)
w8a8_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ Params p) {
    using C = Cfg<TN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[C::kStages], empty[C::kStages];
    __shared__ uint64_t d_full[2], d_empty[2], drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ __align__(16) int sum_sh[2][TN];       // the token tile's sums and scales
    __shared__ __align__(16) float xs_sh[2][TN];
    using GroupsSh = typename std::conditional<kGrouped, Groups, OneGroup>::type;
    __shared__ GroupsSh groups_sh;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // warp-uniform
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], C::kEpiWarps);
        }
        mbar_init(&drain, 1);
        fence_barrier_init();
        prefetch_tensormap(&tmap_x);
    }
    if (warp == 2) {
        tmem_alloc(&tmem_base_sh, C::kTmemCols);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    const Groups *groups = nullptr;
    if constexpr (kGrouped) {
        pdl_wait();
        load_groups<TN, C::kThreads>(p, *reinterpret_cast<Groups *>(&groups_sh));
        groups = reinterpret_cast<const Groups *>(&groups_sh);
    } else if (threadIdx.x == 0) {
        // the first weights into L2 while the previous kernel ends; they are
        // never stale there, whoever writes them
        Deal<TN, false> deal(p, nullptr);
        Tile t;
        if (deal.next(t)) prefetch_l2(p.packed + (int64_t)t.nb * p.KB * kTile, (uint32_t)min(p.KB, kPrefetch) * kTile);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    if (warp == 0) {
        // ---------------------------------------------------- producer
        if (lane == 0) {
            pdl_wait();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            Deal<TN, kGrouped> deal(p, groups);
            Tile t;
            while (ok && deal.next(t)) {
                const uint8_t *w = p.packed + ((int64_t)t.group * p.NB + t.nb) * p.KB * kTile;
                for (int kb = 0; kb < p.KB; kb += kStep) {
                    const int cnt = min(kStep, p.KB - kb), boxes = (cnt + 1) >> 1;
                    if (!mbar_wait(&empty[st], ph ^ 1u, SITE_I8_EMPTY)) { ok = false; break; }
                    uint8_t *ws = ring + st * C::kStageBytes, *xs = ws + kWBytes;
                    mbar_arrive_expect_tx(&full[st], cnt * kTile + boxes * C::kXBox);
                    bulk_g2s(ws, w + (int64_t)kb * kTile, cnt * kTile, &full[st]);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(xs + b * C::kXBox, &tmap_x, (kb + 2 * b) * 64, (int)t.row0, &full[st]);
                    ++issued;
                    if (++st == C::kStages) { st = 0; ph ^= 1u; }
                }
            }
            // every copy has landed before the block can leave
            for (int i = 0; i < C::kStages && i < issued; ++i) {
                if (--st < 0) { st = C::kStages - 1; ph ^= 1u; }
                mbar_wait(&full[st], ph, SITE_I8_DRAIN, 10000000ull);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- products
        // the whole warp walks the steps and one elected lane issues: the
        // operands stay in uniform registers
        pdl_wait();   // before the first bounded wait: its second is this call's own
        int st = 0, d = 0;
        uint32_t ph = 0, dph = 0;
        bool ok = true;
        const uint64_t w_desc0 = smem_desc_kmajor_sw64(smem_u32(ring));
        const uint64_t x_desc0 = smem_desc_kmajor_sw128(smem_u32(ring) + kWBytes);
        Deal<TN, kGrouped> deal(p, groups);
        Tile tile;
        while (ok && deal.next(tile)) {
            const int n = (tile.rows + 15) & ~15;
            const uint32_t idesc = idesc_u8_s8_s32(kBN, n);
            const uint32_t dst = tmem + d * TN;
            if (!warp_all(mbar_wait(&d_empty[d], dph ^ 1u, SITE_I8_DEMPTY))) { ok = false; break; }
            tc_fence_after();
            uint32_t acc = 0;
            for (int kb = 0; kb < p.KB; kb += kStep) {
                const int cnt = min(kStep, p.KB - kb);
                if (!warp_all(mbar_wait(&full[st], ph, SITE_I8_FULL))) { ok = false; break; }
                tc_fence_after();
                // descriptors count in units of 16 bytes; the sums stay within
                // the address field (shared memory < 256 KB)
                const uint64_t wd = w_desc0 + (uint32_t)st * (C::kStageBytes / 16);
                const uint64_t xd = x_desc0 + (uint32_t)st * (C::kStageBytes / 16);
                if (elect_one()) {
#pragma unroll
                    for (int t = 0; t < kStep; ++t) {
                        if (t < cnt) {
                            const uint64_t wt = wd + t * (kTile / 16), xt = xd + (t >> 1) * (C::kXBox / 16) + (t & 1) * 4;
                            tc_mma_ss_i8(dst, wt, xt, idesc, t == 0 ? acc : 1);
                            tc_mma_ss_i8(dst, wt + 2, xt + 2, idesc, 1);
                        }
                    }
                    tc_commit(&empty[st]);
                }
                __syncwarp();
                acc = 1;
                if (++st == C::kStages) { st = 0; ph ^= 1u; }
            }
            if (!ok) break;
            if (elect_one()) tc_commit(&d_full[d]);
            __syncwarp();
            if (++d == 2) { d = 0; dph ^= 1u; }
        }
        // every product is complete before the tensor memory is freed
        if (elect_one()) tc_commit(&drain);
        __syncwarp();
        mbar_wait(&drain, 0, SITE_I8_DRAIN);
    } else if (warp >= 4) {
        // ---------------------------------------------------- scale and store
        pdl_wait();
        constexpr int kEpi = 32 * C::kEpiWarps, kChunk = C::kChunk;
        const int q4 = warp & 3;
        const int r = 32 * q4 + lane;
        const int cb = C::kEpiTokens * ((warp - 4) >> 2);     // this warp's first token
        int d = 0;
        uint32_t dph = 0;
        Deal<TN, kGrouped> deal(p, groups);
        Tile tile;
        while (deal.next(tile)) {
            const int64_t row0 = tile.row0;
            const int nr = tile.rows;
            const int64_t n = (int64_t)tile.nb * kBN + r;
            const bool n_ok = n < p.N;
            const int64_t ch = (int64_t)tile.group * p.N + n;
            const float sc = n_ok ? __half2float(__ushort_as_half(p.scales[ch])) : 0.0f;
            const float bi = (n_ok && p.bias) ? __half2float(__ushort_as_half(p.bias[ch])) : 0.0f;
            const int off = 128 + ((n_ok && p.zeros) ? (int)p.zeros[ch] : 0);
            // the tokens' sums and scales, read while the products run; the
            // other buffer may still be read for the tile before
            if (const int c = threadIdx.x - 128; c < TN) {
                sum_sh[d][c] = c < nr ? p.x_sums[row0 + c] : 0;
                xs_sh[d][c] = c < nr ? p.x_scales[row0 + c] : 0.0f;
            }
            uint16_t *const y0 = p.Y + row0 * p.N + n;
            auto store = [&](const uint32_t (&v)[kChunk], int c0) {
                store_tokens(v, &sum_sh[d][c0], &xs_sh[d][c0], off, sc, bi, y0 + c0 * p.N, p.N, n_ok ? nr - c0 : 0);
            };
            const int c_end = min(nr, cb + C::kEpiTokens);
            const uint32_t src = tmem + ((uint32_t)(32 * q4) << 16) + d * TN;
            // all epilogue warps give up together (and see the sums and scales)
            if (!named_bar_all(1, kEpi, mbar_wait(&d_full[d], dph, SITE_I8_DFULL))) break;
            tc_fence_after();
            for (int c0 = cb; c0 < c_end; c0 += kChunk) {
                uint32_t v[kChunk];
                if constexpr (kChunk == 32) tmem_load_32(src + c0, v); else tmem_load_16(src + c0, v);
                store(v, c0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[d]);
            if (++d == 2) { d = 0; dph ^= 1u; }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace w8a8
}  // namespace w8
