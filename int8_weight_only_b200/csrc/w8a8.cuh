// W8A8 linear: Y[m,n] = s_m s_n sum_k x[m,k] (w[k,n] - z_n) + bias_n with int8
// activations x (scale s_m per token) and int8 weights w (scale s_n and zero
// point z_n per channel), one weight or one per group of tokens (experts).
//
// The packed weight tile holds the bytes u = w + 128 of 128 channels x 64
// features as rows of 64 bytes in the 64-byte-swizzle order, so a tile copied
// to shared memory is an operand of the 8-bit integer tensor-core product as
// it stands: A (unsigned, the 128 channels), B (signed, the tokens), exact
// sums in 32-bit integers in tensor memory.  No weight is ever converted:
//   sum_k x (w - z) = sum_k x u - (128 + z) sum_k x
// and sum_k x, one integer per token, comes with the activations.
//
// Work: the 8 KB weight tiles of all output tiles (128 channels x TN tokens),
// numbered output tile by output tile, are split evenly over the thread
// blocks, so a block's share is a run of consecutive tiles and at most its
// first and last output tile are shared with other blocks.  Shared output
// tiles meet in the workspace: each block stores its 32-bit integer part, the
// last to arrive adds the parts.  Integer sums: the order changes nothing.
//
// Roles: warp 0 producer (weight tiles by one bulk copy, tokens by TMA),
// warp 1 issues the products, warp 2 owns the tensor memory, warps 4-7 scale
// and store.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace w8 {
namespace w8a8 {

constexpr int kBN = 128;                 // channels of an output tile
constexpr int kTile = 8192;              // packed weight tile, 128 x 64
constexpr int kStep = 4;                 // weight tiles per stage (256 features)
constexpr int kWBytes = kStep * kTile;
// Weight tiles that a block gets at least, unless output tiles would then
// share a block: sharing an output tile costs 2-3 us, a run of 16 tiles 1.5 us
// (1 x 1024 x 1024: 9.9 us with runs of one tile, 6.0 with 4, 4.2 with 16;
// 128 x 2048 x 2048: 17.9, 15.1, 10.0, and 7.3 with 32).
constexpr int kMinRun = 32;
// Weight tiles that a block brings into L2 ahead of the previous kernel's end
// (1 x 4096 x 27392: 23.6 us with 1, 21.9 with 16, 21.6 with 32; 4 stages of
// 256 features: 6 stages take 1 us more).
constexpr int kPrefetch = 32;
constexpr int kMaxGroups = 1024;

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
    int32_t *partials;         // [blocks][2 slots][TN][128]
    int *counters;             // [blocks], zero between calls
    int64_t rows;
    int64_t N;
    int groups;
    int NB;                    // ceil(N / 128)
    int KB;                    // ceil(K / 64)
};

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
    for (int e = threadIdx.x; e <= p.groups; e += kThreads_) g.first[e] = (int)max64(0, min64(p.rows, __ldcg(p.offsets + e)));
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

// A run of weight tiles of one output tile.
struct Seg {
    int group, nb, tt;
    int kb0, kb1;
    int64_t unit;      // the output tile's number
};

template <int TN, bool kGrouped>
struct Sched {
    const Groups *g;
    int NB, KB;
    int tt_all;             // token tiles when there is one group
    int64_t it, end, unit;
    int kb, group;
    __device__ Sched(const Params &p, const Groups *groups, int64_t items, int64_t G) : g(groups), NB(p.NB), KB(p.KB) {
        const int64_t c = min64(blockIdx.x, G);   // blocks past G: an empty run
        tt_all = kGrouped ? 0 : (int)((p.rows + TN - 1) / TN);
        it = c * items / G;
        end = c < G ? (c + 1) * items / G : it;
        unit = it / KB;
        kb = (int)(it - unit * KB);
        group = 0;
    }
    __device__ bool next(Seg &s) {
        if (it >= end) return false;
        int64_t local = unit;
        int tt_n = tt_all;
        if constexpr (kGrouped) {
            while (unit >= (int64_t)NB * g->tiles[group + 1]) ++group;
            local -= (int64_t)NB * g->tiles[group];
            tt_n = g->tiles[group + 1] - g->tiles[group];
        }
        s.group = group;
        s.nb = (int)(local / tt_n);
        s.tt = (int)(local - (int64_t)s.nb * tt_n);
        s.unit = unit;
        s.kb0 = kb;
        s.kb1 = (int)min64(KB, kb + (end - it));
        it += s.kb1 - s.kb0;
        kb = 0;
        ++unit;
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
    __shared__ int last_sh;
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
    if constexpr (kGrouped) groups = reinterpret_cast<const Groups *>(&groups_sh);
    // the weight tiles of all output tiles
    auto count = [&]() -> int64_t {
        if constexpr (kGrouped)
            return (int64_t)groups->tiles[p.groups] * p.NB * p.KB;
        else
            return (p.rows + TN - 1) / TN * p.NB * p.KB;
    };
    // blocks with work: every one of them has at least one weight tile, and
    // kMinRun of them unless that would leave output tiles to share a block
    auto blocks = [&](int64_t items) -> int64_t {
        return max64(1, min64(gridDim.x, max64(items / p.KB, items / kMinRun)));
    };
    // The first weights into L2 while the previous kernel ends; they are never
    // stale there, whoever writes them.  The offsets may still be written:
    // here they are only a guess at what to bring, read past L1, and read
    // again below.
    if constexpr (kGrouped) {
        load_groups<TN, C::kThreads>(p, *reinterpret_cast<Groups *>(&groups_sh));
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const int64_t items = count();
        Sched<TN, kGrouped> sched(p, groups, items, blocks(items));
        Seg sg;
        if (sched.next(sg))
            prefetch_l2(p.packed + (((int64_t)sg.group * p.NB + sg.nb) * p.KB + sg.kb0) * kTile,
                        (uint32_t)min(sg.kb1 - sg.kb0, kPrefetch) * kTile);
    }
    if constexpr (kGrouped) {
        pdl_wait();
        __syncthreads();   // the guess has been read
        load_groups<TN, C::kThreads>(p, *reinterpret_cast<Groups *>(&groups_sh));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    const int64_t items = count(), G = blocks(items);
    // rows of a segment's token tile: the first, and how many of the group's
    auto rows_of = [&](const Seg &s, int64_t &row0) -> int {
        int64_t first = 0, end = p.rows;
        if constexpr (kGrouped) {
            first = groups->first[s.group];
            end = groups->first[s.group + 1];
        }
        row0 = first + (int64_t)s.tt * TN;
        return (int)min64(TN, end - row0);
    };

    if (warp == 0) {
        // ---------------------------------------------------- producer
        if (lane == 0) {
            pdl_wait();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            Sched<TN, kGrouped> sched(p, groups, items, G);
            Seg sg;
            while (ok && sched.next(sg)) {
                int64_t row0;
                rows_of(sg, row0);
                const uint8_t *w = p.packed + ((int64_t)sg.group * p.NB + sg.nb) * p.KB * kTile;
                for (int kb = sg.kb0; kb < sg.kb1; kb += kStep) {
                    const int cnt = min(kStep, sg.kb1 - kb), boxes = (cnt + 1) >> 1;
                    if (!mbar_wait(&empty[st], ph ^ 1u, SITE_I8_EMPTY)) { ok = false; break; }
                    uint8_t *ws = ring + st * C::kStageBytes, *xs = ws + kWBytes;
                    mbar_arrive_expect_tx(&full[st], cnt * kTile + boxes * C::kXBox);
                    bulk_g2s(ws, w + (int64_t)kb * kTile, cnt * kTile, &full[st]);
                    for (int b = 0; b < boxes; ++b)
                        tma_load_2d(xs + b * C::kXBox, &tmap_x, (kb + 2 * b) * 64, (int)row0, &full[st]);
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
        int st = 0, d = 0;
        uint32_t ph = 0, dph = 0;
        bool ok = true;
        const uint64_t w_desc0 = smem_desc_kmajor_sw64(smem_u32(ring));
        const uint64_t x_desc0 = smem_desc_kmajor_sw128(smem_u32(ring) + kWBytes);
        Sched<TN, kGrouped> sched(p, groups, items, G);
        Seg sg;
        while (ok && sched.next(sg)) {
            int64_t row0;
            const int n = (rows_of(sg, row0) + 15) & ~15;
            const uint32_t idesc = idesc_u8_s8_s32(kBN, n);
            const uint32_t dst = tmem + d * TN;
            if (!warp_all(mbar_wait(&d_empty[d], dph ^ 1u, SITE_I8_DEMPTY))) { ok = false; break; }
            tc_fence_after();
            uint32_t acc = 0;
            for (int kb = sg.kb0; kb < sg.kb1; kb += kStep) {
                const int cnt = min(kStep, sg.kb1 - kb);
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
        Sched<TN, kGrouped> sched(p, groups, items, G);
        Seg sg;
        while (sched.next(sg)) {
            int64_t row0;
            const int nr = rows_of(sg, row0);
            const int64_t n = (int64_t)sg.nb * kBN + r;
            const bool n_ok = n < p.N;
            const int64_t ch = (int64_t)sg.group * p.N + n;
            const float sc = n_ok ? __half2float(__ushort_as_half(p.scales[ch])) : 0.0f;
            const float bi = (n_ok && p.bias) ? __half2float(__ushort_as_half(p.bias[ch])) : 0.0f;
            const int off = 128 + ((n_ok && p.zeros) ? (int)p.zeros[ch] : 0);
            // the tokens' sums and scales, read while the products run; the
            // other buffer may still be read for the tile before
            if (const int c = threadIdx.x - 128; c < TN) {
                sum_sh[d][c] = c < nr ? __ldg(p.x_sums + row0 + c) : 0;
                xs_sh[d][c] = c < nr ? __ldg(p.x_scales + row0 + c) : 0.0f;
            }
            uint16_t *const y0 = p.Y + row0 * p.N + n;
            auto store = [&](const uint32_t (&v)[kChunk], int c0) {
                store_tokens(v, &sum_sh[d][c0], &xs_sh[d][c0], off, sc, bi, y0 + c0 * p.N, p.N, n_ok ? nr - c0 : 0);
            };
            const int c_end = min(nr, cb + C::kEpiTokens);
            const uint32_t src = tmem + ((uint32_t)(32 * q4) << 16) + d * TN;
            // A block's part of a shared output tile: [4 tokens][channel][4],
            // 16 bytes a thread.  Slot 0 is of the tile that the block's run
            // begins in, slot 1 of the one it ends in.
            auto part_at = [&](int64_t j, int c0) {
                const int64_t begin = j * items / G;
                return reinterpret_cast<int4 *>(p.partials + (j * 2 + (begin / p.KB == sg.unit ? 0 : 1)) * (TN * kBN) +
                                                c0 * kBN + 4 * r);
            };
            // blocks that share this output tile: the owners of its first to
            // last weight tile; the first one's counter is the tile's
            const bool whole = sg.kb0 == 0 && sg.kb1 == p.KB;
            int64_t j0 = 0, j1 = 0;
            if (!whole) {
                const int64_t it0 = sg.unit * p.KB;
                j0 = ((it0 + 1) * G - 1) / items;
                j1 = ((it0 + p.KB) * G - 1) / items;
            }
            int *const cnt = p.counters + j0;
            // all epilogue warps give up together: they meet at barriers
            // below (this one also shows them the sums and scales)
            if (!named_bar_all(1, kEpi, mbar_wait(&d_full[d], dph, SITE_I8_DFULL))) break;
            tc_fence_after();
            // The block that a tile begins in ends its run with it; the
            // others often had theirs done long before, at the start of
            // their runs.  Then it finishes the tile from tensor memory and
            // stores no part of its own.
            bool finish = whole;
            if (!whole && sg.kb0 == 0) {
                if (threadIdx.x == 128) {
                    const int all = ld_acquire_gpu(cnt) == (int)(j1 - j0);
                    if (all) *cnt = 0;
                    last_sh = all;
                }
                named_bar_sync(1, kEpi);
                finish = last_sh;
            }
            if (!finish) {
                for (int c0 = cb; c0 < c_end; c0 += kChunk) {
                    uint32_t v[kChunk];
                    if constexpr (kChunk == 32) tmem_load_32(src + c0, v); else tmem_load_16(src + c0, v);
                    int4 *const mine = part_at(blockIdx.x, c0);
#pragma unroll
                    for (int i = 0; i < kChunk / 4; ++i)
                        __stcg(mine + i * kBN, make_int4((int)v[4 * i], (int)v[4 * i + 1], (int)v[4 * i + 2], (int)v[4 * i + 3]));
                }
                named_bar_sync(1, kEpi);   // the part is written (and last_sh read)
                if (threadIdx.x == 128) {
                    const int last = atomic_add_acq_rel_gpu(cnt, 1) == (int)(j1 - j0);
                    if (last) *cnt = 0;
                    last_sh = last;
                }
                named_bar_sync(1, kEpi);
                finish = last_sh;
            }
            if (finish) {
                for (int c0 = cb; c0 < c_end; c0 += kChunk) {
                    uint32_t v[kChunk];
                    if constexpr (kChunk == 32) tmem_load_32(src + c0, v); else tmem_load_16(src + c0, v);
                    if (!whole) {
                        // the others' parts, several blocks' loads in flight
                        constexpr int kAhead = TN >= 64 ? 2 : TN == 32 ? 3 : 6;
                        for (int64_t j = j0; j <= j1; j += kAhead) {
                            int4 t[kAhead][kChunk / 4];
#pragma unroll
                            for (int a = 0; a < kAhead; ++a) {
                                const bool there = j + a <= j1 && j + a != blockIdx.x;
                                const int4 *const theirs = part_at(there ? j + a : j0, c0);
#pragma unroll
                                for (int i = 0; i < kChunk / 4; ++i)
                                    t[a][i] = there ? __ldcg(theirs + i * kBN) : make_int4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int a = 0; a < kAhead; ++a)
#pragma unroll
                                for (int i = 0; i < kChunk / 4; ++i) {
                                    v[4 * i] += (uint32_t)t[a][i].x;
                                    v[4 * i + 1] += (uint32_t)t[a][i].y;
                                    v[4 * i + 2] += (uint32_t)t[a][i].z;
                                    v[4 * i + 3] += (uint32_t)t[a][i].w;
                                }
                        }
                    }
                    store(v, c0);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_empty[d]);
            if (!whole) named_bar_sync(1, kEpi);   // last_sh is read by all
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
