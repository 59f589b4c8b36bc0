// W8A8 linear for many tokens, on pairs of SMs (tcgen05 cta_group::2): the
// product of w8a8.cuh with output tiles of 256 channels x up to 256 tokens.
// Each block of a cluster of two holds its own 128 channels of the weight and
// half of the tile's tokens in shared memory, so a 128-wide K step brings 32
// KB into each SM for 512 cycles of integer products; the 32-bit sums of two
// tiles fit in tensor memory, and a tile is scaled and stored while the next
// one runs.
//
// Schedule: whole tiles round robin over the pairs; where that leaves pairs
// idle in the last wave for long, the K steps of the last tiles are split
// evenly instead (integer parts, added by the last block to arrive).
//
// Roles in each block: warp 0 producer, warp 1 products (first block), warp 2
// tensor memory, warps 4-11 scale and store.
#pragma once

#include "w8a8.cuh"

namespace w8 {
namespace w8a8 {
namespace pair {

constexpr int kBT = 256;                     // tokens of a tile
constexpr int kStepTiles = 2;                // weight tiles per stage (128 features)
constexpr int kWBytes = kStepTiles * kTile;
constexpr int kXBytes = (kBT / 2) * 128;     // 128 tokens x 128 features
constexpr int kStageBytes = kWBytes + kXBytes;
constexpr int kStages = 6;
constexpr int kSmemBytes = kStages * kStageBytes + 1024;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kTmemCols = 2 * kBT;
constexpr int kPart = kBT * kBN;             // 32-bit sums of one block's share of a tile
constexpr uint16_t kBoth = 0x3;
// K steps per pair that splitting the last tiles has to save
constexpr int kSplitMin = 12;

struct Seg {
    int group, nbp, tt;
    int ks0, ks1;
    int tile;
    int slot;       // -1: the whole tile; else the slot of its part
};

// Tiles [0, dp) go round robin, the K steps of the others evenly over `pairs`.
struct Plan {
    int tiles, dp, pairs;
    int64_t steps;     // K steps of the split tiles
    __device__ Plan(int64_t n, int P, int KS) {
        tiles = (int)n;
        dp = tiles;
        pairs = P;
        steps = 0;
        const int64_t whole = (n + P - 1) / P * KS;
        const int64_t sk = n % P == 0 ? 0 : (n > P ? P + n % P : n);
        const int64_t split = (n - sk) / P * KS + (sk * KS + P - 1) / P;
        if (whole - split >= kSplitMin) {
            dp = (int)(n - sk);
            steps = sk * KS;
            pairs = (int)min64(P, steps);
        }
    }
    __device__ int64_t begin(int64_t q) const { return q * steps / pairs; }
    __device__ int owner(int64_t it) const { return (int)(((it + 1) * pairs - 1) / steps); }
    __device__ int slot(int q, int tile, int KS) const { return dp + (int)(begin(q) / KS) == tile ? 0 : 1; }
};

template <bool kGrouped>
struct Sched {
    const Groups *g;
    Plan plan;
    int NBP, KS, TT, tile, P, group;
    int64_t it, end;
    int q;
    __device__ Sched(const Params &p, const Groups *groups, const Plan &pl, int pair, int P_)
        : g(groups), plan(pl), NBP((p.NB + 1) / 2), KS((p.KB + 1) / 2), TT((int)((p.rows + kBT - 1) / kBT)), tile(pair),
          P(P_), group(0), q(pair) {
        it = end = 0;
        if (plan.steps > 0 && pair < plan.pairs) {
            it = plan.begin(pair);
            end = plan.begin(pair + 1);
        }
    }
    __device__ bool next(Seg &s) {
        if (tile < plan.dp) {
            s.tile = tile;
            s.ks0 = 0;
            s.ks1 = KS;
            s.slot = -1;
            tile += P;
        } else if (it < end) {
            const int t = (int)(it / KS);
            s.tile = plan.dp + t;
            s.ks0 = (int)(it - (int64_t)t * KS);
            s.ks1 = (int)min64(KS, s.ks0 + (end - it));
            s.slot = s.ks0 == 0 && s.ks1 == KS ? -1 : plan.slot(q, s.tile, KS);
            it += s.ks1 - s.ks0;
        } else {
            return false;
        }
        int local = s.tile, tt_n = TT;
        if constexpr (kGrouped) {
            while ((int64_t)s.tile >= (int64_t)NBP * g->tiles[group + 1]) ++group;
            local -= NBP * g->tiles[group];
            tt_n = g->tiles[group + 1] - g->tiles[group];
        }
        s.group = group;
        s.nbp = local / tt_n;
        s.tt = local - s.nbp * tt_n;
        return true;
    }
};

// grid = 2 x pairs blocks in clusters of two.  tmap_w: the packed weights as
// rows of 128 bytes, box 128 x 128 (two tiles), no swizzle; tmap_x: codes
// [rows, K], box 128 features x 128 rows, 128-byte swizzle.
template <bool kGrouped>
__global__ void __launch_bounds__(kThreads, 1)
w8a8_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                 const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint64_t d_full[2], d_empty[2], drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ int last_sh;
    __shared__ __align__(16) int sum_sh[2][kBT];
    __shared__ __align__(16) float xs_sh[2][kBT];
    using GroupsSh = typename std::conditional<kGrouped, Groups, OneGroup>::type;
    __shared__ GroupsSh groups_sh;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // warp-uniform
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair0 = blockIdx.x >> 1, P = gridDim.x >> 1;
    const int KS = (p.KB + 1) / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);            // first block: the bytes of both
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 2 * kEpiWarps);
        }
        mbar_init(&drain, 1);
        fence_barrier_init();
        prefetch_tensormap(&tmap_w);
        prefetch_tensormap(&tmap_x);
    }
    if (warp == 2) {
        tmem_alloc_pair(&tmem_base_sh, kTmemCols);
        tmem_relinquish_pair();
    }
    const Groups *groups = nullptr;
    if constexpr (kGrouped) {
        pdl_wait();
        load_groups<kBT, kThreads>(p, *reinterpret_cast<Groups *>(&groups_sh));
        groups = reinterpret_cast<const Groups *>(&groups_sh);
    }
    tc_fence_before();
    cluster_sync_all();
    pdl_launch_dependents();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    int64_t n_tiles;
    if constexpr (kGrouped) {
        n_tiles = (int64_t)groups->tiles[p.groups] * ((p.NB + 1) / 2);
    } else {
        n_tiles = (p.rows + kBT - 1) / kBT * ((p.NB + 1) / 2);
    }
    const Plan plan(n_tiles, P, KS);
    auto rows_of = [&](const Seg &s, int64_t &row0) -> int {
        int64_t first = 0, end = p.rows;
        if constexpr (kGrouped) {
            first = groups->first[s.group];
            end = groups->first[s.group + 1];
        }
        row0 = first + (int64_t)s.tt * kBT;
        return (int)min64(kBT, end - row0);
    };
    // tokens of the product: the tile's, rounded up so that each block holds
    // half of them
    auto width = [](int nr) -> int { return (nr + 31) & ~31; };
    auto leader = [](uint64_t *bar) -> uint32_t { return mapa_shared(smem_u32(bar), 0); };

    if (warp == 0) {
        // ---------------------------------------------------- producer
        if (lane == 0) {
            pdl_wait();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            Sched<kGrouped> sched(p, groups, plan, pair0, P);
            Seg sg;
            while (ok && sched.next(sg)) {
                int64_t row0;
                const int n = width(rows_of(sg, row0));
                const int64_t block = (int64_t)sg.group * p.NB + min(2 * sg.nbp + (int)rank, p.NB - 1);
                const int wrow = (int)(block * p.KB * (kTile / 128));
                const int xrow = (int)row0 + (int)rank * (n / 2);
                for (int ks = sg.ks0; ks < sg.ks1; ++ks) {
                    if (!mbar_wait(&empty[st], ph ^ 1u, SITE_I8_EMPTY)) { ok = false; break; }
                    uint8_t *ws = ring + st * kStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * kStageBytes);
                    tma_load_2d_pair(ws, &tmap_w, 0, wrow + ks * (kWBytes / 128), leader(&full[st]));
                    tma_load_2d_pair(ws + kWBytes, &tmap_x, ks * 128, xrow, leader(&full[st]));
                    ++issued;
                    if (++st == kStages) { st = 0; ph ^= 1u; }
                }
            }
            // every copy has landed before the pair can leave (the cluster
            // barrier below holds the second block until the first saw both
            // halves complete)
            if (rank == 0) {
                for (int i = 0; i < kStages && i < issued; ++i) {
                    if (--st < 0) { st = kStages - 1; ph ^= 1u; }
                    mbar_wait(&full[st], ph, SITE_I8_DRAIN, 10000000ull);
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- products
        // The whole warp walks the steps and one elected lane issues, so that
        // addresses and descriptors stay in uniform registers: with a branch
        // on the lane number a product took 256 cycles to issue instead of
        // the 128 it runs for (2048 x 4096 x 27392: 198 us).
        if (rank == 0) {
            int st = 0, d = 0;
            uint32_t ph = 0, dph = 0;
            bool ok = true;
            const uint64_t w_desc0 = smem_desc_kmajor_sw64(smem_u32(ring));
            const uint64_t x_desc0 = smem_desc_kmajor_sw128(smem_u32(ring) + kWBytes);
            Sched<kGrouped> sched(p, groups, plan, pair0, P);
            Seg sg;
            while (ok && sched.next(sg)) {
                int64_t row0;
                const uint32_t idesc = idesc_u8_s8_s32(2 * kBN, width(rows_of(sg, row0)));
                const uint32_t dst = tmem + d * kBT;
                if (!warp_all(mbar_wait(&d_empty[d], dph ^ 1u, SITE_I8_DEMPTY))) { ok = false; break; }
                tc_fence_after();
                uint32_t acc = 0;
                for (int ks = sg.ks0; ks < sg.ks1; ++ks) {
                    if (!warp_all(mbar_wait(&full[st], ph, SITE_I8_FULL))) { ok = false; break; }
                    tc_fence_after();
                    // descriptors count in units of 16 bytes; the sums stay
                    // within the address field (shared memory < 256 KB)
                    const uint64_t wd = w_desc0 + (uint32_t)st * (kStageBytes / 16);
                    const uint64_t xd = x_desc0 + (uint32_t)st * (kStageBytes / 16);
                    if (elect_one()) {
                        tc_mma_ss_i8_pair(dst, wd, xd, idesc, acc);
                        tc_mma_ss_i8_pair(dst, wd + 2, xd + 2, idesc, 1);
                        if (kStepTiles * ks + 1 < p.KB) {
                            tc_mma_ss_i8_pair(dst, wd + kTile / 16, xd + 4, idesc, 1);
                            tc_mma_ss_i8_pair(dst, wd + kTile / 16 + 2, xd + 6, idesc, 1);
                        }
                        tc_commit_pair_mc(&empty[st], kBoth);
                    }
                    __syncwarp();
                    acc = 1;
                    if (++st == kStages) { st = 0; ph ^= 1u; }
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair_mc(&d_full[d], kBoth);
                __syncwarp();
                if (++d == 2) { d = 0; dph ^= 1u; }
            }
            if (elect_one()) tc_commit_pair(&drain);
            __syncwarp();
            mbar_wait(&drain, 0, SITE_I8_DRAIN);
        }
    } else if (warp >= 4) {
        // ---------------------------------------------------- scale and store
        pdl_wait();
        const int q4 = warp & 3;
        const int half = (warp - 4) >> 2;     // token columns [128 half, 128 half + 128)
        const int r = 32 * q4 + lane;
        int d = 0;
        uint32_t dph = 0;
        Sched<kGrouped> sched(p, groups, plan, pair0, P);
        Seg sg;
        while (sched.next(sg)) {
            int64_t row0;
            const int nr = rows_of(sg, row0);
            const int64_t n = (int64_t)(2 * sg.nbp + rank) * kBN + r;
            const bool n_ok = n < p.N;
            const int64_t ch = (int64_t)sg.group * p.N + n;
            const float sc = n_ok ? __half2float(__ushort_as_half(p.scales[ch])) : 0.0f;
            const float bi = (n_ok && p.bias) ? __half2float(__ushort_as_half(p.bias[ch])) : 0.0f;
            const int off = 128 + ((n_ok && p.zeros) ? (int)p.zeros[ch] : 0);
            {
                const int c = threadIdx.x - 128;
                sum_sh[d][c] = c < nr ? __ldg(p.x_sums + row0 + c) : 0;
                xs_sh[d][c] = c < nr ? __ldg(p.x_scales + row0 + c) : 0.0f;
            }
            uint16_t *const y0 = p.Y + row0 * p.N + n;
            auto store32 = [&](const uint32_t (&v)[32], int c0) {
                store_tokens(v, &sum_sh[d][c0], &xs_sh[d][c0], off, sc, bi, y0 + c0 * p.N, p.N, n_ok ? nr - c0 : 0);
            };
            if (!named_bar_all(1, 32 * kEpiWarps, mbar_wait(&d_full[d], dph, SITE_I8_DFULL))) break;
            tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(32 * q4) << 16) + d * kBT;
            const int c_end = min(nr, 128 * half + 128);
            int32_t *const mine = sg.slot < 0 ? nullptr : p.partials + ((int64_t)(pair0 * 2 + sg.slot) * 2 + rank) * kPart + r;
            for (int c0 = 128 * half; c0 < c_end; c0 += 32) {
                uint32_t v[32];
                tmem_load_32(src + c0, v);
                if (sg.slot < 0) {
                    store32(v, c0);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) __stcg(mine + (c0 + i) * kBN, (int32_t)v[i]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(leader(&d_empty[d]));
            if (sg.slot >= 0) {
                const int64_t it0 = (int64_t)(sg.tile - plan.dp) * KS;
                const int j0 = plan.owner(it0), j1 = plan.owner(it0 + KS - 1);
                int *const cnt = p.counters + 2 * j0 + rank;
                named_bar_sync(1, 32 * kEpiWarps);   // the part is written
                if (threadIdx.x == 128) {
                    const int last = atomic_add_acq_rel_gpu(cnt, 1) == j1 - j0;
                    if (last) *cnt = 0;
                    last_sh = last;
                }
                named_bar_sync(1, 32 * kEpiWarps);
                if (last_sh) {
                    for (int c0 = 128 * half; c0 < c_end; c0 += 32) {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = 0;
                        for (int j = j0; j <= j1; ++j) {
                            const int32_t *part =
                                p.partials + ((int64_t)(j * 2 + plan.slot(j, sg.tile, KS)) * 2 + rank) * kPart + r;
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] += (uint32_t)__ldcg(part + (c0 + i) * kBN);
                        }
                        store32(v, c0);
                    }
                }
                named_bar_sync(1, 32 * kEpiWarps);   // last_sh is read by all
            }
            if (++d == 2) { d = 0; dph ^= 1u; }
        }
    }

    tc_fence_before();
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

}  // namespace pair
}  // namespace w8a8
}  // namespace w8
