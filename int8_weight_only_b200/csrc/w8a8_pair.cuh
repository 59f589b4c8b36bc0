// W8A8 linear for many tokens, on pairs of SMs (tcgen05 cta_group::2): the
// product of w8a8.cuh with output tiles of 256 channels x BT tokens (256, or
// 128 for groups of few).  Each block of a cluster of
// two holds its own 128 channels of the weight and half of the tile's tokens
// in shared memory, so a 128-wide K step of a 256 x 256 tile brings 32 KB into
// each SM for 512 cycles of integer products; the 32-bit sums of two tiles fit
// in tensor memory, and a tile is scaled and stored while the next one runs.
//
// Schedule: whole tiles, round robin over the pairs.  Splitting the K steps of
// the last tiles evenly over the pairs, the parts added through the workspace,
// was slower wherever it was tried: a block's part of a tile is 128 KB, which
// one SM takes more than a microsecond to write or read (256 x 4096 x 27392,
// two waves of tiles: 29.3 us whole, 34.5 split; 512 x 4096 x 4096, half a
// wave: 14.1 whole, 24.9 split).
//
// Dealing equally many tiles to fewer pairs costs 0.4 to 0.7 us of divisions
// before the first copy and gave less.
//
// Roles in each block: warp 0 producer, warp 1 products (first block), warp 2
// tensor memory, warps 4-11 scale and store.
#pragma once

#include "w8a8.cuh"

namespace w8 {
namespace w8a8 {
namespace pair {

constexpr int kStepTiles = 2;                // weight tiles per stage (128 features)
constexpr int kWBytes = kStepTiles * kTile;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kParts = kEpiWarps / 4;        // a warp reads 32 of the 128 channels, of one part of the tokens
// Outputs on their way out, per warp two buffers of kChunk tokens x its 32
// channels fp16; the 16-byte piece c of token t lies at piece c ^ (t / 2 & 3).
constexpr int kChunk = 32;
constexpr int kOutBuf = kChunk * 32 * 2;
constexpr int kOutBytes = kEpiWarps * 2 * kOutBuf;
constexpr uint16_t kBoth = 0x3;
// The tokens' tensor map comes with three box heights, BT / 2 rows and a half
// and a quarter of that: a short tile takes the lowest that holds its half.
constexpr int kXMaps = 3;

template <int BT>
struct Cfg {
    static constexpr int kXBytes = BT / 2 * 128;             // half of the tokens x 128 features
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = BT == 256 ? 5 : 7;
    static constexpr int kSmemBytes = kStages * kStageBytes + kOutBytes + 1024;
    static constexpr uint32_t kTmemCols = 2 * BT;
    static constexpr int kPartTokens = BT / kParts;
};

struct Maps {
    CUtensorMap x[kXMaps];
};

struct Seg {
    int group, nbp, tt;
};

template <int BT, bool kGrouped>
struct Sched {
    const Groups *g;
    int NBP, TT, group, step;
    int64_t tile, tiles;
    __device__ Sched(const Params &p, const Groups *groups, int64_t n_tiles, int pair, int pairs)
        : g(groups), NBP((p.NB + 1) / 2), TT((int)((p.rows + BT - 1) / BT)), group(0), step(pairs), tile(pair),
          tiles(n_tiles) {}
    __device__ bool next(Seg &s) {
        if (tile >= tiles) return false;
        int64_t local = tile;
        int tt_n = TT;
        if constexpr (kGrouped) {
            while (tile >= (int64_t)NBP * g->tiles[group + 1]) ++group;
            local -= (int64_t)NBP * g->tiles[group];
            tt_n = g->tiles[group + 1] - g->tiles[group];
        }
        s.group = group;
        // the host keeps the tiles of a call below 2^31
        s.nbp = (int)local / tt_n;
        s.tt = (int)local - s.nbp * tt_n;
        tile += step;
        return true;
    }
};

// grid = 2 x pairs blocks in clusters of two.  tmap_w: the packed weights as
// rows of 128 bytes, box 128 x 128 (two tiles), no swizzle; maps: codes
// [rows, K], boxes of 128 features, 128-byte swizzle.
template <int BT, bool kGrouped>
__global__ void __launch_bounds__(kThreads, 1)
w8a8_pair_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ Maps maps,
                 const __grid_constant__ Params p) {
    using C = Cfg<BT>;
    constexpr int kStages = C::kStages, kStageBytes = C::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *out_sh = ring + kStages * kStageBytes;
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint64_t d_full[2], d_empty[2], drain;
    __shared__ uint32_t tmem_base_sh;
    __shared__ __align__(16) int sum_sh[2][BT];
    __shared__ __align__(16) float xs_sh[2][BT];
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
        prefetch_tensormap(&maps.x[0]);
    }
    if (warp == 2) {
        tmem_alloc_pair(&tmem_base_sh, C::kTmemCols);
        tmem_relinquish_pair();
    }
    pdl_launch_dependents();
    const Groups *groups = nullptr;
    if constexpr (kGrouped) groups = reinterpret_cast<const Groups *>(&groups_sh);
    auto count = [&]() -> int64_t {
        if constexpr (kGrouped)
            return (int64_t)groups->tiles[p.groups] * ((p.NB + 1) / 2);
        else
            return (p.rows + BT - 1) / BT * ((p.NB + 1) / 2);
    };
    // a block's weights of an output tile (the last tile of an odd number of
    // channel blocks has one block twice)
    auto block_of = [&](const Seg &s) -> int64_t {
        return (int64_t)s.group * p.NB + min(2 * s.nbp + (int)rank, p.NB - 1);
    };
    // (Bringing the first weights into L2 ahead of the previous kernel's end,
    // as the kernels for few tokens do, takes a microsecond more here.)
    if constexpr (kGrouped) {
        pdl_wait();
        load_groups<BT, kThreads>(p, *reinterpret_cast<Groups *>(&groups_sh));
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    const int64_t n_tiles = count();
    auto rows_of = [&](const Seg &s, int64_t &row0) -> int {
        int64_t first = 0, end = p.rows;
        if constexpr (kGrouped) {
            first = groups->first[s.group];
            end = groups->first[s.group + 1];
        }
        row0 = first + (int64_t)s.tt * BT;
        return (int)min64(BT, end - row0);
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
            Sched<BT, kGrouped> sched(p, groups, n_tiles, pair0, P);
            Seg sg;
            while (ok && sched.next(sg)) {
                int64_t row0;
                const int n = width(rows_of(sg, row0));
                const int wrow = (int)(block_of(sg) * p.KB * (kTile / 128));
                const int xrow = (int)row0 + (int)rank * (n / 2);
                const int low = n <= BT / 4 ? 2 : n <= BT / 2 ? 1 : 0;
                const CUtensorMap *const tmap_x = &maps.x[low];
                const uint32_t bytes = 2 * (kWBytes + (C::kXBytes >> low));
                for (int ks = 0; ks < KS; ++ks) {
                    if (!mbar_wait(&empty[st], ph ^ 1u, SITE_I8_EMPTY)) { ok = false; break; }
                    uint8_t *ws = ring + st * kStageBytes;
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
                    tma_load_2d_pair(ws, &tmap_w, 0, wrow + ks * (kWBytes / 128), leader(&full[st]));
                    tma_load_2d_pair(ws + kWBytes, tmap_x, ks * 128, xrow, leader(&full[st]));
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
            pdl_wait();   // before the first bounded wait: its second is this call's own
            int st = 0, d = 0;
            uint32_t ph = 0, dph = 0;
            bool ok = true;
            const uint64_t w_desc0 = smem_desc_kmajor_sw64(smem_u32(ring));
            const uint64_t x_desc0 = smem_desc_kmajor_sw128(smem_u32(ring) + kWBytes);
            Sched<BT, kGrouped> sched(p, groups, n_tiles, pair0, P);
            Seg sg;
            while (ok && sched.next(sg)) {
                int64_t row0;
                const uint32_t idesc = idesc_u8_s8_s32(2 * kBN, width(rows_of(sg, row0)));
                const uint32_t dst = tmem + d * BT;
                if (!warp_all(mbar_wait(&d_empty[d], dph ^ 1u, SITE_I8_DEMPTY))) { ok = false; break; }
                tc_fence_after();
                uint32_t acc = 0;
                for (int ks = 0; ks < KS; ++ks) {
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
        const int part = (warp - 4) >> 2;     // token columns [kPartTokens part, + kPartTokens)
        // Sums come as fragments: this thread holds channels ch0 + 8 j of the
        // block, j < 4, and tokens 8 i + t0, + 1 of a chunk, i < 4.
        const int ch0 = 32 * q4 + (lane >> 2);
        const int t0 = 2 * (lane & 3);
        int d = 0, buffer = 0;
        uint32_t dph = 0;
        Sched<BT, kGrouped> sched(p, groups, n_tiles, pair0, P);
        // What the scaling of a tile reads from global memory: its channels'
        // scales, biases and zero points and one token's scale and sum.
        // Loaded a tile ahead, since a tile of short K is over before the
        // loads are.
        struct Operands {
            Seg sg;
            int64_t row0;
            int nr;
            uint16_t sc[4], bi[4];
            int8_t z[4];
            int sum;
            float xs;
        };
        const int c_own = threadIdx.x - 128;     // this thread's token of the tile
        auto fetch = [&](Operands &o) -> bool {
            if (!sched.next(o.sg)) return false;
            o.nr = rows_of(o.sg, o.row0);
            const int64_t n0 = (int64_t)(2 * o.sg.nbp + rank) * kBN + ch0;
            const int64_t at = (int64_t)o.sg.group * p.N + n0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool ok = n0 + 8 * j < p.N;
                o.sc[j] = ok ? p.scales[at + 8 * j] : (uint16_t)0;
                o.bi[j] = ok && p.bias ? p.bias[at + 8 * j] : (uint16_t)0;
                o.z[j] = ok && p.zeros ? p.zeros[at + 8 * j] : (int8_t)0;
            }
            o.sum = c_own < o.nr ? p.x_sums[o.row0 + c_own] : 0;
            o.xs = c_own < o.nr ? p.x_scales[o.row0 + c_own] : 0.0f;
            return true;
        };
        Operands next;
        bool more = fetch(next);
        while (more) {
            const Seg sg = next.sg;
            const int nr = next.nr;
            uint64_t sc2[4], bi2[4];
            int off[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float sc = __half2float(__ushort_as_half(next.sc[j])), bi = __half2float(__ushort_as_half(next.bi[j]));
                sc2[j] = f32x2(sc, sc);
                bi2[j] = f32x2(bi, bi);
                off[j] = 128 + (int)next.z[j];
            }
            if (c_own < BT) {
                sum_sh[d][c_own] = next.sum;
                xs_sh[d][c_own] = next.xs;
            }
            // kChunk tokens from column c0 leave through this warp's part of
            // shared memory as runs of its 32 channels, 16 bytes a lane.
            // (Whole rows of 128 channels need a barrier of four warps a
            // chunk, which cost more than the longer runs gave: 0.2 us.)
            const int64_t n0 = (int64_t)(2 * sg.nbp + rank) * kBN + 32 * q4 + 8 * (lane & 3);
            uint16_t *const y0 = p.Y + next.row0 * p.N + n0;
            const bool piece_ok = n0 < p.N;
            more = fetch(next);
            auto store = [&](const uint32_t (&v)[kChunk], int c0) {
                uint8_t *buf = out_sh + (2 * (warp - 4) + buffer) * kOutBuf;
                buffer ^= 1;
                int2 s[kChunk / 8];
                uint64_t x2[kChunk / 8];
#pragma unroll
                for (int i = 0; i < kChunk / 8; ++i) {
                    s[i] = *reinterpret_cast<const int2 *>(&sum_sh[d][c0 + 8 * i + t0]);
                    x2[i] = *reinterpret_cast<const uint64_t *>(&xs_sh[d][c0 + 8 * i + t0]);
                }
                // row of 16 bytes that this thread addresses: token lane % 8
                // of a group of eight, piece lane / 8
                const uint32_t row = smem_u32(buf) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
#pragma unroll
                for (int i = 0; i < kChunk / 8; ++i) {
                    uint32_t h[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int e = 16 * (j >> 1) + 4 * i + 2 * (j & 1);
                        const uint64_t a = f32x2((float)((int)v[e] - off[j] * s[i].x), (float)((int)v[e + 1] - off[j] * s[i].y));
                        const __half2 y = __float22half2_rn(f32x2_parts(f32x2_fma(f32x2_mul(a, x2[i]), sc2[j], bi2[j])));
                        h[j] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                    stmatrix_x4_trans(row + i * 8 * 64, h[0], h[1], h[2], h[3]);
                }
                __syncwarp();
                uint4 w[kChunk / 8];
#pragma unroll
                for (int i = 0; i < kChunk / 8; ++i)
                    w[i] = *reinterpret_cast<const uint4 *>(buf + i * 8 * 64 + (lane >> 2) * 64 +
                                                            (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
#pragma unroll
                for (int i = 0; i < kChunk / 8; ++i) {
                    const int t = c0 + 8 * i + (lane >> 2);
                    if (piece_ok && t < nr) *reinterpret_cast<uint4 *>(y0 + t * p.N) = w[i];
                }
            };
            if (!named_bar_all(1, 32 * kEpiWarps, mbar_wait(&d_full[d], dph, SITE_I8_DFULL))) break;
            tc_fence_after();
            const uint32_t src = tmem + ((uint32_t)(32 * q4) << 16) + d * BT;
            const int c_end = min(nr, C::kPartTokens * (part + 1));
            for (int c0 = C::kPartTokens * part; c0 < c_end; c0 += kChunk) {
                uint32_t v[kChunk];
                tmem_load_frag_16x32(src + c0, v);
                tmem_load_frag_16x32(src + (16u << 16) + c0, v + 16);
                store(v, c0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(leader(&d_empty[d]));
            if (++d == 2) { d = 0; dph ^= 1u; }
        }
    }

    tc_fence_before();
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, C::kTmemCols);
    }
}

}  // namespace pair
}  // namespace w8a8
}  // namespace w8
