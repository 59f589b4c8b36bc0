// W8A8 linear for few tokens and few channel blocks (a 4096 x 4096 weight has
// 32 blocks for 148 SMs): a cluster of C thread blocks owns one output tile of
// w8a8.cuh and splits its K range evenly.  At the end block k gathers the
// integer sums of channels [128 k / C, 128 (k + 1) / C) from all C blocks in
// its shared memory, by asynchronous distributed-shared-memory stores counted
// on its barrier, adds, scales and stores them: no workspace, no counter, no
// fence, and every block finishes a share of the tile.  Bound by what one SM
// takes in, and when that is short by one start, one gather and one store: a
// block loads all tokens of the tile for its share of K beside its weights, 602
// KB an SM of which 164 are tokens for 48 x 13696 x 4096, at 56 KB a microsecond
// (SMs that stream weights alone take 61).  1 x 4096 x 4096 5.0 us (8.8 with the
// parts added through a workspace), 128 x 4096 x 4096 8.3 (16.1), 48 x 13696 x
// 4096 13.0 (17.2).
#pragma once

#include "w8a8.cuh"

namespace w8 {
namespace w8a8 {
namespace cluster {

constexpr int kMaxCluster = 8;

template <int TN>
struct Cfg {
    static constexpr int kStep = TN >= 128 ? 2 : 4;          // weight tiles per stage
    static constexpr int kWBytes = kStep * kTile;
    static constexpr int kXBox = TN * 128;
    static constexpr int kStageBytes = kWBytes + kStep / 2 * kXBox;
    static constexpr int kGather = TN * kBN * 4;             // the gathered sums: [C][token quad][channel][4]
    static constexpr int kStages = TN <= 16 ? 6 : TN <= 32 ? 5 : TN <= 64 ? 4 : 5;
    static constexpr int kSmemBytes = kStages * kStageBytes + kGather + 1024;
    static constexpr uint32_t kTmemCols = TN < 32 ? 32 : TN;
    static constexpr int kEpiWarps = TN >= 64 ? 8 : 4;
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    static constexpr int kEpiTokens = TN / (kEpiWarps / 4);
    static_assert(kSmemBytes <= 227 * 1024 - 2048, "shared memory budget");
};

// A block whose waits run out sends no sums: the count of every block that
// should have had them stays short, so no block of the cluster stores.

// grid = output tiles x C blocks in clusters of C (2, 4 or 8).  kStall, for the
// tests: the second block of each cluster copies nothing, and waits last 2 ms.
template <int TN, bool kStall = false>
__global__ void __launch_bounds__(Cfg<TN>::kThreads, 1)
w8a8_cluster_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ Params p) {
    using C = Cfg<TN>;
    constexpr unsigned long long kLimitNs = kStall ? 2000000ull : kWaitLimitNs;
    constexpr int kEpi = 32 * C::kEpiWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *gather = ring + C::kStages * C::kStageBytes;
    __shared__ uint64_t full[C::kStages], empty[C::kStages];
    __shared__ uint64_t d_full, drain, gathered;
    __shared__ uint32_t tmem_base_sh;
    __shared__ __align__(16) int sum_sh[TN];
    __shared__ __align__(16) float xs_sh[TN];

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // warp-uniform
    const int lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), csz = (int)cluster_size();
    const int width = kBN / csz;                      // channels this block finishes
    const int unit = blockIdx.x / csz;
    const int tt_n = (int)((p.rows + TN - 1) / TN);
    const int nb = unit / tt_n;
    const int64_t row0 = (int64_t)(unit - nb * tt_n) * TN;
    const int nr = (int)min64(TN, p.rows - row0);
    const int n16 = (nr + 15) & ~15;                  // tokens of the product
    const int kb0 = (int)((int64_t)rank * p.KB / csz), kb1 = (int)((int64_t)(rank + 1) * p.KB / csz);
    const uint8_t *const w = p.packed + ((int64_t)nb * p.KB + kb0) * kTile;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&d_full, 1);
        mbar_init(&drain, 1);
        mbar_init(&gathered, 1);
        mbar_arrive_expect_tx(&gathered, (uint32_t)((csz - 1) * width * n16 * 4));
        fence_barrier_init();
        prefetch_tensormap(&tmap_x);
        // the first weights of a long run into L2 while the previous kernel
        // ends (1 x 13696 x 4096, runs of 53 tiles: 10.8 us with 32 of them,
        // 12.0 with 1; 1 x 4096 x 4096, runs of 16: 5.7 with all, 5.3 with 1)
        if (kb1 - kb0 > 16) prefetch_l2(w, (uint32_t)min(kb1 - kb0 - 16, 32) * kTile);
    }
    if (warp == 2) {
        tmem_alloc(&tmem_base_sh, C::kTmemCols);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;

    if (warp == 0) {
        // ---------------------------------------------------- producer
        if (lane == 0) {
            pdl_wait();
            int st = 0, issued = 0;
            uint32_t ph = 0;
            for (int kb = kStall && rank == 1 ? kb1 : kb0; kb < kb1; kb += C::kStep) {
                const int cnt = min(C::kStep, kb1 - kb), boxes = (cnt + 1) >> 1;
                if (!mbar_wait(&empty[st], ph ^ 1u, SITE_I8_EMPTY, kLimitNs)) break;
                uint8_t *ws = ring + st * C::kStageBytes, *xs = ws + C::kWBytes;
                mbar_arrive_expect_tx(&full[st], cnt * kTile + boxes * C::kXBox);
                bulk_g2s(ws, w + (int64_t)(kb - kb0) * kTile, cnt * kTile, &full[st]);
                for (int b = 0; b < boxes; ++b)
                    tma_load_2d(xs + b * C::kXBox, &tmap_x, (kb + 2 * b) * 64, (int)row0, &full[st]);
                ++issued;
                if (++st == C::kStages) { st = 0; ph ^= 1u; }
            }
            // every copy has landed before the block can leave
            for (int i = 0; i < C::kStages && i < issued; ++i) {
                if (--st < 0) { st = C::kStages - 1; ph ^= 1u; }
                mbar_wait(&full[st], ph, SITE_I8_DRAIN, 10000000ull);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- products
        pdl_wait();   // before the first bounded wait: its second is this call's own
        int st = 0;
        uint32_t ph = 0, acc = 0;
        bool ok = true;
        const uint64_t w_desc0 = smem_desc_kmajor_sw64(smem_u32(ring));
        const uint64_t x_desc0 = smem_desc_kmajor_sw128(smem_u32(ring) + C::kWBytes);
        const uint32_t idesc = idesc_u8_s8_s32(kBN, n16);
        for (int kb = kb0; kb < kb1; kb += C::kStep) {
            const int cnt = min(C::kStep, kb1 - kb);
            if (!warp_all(mbar_wait(&full[st], ph, SITE_I8_FULL, kLimitNs))) { ok = false; break; }
            tc_fence_after();
            const uint64_t wd = w_desc0 + (uint32_t)st * (C::kStageBytes / 16);
            const uint64_t xd = x_desc0 + (uint32_t)st * (C::kStageBytes / 16);
            if (elect_one()) {
#pragma unroll
                for (int t = 0; t < C::kStep; ++t) {
                    if (t < cnt) {
                        const uint64_t wt = wd + t * (kTile / 16), xt = xd + (t >> 1) * (C::kXBox / 16) + (t & 1) * 4;
                        tc_mma_ss_i8(tmem, wt, xt, idesc, t == 0 ? acc : 1);
                        tc_mma_ss_i8(tmem, wt + 2, xt + 2, idesc, 1);
                    }
                }
                tc_commit(&empty[st]);
            }
            __syncwarp();
            acc = 1;
            if (++st == C::kStages) { st = 0; ph ^= 1u; }
        }
        // every product is complete before the tensor memory is read or freed;
        // sums that miss some are not passed on
        uint64_t *const done = ok ? &d_full : &drain;
        if (elect_one()) tc_commit(done);
        __syncwarp();
        mbar_wait(done, 0, SITE_I8_DRAIN);
    } else if (warp >= 4) {
        // ---------------------------------------------------- gather, scale and store
        pdl_wait();
        const int tid = threadIdx.x - 128;
        const int q4 = warp & 3;
        const int r = 32 * q4 + lane;                         // this thread's channel of the sums
        const int cb = C::kEpiTokens * ((warp - 4) >> 2);     // and its warp's first token
        // this thread's channel of the outputs
        const int c = tid % width;
        const int64_t n = (int64_t)nb * kBN + rank * width + c;
        const bool n_ok = n < p.N;
        const float sc = n_ok ? __half2float(__ushort_as_half(p.scales[n])) : 0.0f;
        const float bi = (n_ok && p.bias) ? __half2float(__ushort_as_half(p.bias[n])) : 0.0f;
        const int off = 128 + ((n_ok && p.zeros) ? (int)p.zeros[n] : 0);
        for (int t = tid; t < TN; t += kEpi) {
            sum_sh[t] = t < nr ? p.x_sums[row0 + t] : 0;
            xs_sh[t] = t < nr ? p.x_scales[row0 + t] : 0.0f;
        }
        const bool ok = warp_all(mbar_wait(&d_full, 0, SITE_I8_DFULL, kLimitNs));
        tc_fence_after();
        // [source block][token quad][channel of the receiver][4]
        const int quads = TN / 4;
        const int to = r / width;
        const uint32_t slot = (uint32_t)((rank * quads * width + r % width) * 16);
        const uint32_t dst = mapa_shared(smem_u32(gather), to) + slot, bar = mapa_shared(smem_u32(&gathered), to);
        const int c_end = ok ? min(n16, cb + C::kEpiTokens) : cb;
        for (int c0 = cb; c0 < c_end; c0 += 16) {
            uint32_t v[16];
            tmem_load_16(tmem + ((uint32_t)(32 * q4) << 16) + c0, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = (uint32_t)((c0 / 4 + i) * width * 16);
                if (to == rank)
                    *reinterpret_cast<uint4 *>(gather + slot + at) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                else
                    st_async_dsmem_v4(dst + at, __uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                      __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]), bar);
            }
        }
        named_bar_sync(1, kEpi);   // this block's own sums, the tokens' sums and scales
        // (a block without sums of its own waits as well: the others' are on
        // their way into its shared memory)
        const bool all = mbar_wait_cluster(&gathered, 0, SITE_I8_DRAIN, kLimitNs);
        if (named_bar_all(1, kEpi, ok && all)) {
            uint16_t *const y = p.Y + row0 * p.N + n;
            for (int qd = tid / width; 4 * qd < nr; qd += kEpi / width) {
                int4 s = make_int4(0, 0, 0, 0);
                for (int j = 0; j < csz; ++j) {
                    const int4 t = *reinterpret_cast<const int4 *>(gather + ((j * quads + qd) * width + c) * 16);
                    s.x += t.x;
                    s.y += t.y;
                    s.z += t.z;
                    s.w += t.w;
                }
                const uint32_t v[4] = {(uint32_t)s.x, (uint32_t)s.y, (uint32_t)s.z, (uint32_t)s.w};
                store_tokens<4>(v, &sum_sh[4 * qd], &xs_sh[4 * qd], off, sc, bi, y + 4 * qd * p.N, p.N, n_ok ? nr - 4 * qd : 0);
            }
        }
    }

    // no block leaves while another may still store into it
    tc_fence_before();
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

}  // namespace cluster
}  // namespace w8a8
}  // namespace w8
