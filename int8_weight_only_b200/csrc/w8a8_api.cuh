// Entry points of the int8-activation operators (per-token quantization, the
// W8A8 linear and its grouped form).  Included by w8a16.cu after its helpers
// (device_info, tensor maps, alignment and overlap checks).
#pragma once

#include "tokens.cuh"
#include "w8a8.cuh"
#include "w8a8_cluster.cuh"
#include "w8a8_pair.cuh"

namespace {

// Sums of 128 x 255 x K must stay below 2^31.
constexpr int64_t kMaxSumK = 65536;
// So must the sum of a row's codes, 127 K at most.
constexpr int64_t kMaxTokenK = INT32_MAX / 127;
// Rows of a grouped call: the token tiles of 1024 groups stay below 2^31
// whatever the offsets on the device are.
constexpr int64_t kMaxGroupedRows = 1 << 24;

// Bytes from the first to past the last element of `rows` rows of `width`
// elements, `pitch` elements apart.
inline size_t span(int64_t rows, int64_t pitch, int64_t width, size_t elem) {
    return rows < 1 ? 0 : ((size_t)(rows - 1) * (size_t)pitch + (size_t)width) * elem;
}

// ---------------------------------------------------------------- per-token quantization
template <int kSrc, int TPR, int V, bool kFirst>
int launch_tokens_as(const tokens::Params &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(TPR == 32 ? cdiv(p.M, 8) : p.M), 1, 1);
    cfg.blockDim = dim3(tokens::kBlock<TPR>, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, tokens::quantize_tokens_kernel<kSrc, TPR, V, kFirst>, p) != cudaSuccess) return cuda_fail();
    return launch_status();
}

// A row by one warp up to 1024 elements, by 256 threads up to 16384 where
// there are rows enough to fill the GPU, else by 512 (a row's latency counts);
// longer rows are read twice.
template <int kSrc, bool kFirst>
int launch_tokens_256(const tokens::Params &p, cudaStream_t st) {
    switch (cdiv(p.K, 2048)) {
        case 1: return launch_tokens_as<kSrc, 256, 1, kFirst>(p, st);
        case 2: return launch_tokens_as<kSrc, 256, 2, kFirst>(p, st);
        case 3: return launch_tokens_as<kSrc, 256, 3, kFirst>(p, st);
        case 4: return launch_tokens_as<kSrc, 256, 4, kFirst>(p, st);
        case 5: return launch_tokens_as<kSrc, 256, 5, kFirst>(p, st);
        case 6: return launch_tokens_as<kSrc, 256, 6, kFirst>(p, st);
        case 7: return launch_tokens_as<kSrc, 256, 7, kFirst>(p, st);
        default: return launch_tokens_as<kSrc, 256, 8, kFirst>(p, st);
    }
}

template <int kSrc, int V>
int launch_tokens_512(DeviceInfo *d, const tokens::Params &p, cudaStream_t st) {
    if constexpr (kSrc == tokens::kSwiglu)
        if (p.M <= 2 * d->sms) return launch_tokens_as<kSrc, 512, V, true>(p, st);
    return launch_tokens_as<kSrc, 512, V, false>(p, st);
}

template <int kSrc>
int launch_tokens(DeviceInfo *d, const tokens::Params &p, cudaStream_t st) {
    constexpr bool kLong = kSrc == tokens::kSwiglu;     // long arithmetic: loads first
    const bool many = p.M > 4 * d->sms;
    if (p.K <= 1024 && (many || p.K <= 256)) {
        switch (cdiv(p.K, 256)) {
            case 1: return launch_tokens_as<kSrc, 32, 1, false>(p, st);
            case 2: return launch_tokens_as<kSrc, 32, 2, false>(p, st);
            default: return launch_tokens_as<kSrc, 32, 4, false>(p, st);
        }
    }
    if (p.K <= 16384 && p.M > (kLong ? 6 : 4) * d->sms) return launch_tokens_256<kSrc, kLong>(p, st);
    switch (cdiv(p.K, 4096)) {
        case 1: return launch_tokens_512<kSrc, 1>(d, p, st);
        case 2: return launch_tokens_512<kSrc, 2>(d, p, st);
        case 3:
        case 4: return launch_tokens_512<kSrc, 4>(d, p, st);
        default: return launch_tokens_as<kSrc, 512, 0, false>(p, st);
    }
}

int tokens_common(const void *X, int dtype, bool swiglu, int64_t ldx, int64_t M, int64_t K, int8_t *q, int64_t ldq,
                  float *scales, int32_t *sums, void *stream) {
    if (dtype != W8_F32 && dtype != W8_F16) return W8_ERR_DTYPE;
    if (M < 0 || K < 1 || K % 8 != 0 || M > (int64_t)INT32_MAX || K > kMaxTokenK) return W8_ERR_SHAPE;
    const int64_t cols = swiglu ? 2 * K : K;   // elements of a row that are read
    if (ldx < cols || ldq < K || ldq % 16 != 0 || ldx > (1LL << 40) || ldq > (1LL << 40)) return W8_ERR_SHAPE;
    if (M == 0) return W8_OK;
    if (!X || !q || !scales || !sums) return W8_ERR_NULL;
    const size_t elem = dtype == W8_F32 ? 4 : 2;
    if (!aligned16(X) || !aligned16(q) || !aligned16(scales) || !aligned16(sums) || (M > 1 && ldx * elem % 16 != 0))
        return W8_ERR_ALIGN;
    const size_t xb = span(M, ldx, cols, elem), qb = span(M, ldq, K, 1), sb = (size_t)M * 4;
    if (overlap(X, xb, q, qb) || overlap(X, xb, scales, sb) || overlap(X, xb, sums, sb) || overlap(q, qb, scales, sb) ||
        overlap(q, qb, sums, sb) || overlap(scales, sb, sums, sb))
        return W8_ERR_ALIAS;
    DeviceInfo *d = nullptr;
    const int rc = device_info(&d);
    if (rc != W8_OK) return rc;
    const tokens::Params p = {X, ldx, M, K, q, ldq, scales, sums};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (swiglu) return launch_tokens<tokens::kSwiglu>(d, p, st);
    return dtype == W8_F32 ? launch_tokens<tokens::kF32>(d, p, st) : launch_tokens<tokens::kF16>(d, p, st);
}

// ---------------------------------------------------------------- W8A8 linear
// Codes [rows, K], box 128 features x box_rows rows, 128-byte swizzle;
// features past K and rows past the last read as zero.
int make_map_codes(CUtensorMap *map, const int8_t *q, int64_t ldq, int64_t rows, int64_t K, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return W8_ERR_CUDA;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ldq};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(q), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? W8_OK : W8_ERR_CUDA;
}

// Whether `units` clusters of c blocks (w8a8_cluster.cuh) can all run at once,
// with two weight tiles at least for each block.
template <int TN>
bool w8a8_cluster_fits(DeviceInfo *d, int c, int64_t units, int64_t KB) {
    if (units * c > d->sms || KB < 2 * c) return false;
    const void *fn = (const void *)w8a8::cluster::w8a8_cluster_kernel<TN>;
    std::lock_guard<std::mutex> lock(g_mu);
    int &cached = d->dclusters[{fn, c}];
    if (cached == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(d->sms / c * c), 1, 1);
        cfg.blockDim = dim3(w8a8::cluster::Cfg<TN>::kThreads, 1, 1);
        cfg.dynamicSmemBytes = w8a8::cluster::Cfg<TN>::kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = c;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, w8a8::cluster::w8a8_cluster_kernel<TN>, &cfg) != cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        cached = n > 0 ? n : -1;
    }
    return cached >= units;
}

template <int TN, bool kStall = false>
int launch_w8a8_cluster(int c, int64_t units, const int8_t *q, int64_t ldq, int64_t K, const w8a8::Params &p,
                        cudaStream_t st) {
    CUtensorMap map;
    const int rc = make_map_codes(&map, q, ldq, p.rows, K, TN);
    if (rc != W8_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * c), 1, 1);
    cfg.blockDim = dim3(w8a8::cluster::Cfg<TN>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = w8a8::cluster::Cfg<TN>::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, w8a8::cluster::w8a8_cluster_kernel<TN, kStall>, map, p) != cudaSuccess) return cuda_fail();
    return launch_status();
}

// One weight on single SMs: clusters of c blocks, or (c == 0) whole tiles.
template <int TN>
int launch_w8a8_as(DeviceInfo *d, int c, const int8_t *q, int64_t ldq, int64_t K, const w8a8::Params &p, cudaStream_t st) {
    const int64_t units = cdiv(p.rows, TN) * p.NB;
    if (c > 0) return launch_w8a8_cluster<TN>(c, units, q, ldq, K, p, st);
    CUtensorMap map;
    const int rc = make_map_codes(&map, q, ldq, p.rows, K, TN);
    if (rc != W8_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    // blocks with equally many output tiles, as far as they divide
    const int64_t each = cdiv(units, d->sms);
    cfg.gridDim = dim3((unsigned)cdiv(units, each), 1, 1);
    cfg.blockDim = dim3(w8a8::Cfg<TN>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = w8a8::Cfg<TN>::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, w8a8::w8a8_kernel<TN, false>, map, p) != cudaSuccess) return cuda_fail();
    return launch_status();
}

// Many tokens: pairs of SMs (w8a8_pair.cuh).
template <int BT, bool kGrouped>
int launch_w8a8_pair(DeviceInfo *d, const int8_t *q, int64_t ldq, int64_t K, const w8a8::Params &p, cudaStream_t st) {
    namespace wp = w8a8::pair;
    wp::Maps maps;
    CUtensorMap map_w;
    int rc = W8_OK;
    for (int i = 0; i < wp::kXMaps && rc == W8_OK; ++i) rc = make_map_codes(&maps.x[i], q, ldq, p.rows, K, BT / 2 >> i);
    if (rc != W8_OK) return rc;
    // coordinates of rows of 128 packed bytes and tile numbers are 32-bit
    const int64_t wrows = (int64_t)p.groups * p.NB * p.KB * (w8a8::kTile / 128);
    const int64_t most_tiles = (cdiv(p.rows, BT) + p.groups) * cdiv(p.NB, 2);
    if (wrows > (int64_t)INT32_MAX - 128 || most_tiles > INT32_MAX / 2) return W8_ERR_SHAPE;
    rc = make_map_2d(&map_w, p.packed, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, (uint64_t)wrows, 128, 128,
                     CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc != W8_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(wp::kThreads, 1, 1);
    cfg.dynamicSmemBytes = wp::Cfg<BT>::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;   // the occupancy query takes the cluster shape only
    const void *fn = (const void *)wp::w8a8_pair_kernel<BT, kGrouped>;
    int pairs = 0;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        int &cached = d->dclusters[{fn, 2}];
        if (cached == 0) {
            cfg.gridDim = dim3((unsigned)(d->sms / 2 * 2), 1, 1);
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, wp::w8a8_pair_kernel<BT, kGrouped>, &cfg) != cudaSuccess || n < 1) {
                cudaGetLastError();
                n = d->sms / 2;
            }
            cached = std::max(1, n);
        }
        pairs = cached;
    }
    if (!kGrouped) pairs = (int)std::min<int64_t>(pairs, most_tiles);
    cfg.gridDim = dim3((unsigned)(2 * pairs), 1, 1);
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, wp::w8a8_pair_kernel<BT, kGrouped>, map_w, maps, p) != cudaSuccess) return cuda_fail();
    return launch_status();
}

enum class Kernel { kTiles = 1, kCluster = 2, kPair = 3 };
struct Choice {
    Kernel kernel;
    int tokens;    // of a tile
    int cluster;   // blocks of a cluster, of kCluster
};

// The kernel of a product of one weight: whichever is shortest by a line through
// its measured times, in microseconds.
//   whole tiles on single SMs (w8a8.cuh):  a + waves (e + b weight tiles of K)
//   clusters (w8a8_cluster.cuh):           a + e blocks + b weight tiles a block
//   pairs of SMs (w8a8_pair.cuh):          a + waves (e + b steps of 128 features)
// with tiles of 16, 32, 64 or 128 tokens on single SMs and of 256 on pairs, for
// more than 128 tokens.  Over 1052 sizes of 1 to 4096 tokens, each measured with
// every kernel that takes it, the choice is 0.9 % above the best in the mean, 1.27
// times it at worst (16 x 256 x 256, 2.8 against 2.2).  Measured and (by the line):
//                        tiles        clusters of 2   of 4        pairs
//   16 x 512 x 9216      2.8 (2.8)    4.1 (4.3)
//   1 x 4096 x 4096      7.8 (7.6)    6.0 (6.0)       6.1 (5.3)
//   512 x 768 x 2304     4.4 (4.9)    7.0 (7.3)                   6.3 (6.1)
//   512 x 4096 x 4096    10.4 (10.4)                              14.4 (13.5)
//   1024 x 4096 x 4096   17.8 (18.9)                              15.1 (13.5)
// Pairs with tiles of 128 tokens (512 x 768 x 2304 5.1, 512 x 4096 x 4096 12.0)
// would be 5 % or more ahead of the choice for 39 of 484 sizes above 128 tokens,
// but no line tells which: with them in it the choice was 0.03 % better in the
// mean.  Groups take them.
struct Line {
    double a, e, b;
};
constexpr Line kTileLine[4] = {{1.1, 1.05, 0.0845}, {1.1, 1.4, 0.0845}, {1.1, 1.75, 0.0845}, {2.0, 1.6, 0.107}};
constexpr Line kClusterLine[4] = {{2.25, 0.012, 0.092}, {2.75, 0.013, 0.092}, {3.1, 0.014, 0.10}, {4.5, 0.013, 0.155}};
constexpr Line kPairLine = {2.65, 1.75, 0.284};

Choice choose_w8a8(DeviceInfo *d, int64_t M, int64_t NB, int64_t KB) {
    const int i = M <= 16 ? 0 : M <= 32 ? 1 : M <= 64 ? 2 : 3, tn = 16 << i;
    const int64_t units = cdiv(M, tn) * NB;
    Choice best = {Kernel::kTiles, tn, 0};
    double least = kTileLine[i].a + (double)cdiv(units, d->sms) * (kTileLine[i].e + kTileLine[i].b * (double)KB);
    for (int c = w8a8::cluster::kMaxCluster; c >= 2; c >>= 1) {
        const double t = kClusterLine[i].a + kClusterLine[i].e * (double)(units * c) + kClusterLine[i].b * (double)cdiv(KB, c);
        if (t >= least) continue;
        const bool fits = i == 0   ? w8a8_cluster_fits<16>(d, c, units, KB)
                          : i == 1 ? w8a8_cluster_fits<32>(d, c, units, KB)
                          : i == 2 ? w8a8_cluster_fits<64>(d, c, units, KB)
                                   : w8a8_cluster_fits<128>(d, c, units, KB);
        if (fits) {
            least = t;
            best = {Kernel::kCluster, tn, c};
        }
    }
    if (M > 128) {
        const int64_t waves = cdiv(cdiv(M, 256) * cdiv(NB, 2), std::max(1, d->sms / 2));
        if (kPairLine.a + (double)waves * (kPairLine.e + kPairLine.b * (double)cdiv(KB, 2)) < least) best = {Kernel::kPair, 256, 0};
    }
    return best;
}

int launch_w8a8(DeviceInfo *d, const int8_t *q, int64_t ldq, int64_t K, const w8a8::Params &p, cudaStream_t st) {
    const Choice c = choose_w8a8(d, p.rows, p.NB, p.KB);
    if (c.kernel == Kernel::kPair) return launch_w8a8_pair<256, false>(d, q, ldq, K, p, st);
    switch (c.tokens) {
        case 16: return launch_w8a8_as<16>(d, c.cluster, q, ldq, K, p, st);
        case 32: return launch_w8a8_as<32>(d, c.cluster, q, ldq, K, p, st);
        case 64: return launch_w8a8_as<64>(d, c.cluster, q, ldq, K, p, st);
        default: return launch_w8a8_as<128>(d, c.cluster, q, ldq, K, p, st);
    }
}

// Groups on single SMs (w8a8.cuh): one block each, the kernel deals the tiles.
template <int TN>
int launch_w8a8_groups(DeviceInfo *d, const int8_t *q, int64_t ldq, int64_t K, const w8a8::Params &p, cudaStream_t st) {
    if ((cdiv(p.rows, TN) + p.groups) * p.NB > INT32_MAX / 2) return W8_ERR_SHAPE;   // tile numbers are 32-bit
    CUtensorMap map;
    const int rc = make_map_codes(&map, q, ldq, p.rows, K, TN);
    if (rc != W8_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)d->sms, 1, 1);
    cfg.blockDim = dim3(w8a8::Cfg<TN>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = w8a8::Cfg<TN>::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, w8a8::w8a8_kernel<TN, true>, map, p) != cudaSuccess) return cuda_fail();
    return launch_status();
}

// The kernel of a grouped product, by the mean group (the groups themselves
// are known on the device only).  Up to 4 tokens, and up to 16 where the
// products are long enough to hide its stores, single SMs with tiles of 16 and
// 32 tokens; else pairs of SMs, with tiles of 256 tokens from 96 tokens on.
// Microseconds with tiles of 16 / 32 on single SMs, 128 / 256 on pairs, 8
// groups of 4096 x 4096: 2 tokens each 21.3 / 21.7, 23.5 / -, 8 23.0 / 23.4,
// 24.0 / -, 16 25.6 / 23.7, 24.3 / 25.9, 64 54.6 / 37.2, 25.7 / 27.6, 128 - / -,
// 31.2 / 30.2, 256 - / -, 46.0 / 40.0; 39 groups of 288 x 11040, 23 tokens each:
// 53.4 / 50.7, 33.0 / 33.2.  How the rows spread the host cannot see: with all of
// them in one group the mean misleads most (128 rows in one of 8 groups of 4096 x
// 13696, taken with tiles of 32: 23.6, where tiles of 128 on pairs take 14.2).
Choice choose_w8a8_grouped(int64_t M, int64_t groups, int64_t K) {
    if (M <= 4 * groups) return {Kernel::kTiles, 16, 0};
    if (M <= 16 * groups && K >= 1024) return {Kernel::kTiles, 32, 0};
    return {Kernel::kPair, M > 96 * groups ? 256 : 128, 0};
}

int launch_w8a8_grouped(DeviceInfo *d, const int8_t *q, int64_t ldq, int64_t K, const w8a8::Params &p, cudaStream_t st) {
    const Choice c = choose_w8a8_grouped(p.rows, p.groups, K);
    if (c.kernel == Kernel::kTiles)
        return c.tokens == 16 ? launch_w8a8_groups<16>(d, q, ldq, K, p, st) : launch_w8a8_groups<32>(d, q, ldq, K, p, st);
    return c.tokens == 128 ? launch_w8a8_pair<128, true>(d, q, ldq, K, p, st)
                           : launch_w8a8_pair<256, true>(d, q, ldq, K, p, st);
}

cudaError_t w8a8_attributes() {
    cudaError_t e = cudaSuccess;
#define W8_I8_CLUSTER_SMEM(TN, STALL)                                                                     \
    if (e == cudaSuccess)                                                                                     \
        e = cudaFuncSetAttribute((const void *)w8a8::cluster::w8a8_cluster_kernel<TN, STALL>,                \
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, w8a8::cluster::Cfg<TN>::kSmemBytes);
    W8_I8_CLUSTER_SMEM(16, false)
    W8_I8_CLUSTER_SMEM(32, false)
    W8_I8_CLUSTER_SMEM(64, false)
    W8_I8_CLUSTER_SMEM(128, false)
    W8_I8_CLUSTER_SMEM(128, true)
#undef W8_I8_CLUSTER_SMEM
#define W8_I8_SMEM(TN)                                                                                        \
    if (e == cudaSuccess)                                                                                     \
        e = cudaFuncSetAttribute((const void *)w8a8::w8a8_kernel<TN, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, \
                                 w8a8::Cfg<TN>::kSmemBytes);
    W8_I8_SMEM(16)
    W8_I8_SMEM(32)
    W8_I8_SMEM(64)
    W8_I8_SMEM(128)
#undef W8_I8_SMEM
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute((const void *)w8a8::w8a8_kernel<16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 w8a8::Cfg<16>::kSmemBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute((const void *)w8a8::w8a8_kernel<32, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 w8a8::Cfg<32>::kSmemBytes);
#define W8_I8_PAIR_SMEM(BT, GROUPED)                                                                          \
    if (e == cudaSuccess)                                                                                     \
        e = cudaFuncSetAttribute((const void *)w8a8::pair::w8a8_pair_kernel<BT, GROUPED>,                    \
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, w8a8::pair::Cfg<BT>::kSmemBytes);
    W8_I8_PAIR_SMEM(256, false)
    W8_I8_PAIR_SMEM(128, true)
    W8_I8_PAIR_SMEM(256, true)
#undef W8_I8_PAIR_SMEM
    return e;
}

// The linear of one weight (offsets == nullptr, groups == 1), of one weight per
// group, or of one weight with a block of each cluster stalled.
enum class Form { kOne, kGrouped, kStalled };
int w8a8_common(const int8_t *q, int64_t ldq, const float *x_scales, const int32_t *x_sums, const int32_t *offsets,
                Form form, int64_t groups, const uint8_t *packed, const uint16_t *scales, const int8_t *zeros,
                const uint16_t *bias, uint16_t *Y, int64_t M, int64_t K, int64_t N, void *stream) {
    const bool grouped = form == Form::kGrouped;
    if (M < 0 || K < 1 || N < 1 || K % 8 != 0 || N % 8 != 0 || K > kMaxSumK || M > (int64_t)INT32_MAX - 512 ||
        N > (1LL << 30) || ldq < K || ldq % 16 != 0 || ldq >= (1LL << 40))
        return W8_ERR_SHAPE;
    if (grouped && (groups < 1 || groups > w8a8::kMaxGroups || M > kMaxGroupedRows)) return W8_ERR_SHAPE;
    if (!packed || !scales || (grouped && !offsets)) return W8_ERR_NULL;
    if (M == 0) return W8_OK;   // no rows: nothing to read or write
    if (!q || !x_scales || !x_sums || !Y) return W8_ERR_NULL;
    if (!aligned16(q) || !aligned16(x_scales) || !aligned16(x_sums) || !aligned16(packed) || !aligned16(scales) ||
        !aligned16(Y) || (bias && !aligned16(bias)) || (zeros && !aligned16(zeros)) || (offsets && !aligned16(offsets)))
        return W8_ERR_ALIGN;
    const size_t yb = (size_t)M * N * 2, qb = span(M, ldq, K, 1), wb = (size_t)groups * w8_prepacked_bytes(K, N),
                 sb = (size_t)groups * N * 2;
    if (overlap(Y, yb, q, qb) || overlap(Y, yb, x_scales, (size_t)M * 4) || overlap(Y, yb, x_sums, (size_t)M * 4) ||
        overlap(Y, yb, packed, wb) || overlap(Y, yb, scales, sb) || (bias && overlap(Y, yb, bias, sb)) ||
        (zeros && overlap(Y, yb, zeros, sb / 2)) || (grouped && overlap(Y, yb, offsets, (size_t)(groups + 1) * 4)))
        return W8_ERR_ALIAS;
    DeviceInfo *d = nullptr;
    int rc = device_info(&d);
    if (rc != W8_OK) return rc;
    w8a8::Params p = {};
    p.packed = packed;
    p.scales = scales;
    p.zeros = zeros;
    p.bias = bias;
    p.x_scales = x_scales;
    p.x_sums = x_sums;
    p.offsets = offsets;
    p.Y = Y;
    p.rows = M;
    p.N = N;
    p.groups = (int)groups;
    p.NB = (int)cdiv(N, 128);
    p.KB = (int)cdiv(K, 64);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (form == Form::kStalled) {
        const int64_t units = cdiv(M, 128) * p.NB;
        for (int c = w8a8::cluster::kMaxCluster; c >= 2; c >>= 1)
            if (w8a8_cluster_fits<128>(d, c, units, p.KB)) return launch_w8a8_cluster<128, true>(c, units, q, ldq, K, p, st);
        return W8_ERR_SHAPE;
    }
    return grouped ? launch_w8a8_grouped(d, q, ldq, K, p, st) : launch_w8a8(d, q, ldq, K, p, st);
}

}  // namespace

extern "C" {

int w8_quantize_per_token(const void *X, int x_dtype, int64_t ldx, int64_t M, int64_t K, int8_t *q, int64_t ldq,
                          float *scales, int32_t *sums, void *stream) {
    return tokens_common(X, x_dtype, false, ldx, M, K, q, ldq, scales, sums, stream);
}

int w8_swiglu_quantize_per_token(const uint16_t *H, int64_t ldh, int64_t M, int64_t K, int8_t *q, int64_t ldq,
                                 float *scales, int32_t *sums, void *stream) {
    return tokens_common(H, W8_F16, true, ldh, M, K, q, ldq, scales, sums, stream);
}

int w8a8_linear(const int8_t *q, int64_t ldq, const float *x_scales, const int32_t *x_sums, const uint8_t *packed,
                const uint16_t *scales, const int8_t *zeros, const uint16_t *bias, uint16_t *Y, int64_t M, int64_t K,
                int64_t N, void *stream) {
    return w8a8_common(q, ldq, x_scales, x_sums, nullptr, Form::kOne, 1, packed, scales, zeros, bias, Y, M, K, N, stream);
}

int w8_test_w8a8_cluster_stall(const int8_t *q, int64_t ldq, const float *x_scales, const int32_t *x_sums,
                               const uint8_t *packed, const uint16_t *scales, uint16_t *Y, int64_t M, int64_t K,
                               int64_t N, void *stream) {
    return w8a8_common(q, ldq, x_scales, x_sums, nullptr, Form::kStalled, 1, packed, scales, nullptr, nullptr, Y, M, K, N,
                       stream);
}

int w8a8_linear_grouped(const int8_t *q, int64_t ldq, const float *x_scales, const int32_t *x_sums,
                        const int32_t *offsets, int64_t groups, const uint8_t *packed, const uint16_t *scales,
                        const int8_t *zeros, const uint16_t *bias, uint16_t *Y, int64_t M, int64_t K, int64_t N,
                        void *stream) {
    return w8a8_common(q, ldq, x_scales, x_sums, offsets, Form::kGrouped, groups, packed, scales, zeros, bias, Y, M, K, N,
                       stream);
}

int w8_test_w8a8_kernel(int64_t M, int64_t K, int64_t N, int64_t groups) {
    if (M < 1 || M > (int64_t)INT32_MAX - 512 || K < 1 || K > kMaxSumK || N < 1 || N > (1LL << 30) || groups < 0 ||
        groups > w8a8::kMaxGroups)
        return W8_ERR_SHAPE;
    DeviceInfo *d = nullptr;
    const int rc = device_info(&d);
    if (rc != W8_OK) return rc;
    const Choice c = groups > 0 ? choose_w8a8_grouped(M, groups, K) : choose_w8a8(d, M, cdiv(N, 128), cdiv(K, 64));
    return 1000 * (int)c.kernel + c.tokens;
}

}  // extern "C"
