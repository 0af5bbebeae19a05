// grouped_gemm.cu -- host side of the products grouped by rows and of low-rank adapters
// beside a shared product: checks, tensor maps, the choice of a tile, launches (see
// grouped_ops.h).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "grouped_few_kernel.cuh"
#include "grouped_kernel.cuh"

namespace linear_ops {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
constexpr int64_t kDefaultTimeoutNs = 4000000000LL;

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        }
        cudaGetLastError();
    });
    return fn;
}

// Matrices of rows x cols 16-bit elements, `depth` of them (0: one, a map of two
// axes), boxes of box_rows x 64 elements, 128-byte swizzle, zeros past the edges.
struct Matrix {
    const void *ptr;
    int64_t rows, cols, stride;
    int64_t depth, depth_stride;
};

bool encode(CUtensorMap *map, const Matrix &m, uint32_t box_rows) {
    const cuuint64_t dim[3] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows),
                               static_cast<cuuint64_t>(m.depth)};
    // the strides of axes of one element count for nothing but have to be valid
    const cuuint64_t step = static_cast<cuuint64_t>(m.rows > 1 ? m.stride : m.cols) * 2;
    const cuuint64_t stride[2] = {step, m.depth > 1 ? static_cast<cuuint64_t>(m.depth_stride) * 2 : step * dim[1]};
    const cuuint32_t box[3] = {64u, box_rows, 1u}, one[3] = {1u, 1u, 1u};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, m.depth > 0 ? 3 : 2, const_cast<void *>(m.ptr), dim, stride, box,
                     one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Call {
    Matrix P, Q, D;
    Matrix U, H;           // LORA: up, and h as 16-bit numbers
    GroupParams p;
    int max_clusters;
    int sms;
    cudaStream_t stream;
};

uint32_t band_inverse(int64_t i_tiles) {
    const uint64_t band = static_cast<uint64_t>(i_tiles) * kGroupBand;
    return static_cast<uint32_t>(((uint64_t(1) << 32) + band - 1) / band);
}

// What TileWalk moves on by.  A group's last rows are a tile that costs less, and such come again
// after as many tiles as a band has.  Where that number and `clusters` have a common factor, some
// clusters would get only such tiles and others none: then a turn with which clusters + turn has
// none of the widths' factors 2, 3, 5 and 7.  4096 x 4096, 76 pairs, with and without, us:
//   16 groups of 300 rows (2 tiles)  130, 140      8 of 1400 (6)  211, 215   weights 32 of 16, 1416 x 2040 (6)  41.9, 42.9
//   8 of 700 (3)                     119, 117      8 of 1030 (5)  170, 169   (no common factor: without)
// Adapters share one matrix, which a turn spreads over more tiles at a time: 11 requests of 372 rows (2)
// 109, 107; without.
int32_t turn_of(int mode, const GroupParams &p, int tile, int64_t clusters) {
    if (mode == kGroupLora || mode == kGroupDown || p.groups == 0) return 0;
    const int64_t each = mode == kGroupTN ? p.J : (static_cast<int64_t>(p.rows) + p.groups - 1) / p.groups;
    const int64_t j_tiles = (each + tile - 1) / tile, width = j_tiles < kGroupBand ? j_tiles : kGroupBand;
    bool common = false;
    for (int64_t d = 2; d <= width; ++d) common = common || (width % d == 0 && clusters % d == 0);
    static_assert(kGroupBand <= 10, "the widths' factors");
    for (int32_t turn = 0; common && turn < clusters; ++turn) {
        const int64_t n = clusters + turn;
        if (n % 2 != 0 && n % 3 != 0 && n % 5 != 0 && n % 7 != 0) return turn;
    }
    return 0;
}

template <typename... P>
int launch_clusters(void (*kernel)(P...), dim3 grid, unsigned threads, dim3 cluster, size_t smem, cudaStream_t stream,
                    const P &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

template <typename... P>
int launch_cluster(void (*kernel)(P...), int64_t ctas, unsigned threads, unsigned cluster, size_t smem, cudaStream_t stream,
                   const P &...args) {
    return launch_clusters(kernel, dim3(static_cast<unsigned>(ctas)), threads, dim3(cluster), smem, stream, args...);
}

// Maps of sums over rows with boxes of 2^k rows.
template <int MODE>
bool encode_tails(const Call &c, GroupTails<MODE> *tails) {
    if constexpr (MODE == kGroupTN) {
        for (uint32_t k = 0; k < 5 && c.p.rows > 0; ++k) {
            if (!encode(&tails->P[k], c.P, 1u << k) || !encode(&tails->Q[k], c.Q, 1u << k)) return false;
        }
    }
    return true;
}

// Clusters of a kernel that run at once on the current device, asked once of each; 0: an error.  `fit` is the kernel's.
template <typename K>
int clusters_at_once(K *kernel, unsigned ctas, unsigned threads, size_t smem, std::atomic<int> (&fit)[kMaxDevices]) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int clusters = fit[dev].load(std::memory_order_relaxed);
    if (clusters > 0) return clusters;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters <= 0) {
        cudaGetLastError();
        return 0;
    }
    fit[dev].store(clusters, std::memory_order_relaxed);
    return clusters;
}

template <int CG, int TN, int MODE>
int launch_tile(const Call &c) {
    using C = GroupShape<CG, TN, MODE>;
    auto *kernel = grouped_kernel<CG, TN, MODE>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, C::SMEM_ALLOC, done)) return GEMM_ERR_CUDA;
    GroupParams p = c.p;
    const int64_t i_tiles = (static_cast<int64_t>(p.I) + 128 * CG - 1) / (128 * CG);
    const int64_t j_tiles = MODE == kGroupTN ? (static_cast<int64_t>(p.J) + TN - 1) / TN : 0;
    const int64_t groups = MODE == kGroupLora ? int64_t(p.groups) + 2 : p.groups;
    const int64_t most = MODE == kGroupTN ? p.groups * i_tiles * j_tiles : most_tiles(p.rows, groups, TN) * i_tiles;
    if (most > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    p.i_tiles = static_cast<int32_t>(i_tiles);
    p.band_inverse = band_inverse(i_tiles);
    p.j_tiles = static_cast<int32_t>(j_tiles);
    CUtensorMap tmP = {}, tmQ = {}, tmD = {}, tmU = {}, tmH = {};  // P's and Q's are not used by sums of nothing
    if (MODE != kGroupDown && !encode(&tmD, c.D, 32)) return GEMM_ERR_CUDA;
    if (MODE == kGroupLora && p.groups > 0) {
        if (!encode(&tmU, c.U, 128) || !encode(&tmH, c.H, C::Q_BOX)) return GEMM_ERR_CUDA;
    }
    if (groups > 0 && c.P.rows > 0 && c.P.cols > 0 && c.Q.rows > 0 && c.Q.cols > 0) {
        const uint32_t p_rows = MODE == kGroupDown ? static_cast<uint32_t>(p.rank) : (MODE == kGroupNN || MODE == kGroupTN ? 64 : 128);
        if (!encode(&tmP, c.P, p_rows) || !encode(&tmQ, c.Q, C::Q_BOX)) {
            return GEMM_ERR_CUDA;
        }
    }
    GroupTails<MODE> tails = {};
    if (!encode_tails(c, &tails)) return GEMM_ERR_CUDA;
    int64_t grid = c.sms / CG;
    if constexpr (CG == 2) {
        static std::atomic<int> fit[kMaxDevices];
        grid = clusters_at_once(kernel, 2, C::THREADS, C::SMEM_ALLOC, fit);
        if (grid == 0) return GEMM_ERR_CUDA;
    }
    if (!p.zero_rest && most < grid) grid = most;
    if (c.max_clusters > 0 && c.max_clusters < grid) grid = c.max_clusters;
    if (grid == 0) return GEMM_OK;
    p.turn = turn_of(MODE, p, TN, grid);
    return launch_cluster(kernel, CG * grid, C::THREADS, CG, C::SMEM_ALLOC, c.stream, tmP, tmQ, tmD, tmU, tmH, tails, p);
}

template <int TN, int KS, int MODE>
int launch_few(const Call &c) {
    using C = FewShape<TN, MODE == kGroupLora>;
    auto *kernel = grouped_few_kernel<TN, KS, MODE>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, C::smem(C::ALONE), done)) return GEMM_ERR_CUDA;
    GroupParams p = c.p;
    const int64_t i_tiles = (static_cast<int64_t>(p.I) + 127) / 128;
    const int64_t j_tiles = MODE == kGroupTN ? (static_cast<int64_t>(p.J) + TN - 1) / TN : 0;
    const int64_t most = MODE == kGroupTN ? p.groups * i_tiles * j_tiles : most_tiles(p.rows, MODE == kGroupLora ? 1 : p.groups, TN) * i_tiles;
    if (most * KS > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    p.i_tiles = static_cast<int32_t>(i_tiles);
    p.j_tiles = static_cast<int32_t>(j_tiles);
    p.band_inverse = band_inverse(i_tiles);
    CUtensorMap tmP = {}, tmQ = {}, tmU = {}, tmH = {};  // not used by sums of nothing
    if (c.P.rows > 0 && c.P.cols > 0 && c.Q.rows > 0 && c.Q.cols > 0) {
        if (!encode(&tmP, c.P, MODE == kGroupNN || MODE == kGroupTN ? 64 : 128) || !encode(&tmQ, c.Q, MODE == kGroupTN ? 64 : TN)) {
            return GEMM_ERR_CUDA;
        }
    }
    GroupTails<MODE> tails = {};
    if (!encode_tails(c, &tails)) return GEMM_ERR_CUDA;
    if (MODE == kGroupLora && p.groups > 0) {
        if (!encode(&tmU, c.U, 128) || !encode(&tmH, c.H, 16)) return GEMM_ERR_CUDA;
    }
    const int64_t tiles = most > 0 ? most : 1;  // one for the rows without a group
    int stages = C::ALONE;
    if constexpr (MODE != kGroupLora) {
        // An SM for each CTA while all clusters have that at once (one lies within a GPC, and clusters of 8 and 4 leave
        // some SMs of one without).  Past that two share an SM: 1 x 2048 x 4096, 16 clusters of 8 where 15 have SMs
        // of their own, 5.3 us; where the last waits for them 9.1.
        int64_t alone = c.sms;
        if constexpr (KS > 1) {
            static std::atomic<int> fit[kMaxDevices];
            alone = clusters_at_once(kernel, KS, C::THREADS, static_cast<size_t>(C::smem(C::ALONE)), fit);
            if (alone == 0) return GEMM_ERR_CUDA;
        }
        if (tiles > alone) stages = C::PAIRED;
    }
    return launch_cluster(kernel, KS * tiles, C::THREADS, KS, static_cast<size_t>(C::smem(stages)), c.stream, tmP, tmQ, tmU, tmH, tails,
                          p, stages);
}

template <int TN, int MODE>
int launch_split(const Call &c, int split) {
    switch (split) {
        case 8: return launch_few<TN, 8, MODE>(c);
        case 4: return launch_few<TN, 4, MODE>(c);
        case 2: return launch_few<TN, 2, MODE>(c);
        default: return launch_few<TN, 1, MODE>(c);
    }
}

template <int MODE>
int launch_few_mode(const Call &c, int tile, int split) {
    switch (tile) {
        case 16:
            if constexpr (MODE != kGroupTN) return launch_split<16, MODE>(c, split);
        case 32:
            if constexpr (MODE != kGroupTN) return launch_split<32, MODE>(c, split);
        case 64: return launch_split<64, MODE>(c, split);
        default: return launch_split<128, MODE>(c, split);
    }
}

template <int MODE>
int launch_mode(const Call &c, const Choice &how) {
    if (how.split > 0) return launch_few_mode<MODE>(c, how.tile, how.split);
    if constexpr (MODE != kGroupTN) {
        if (how.tile == 32) return launch_tile<1, 32, MODE>(c);
    }
    switch (how.tile) {
        case 64: return launch_tile<1, 64, MODE>(c);
        case 128: return launch_tile<1, 128, MODE>(c);
        default: return launch_tile<2, 256, MODE>(c);
    }
}

int check_options(const grouped_options *opts, grouped_options *o) {
    *o = opts ? *opts : grouped_options{};
    if ((o->tile != 0 && o->tile != 16 && o->tile != 32 && o->tile != 64 && o->tile != 128 && o->tile != 256) ||
        (o->split != 0 && o->split != -1 && o->split != 1 && o->split != 2 && o->split != 4 && o->split != 8) ||
        o->max_clusters < 0 || (o->debug_flags & ~1) != 0 || o->timeout_ns < 0) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (o->timeout_ns == 0) o->timeout_ns = kDefaultTimeoutNs;
    return GEMM_OK;
}

// One operand: its rows step by whole 16-byte units, at least a row's width apart.
int check_matrix(const Matrix &m) {
    if (m.rows == 0 || m.cols == 0) return GEMM_OK;
    if (!m.ptr || (m.rows > 1 && m.stride < m.cols) || m.depth_stride < 0) return GEMM_ERR_INVALID_ARG;
    if (m.depth > 1 && m.depth_stride < (m.rows - 1) * m.stride + m.cols) return GEMM_ERR_INVALID_ARG;
    if (!aligned(m.ptr, 16) || (m.rows > 1 && m.stride % 8 != 0) || (m.depth > 1 && m.depth_stride % 8 != 0)) {
        return GEMM_ERR_MISALIGNED;
    }
    return GEMM_OK;
}

int64_t matrix_bytes(const Matrix &m) {
    if (m.rows <= 0 || m.cols <= 0) return 0;
    const int64_t one = (m.rows > 1 ? (m.rows - 1) * m.stride : 0) + m.cols;
    return 2 * (one + (m.depth > 1 ? (m.depth - 1) * m.depth_stride : 0));
}

// Whether two matrices of as many rows share memory; rows of one stride may lie between each other's.
bool rows_shared(const Matrix &m, const Matrix &n) {
    return rows_overlap(m.ptr, 2 * m.cols, m.rows > 1 ? 2 * m.stride : 0, n.ptr, 2 * n.cols, n.rows > 1 ? 2 * n.stride : 0, m.rows);
}

// The checks that all three directions share, and the launch.
int grouped(int mode, Matrix ragged, Matrix other, Matrix out, const void *offsets, int32_t offsets_type, int64_t rows,
            int64_t groups, int64_t N, int64_t K, int32_t type, int32_t zero_rest, void *stream,
            const grouped_options *opts) {
    grouped_options o;
    int st = check_options(opts, &o);
    if (st != GEMM_OK) return st;
    if (rows < 0 || groups < 0 || N < 0 || K < 0 || (type != LINEAR_F16 && type != LINEAR_BF16) ||
        (offsets_type != 0 && offsets_type != 1) || (o.tile == 256 && o.split > 0) || (o.tile == 16 && o.split < 0) ||
        (mode == kGroupTN && o.tile != 0 && o.tile < 64)) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (N % 8 != 0 || K % 8 != 0 || rows > kMaxDim || N > kMaxDim || K > kMaxDim || groups > GROUPED_MAX_GROUPS) {
        return GEMM_ERR_UNSUPPORTED_SHAPE;
    }
    const bool nothing = mode == kGroupTN ? groups == 0 || N == 0 || K == 0 : rows == 0 || out.cols == 0;
    if (nothing) return GEMM_OK;
    if (!offsets || !out.ptr) return GEMM_ERR_INVALID_ARG;
    for (const Matrix *m : {&ragged, &other, &out}) {
        st = check_matrix(*m);
        if (st != GEMM_OK) return st;
    }
    if (!aligned(offsets, offsets_type ? 8 : 4)) return GEMM_ERR_MISALIGNED;
    const int64_t out_bytes = matrix_bytes(out);
    if ((mode == kGroupTN ? overlap(out.ptr, out_bytes, ragged.ptr, matrix_bytes(ragged)) : rows_shared(out, ragged)) ||
        overlap(out.ptr, out_bytes, other.ptr, matrix_bytes(other)) ||
        overlap(out.ptr, out_bytes, offsets, (groups + 1) * (offsets_type ? 8 : 4))) {
        return GEMM_ERR_INVALID_ARG;
    }
    Call c = {};
    st = gb300_sms(&c.sms);
    if (st != GEMM_OK) return st;
    if (!encoder()) return GEMM_ERR_CUDA;
    c.P = other;
    c.Q = ragged;
    c.D = out;
    c.max_clusters = o.max_clusters;
    c.stream = static_cast<cudaStream_t>(stream);
    GroupParams &p = c.p;
    p.offsets = offsets;
    p.offsets_64 = offsets_type;
    p.out = const_cast<void *>(out.ptr);
    p.out_row = out.rows > 1 ? out.stride : 0;
    p.out_group = out.depth > 1 ? out.depth_stride : 0;
    p.groups = static_cast<int32_t>(groups);
    p.rows = static_cast<int32_t>(rows);
    p.I = static_cast<int32_t>(out.cols);
    p.J = static_cast<int32_t>(mode == kGroupTN ? N : 0);
    p.R = static_cast<int32_t>(mode == kGroupNT ? K : N);
    p.bf16 = type == LINEAR_BF16;
    p.zero_rest = zero_rest != 0;
    p.debug_flags = static_cast<uint32_t>(o.debug_flags);
    p.timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    const Choice how = choose(mode, p, c.sms, o);
    switch (mode) {
        case kGroupNT: return launch_mode<kGroupNT>(c, how);
        case kGroupNN: return launch_mode<kGroupNN>(c, how);
        default: return launch_mode<kGroupTN>(c, how);
    }
}

// ------------------------------------------------------------- adapters --

constexpr int64_t kMaxRank = 128;

struct Lora {
    Matrix x, W, down, up, D;
    const float *scales;
    const void *offsets;
    const int32_t *adapters;
    int64_t rows, requests, adapter_count, N, K, rank;
    void *workspace;
};

// h, by CUDA cores, whose time goes with rows and ranks, or by the tensor cores in tiles of one
// request each, whose time hardly does: about alike from 10 to 18 thousand rows x ranks on.  A whole
// call of 4096 x 4096, by the former and the latter, us:
//   64 requests of 1 row, rank 16   16.9, 30.5    64 of 4, 32   32.8, 40.4    128 of 4, 16   49.6, 59.0
//   2 of 64, 64                     21.3, 21.6    64 of 4, 64   48.3, 41.8    128 of 4, 64   80.5, 62.3
//   2 of 64, 128                    29.6, 22.1    1 of 256, 64  34.3, 22.8
//   fp16: 64 of 1, 16               18.4, 31.0    2 of 64, 64   19.4, 21.8    1 of 90, 128   27.2, 22.4
constexpr int64_t kDownByCores = 12288;

// Of fp16 a row's CTAs agree on the power of two that its h is held in, so they are a cluster; and tiles of 256 rows
// take h from the tensor cores' launch, which leaves what they ask of each 32 rows.
int lora_down(Call &c, const Lora &l, const Choice &how) {
    if (c.p.groups == 0) return GEMM_OK;
    int st;
    if (l.rows * l.rank <= kDownByCores && (c.p.bf16 || how.tile != 256)) {
        const int64_t padded = (l.rank + 15) / 16 * 16;
        int64_t ranks = 4, each = 1, parts = padded / ranks;  // a CTA's at a time, how many times, CTAs of a row
        if (c.p.bf16) {
            // three CTAs an SM, with as few ranks each as that allows
            while (each < padded / ranks && l.rows * parts > 3 * c.sms) {
                ++each;
                parts = (padded / ranks + each - 1) / each;
            }
        } else if (l.rows <= 2) {
            // the chain is what counts: all at once, in a cluster's 8 CTAs.  A stream of calls of one row, rank 16, 10.8 us
            // (two CTAs with two turns 12.0, one 11.2), rank 64 11.0 (8 with two turns 12.7)
            while (padded / ranks > 8) ranks *= 2;
            parts = padded / ranks;
        } else if (l.rank <= 16 && l.rows <= 32) {
            // one CTA, which agrees with itself: 16 rows 11.7 us, clusters of 4 13.1
            ranks = 16, parts = 1;
        } else {
            // clusters that all run at once, of CTAs with two turns at least: 64 rows of rank 64, 4 CTAs each 13.8 us, 6
            // 18.6, 8 16.8; 128 of rank 32, 2 15.6, 4 18.4
            const int64_t units = padded / ranks;
            for (parts = 1; parts < 8 && 4 * parts <= units && 2 * parts * l.rows <= 256;) parts *= 2;
            each = (units + parts - 1) / parts;
        }
        const DownParams d = {static_cast<const uint16_t *>(l.x.ptr), static_cast<const uint16_t *>(l.down.ptr), l.x.stride,
                              l.down.stride, l.down.depth_stride, static_cast<uint16_t *>(l.workspace), static_cast<int32_t>(each)};
        const dim3 grid(static_cast<unsigned>(l.rows), static_cast<unsigned>(parts)), cluster(1, static_cast<unsigned>(parts));
        st = c.p.bf16      ? launch(lora_down_kernel<false, 4>, grid, dim3(256), 0, c.stream, c.p, d)
             : ranks == 16 ? launch_clusters(lora_down_kernel<true, 16>, grid, 1024, cluster, 0, c.stream, c.p, d)
             : ranks == 8  ? launch_clusters(lora_down_kernel<true, 8>, grid, 512, cluster, 0, c.stream, c.p, d)
                           : launch_clusters(lora_down_kernel<true, 4>, grid, 256, cluster, 0, c.stream, c.p, d);
    } else {
        Call d = c;
        d.P = l.down;
        d.Q = l.x;
        d.p.I = c.p.rank;
        d.p.out = l.workspace;
        d.p.out_row = 2 * c.p.rank_pad;
        d.max_clusters = 0;
        st = launch_tile<1, 32, kGroupDown>(d);
    }
    c.p.follows = 1;
    return st;
}

// Requests of many rows: tiles of one request each, the adapter as more of the sum.
// Requests of few: tiles of any rows, the adapters run by run.
int lora(Call &c, const Lora &l, const Choice &how) {
    const int st = lora_down(c, l, how);
    if (st != GEMM_OK) return st;
    c.P = l.W;
    c.Q = l.x;
    c.D = l.D;
    c.U = l.up;
    c.H = {l.workspace, l.rows, 2 * c.p.rank_pad, 2 * c.p.rank_pad, 0, 0};
    return how.tile == 256 ? launch_tile<2, 256, kGroupLora>(c) : launch_few_mode<kGroupLora>(c, how.tile, how.split);
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int grouped_gemm_nt(const void *A, int64_t lda, const void *B, int64_t ldb, int64_t b_stride, const void *offsets,
                    int32_t offsets_type, void *D, int64_t ldd, int64_t rows, int64_t groups, int64_t N, int64_t K,
                    int32_t type, int32_t zero_rest, void *stream, const grouped_options *opts) {
    return grouped(kGroupNT, {A, rows, K, lda, 0, 0}, {B, groups ? N : 0, K, ldb, groups, b_stride}, {D, rows, N, ldd, 0, 0}, offsets,
                   offsets_type, rows, groups, N, K, type, zero_rest, stream, opts);
}

int grouped_gemm_nn(const void *dD, int64_t ldd, const void *B, int64_t ldb, int64_t b_stride, const void *offsets,
                    int32_t offsets_type, void *dA, int64_t lda, int64_t rows, int64_t groups, int64_t N, int64_t K,
                    int32_t type, int32_t zero_rest, void *stream, const grouped_options *opts) {
    return grouped(kGroupNN, {dD, rows, N, ldd, 0, 0}, {B, groups ? N : 0, K, ldb, groups, b_stride}, {dA, rows, K, lda, 0, 0},
                   offsets, offsets_type, rows, groups, N, K, type, zero_rest, stream, opts);
}

int grouped_gemm_tn(const void *dD, int64_t ldd, const void *A, int64_t lda, const void *offsets, int32_t offsets_type,
                    void *dB, int64_t ldb, int64_t b_stride, int64_t rows, int64_t groups, int64_t N, int64_t K,
                    int32_t type, void *stream, const grouped_options *opts) {
    return grouped(kGroupTN, {dD, rows, N, ldd, 0, 0}, {A, rows, K, lda, 0, 0}, {dB, N, K, ldb, groups, b_stride},
                   offsets, offsets_type, rows, groups, N, K, type, 0, stream, opts);
}

int64_t gemm_lora_workspace_size(int64_t rows, int64_t rank) {
    if (rows < 0 || rank < 0) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxDim || rank > kMaxRank || rank % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return rows * ((rank + 63) / 64 * 64 * 4 + 8);  // two 16-bit numbers; of a row, row_scale and some_scaled
}

int gemm_lora_nt(const void *x, int64_t ldx, const void *W, int64_t ldw, const void *down, int64_t ld_down,
                 int64_t down_stride, const void *up, int64_t ld_up, int64_t up_stride, const float *scales,
                 const void *offsets, int32_t offsets_type, const int32_t *adapters, void *D, int64_t ldd, int64_t rows,
                 int64_t requests, int64_t adapter_count, int64_t N, int64_t K, int64_t rank, int32_t type,
                 void *workspace, int64_t workspace_bytes, void *stream, const grouped_options *opts) {
    grouped_options o;
    int st = check_options(opts, &o);
    if (st != GEMM_OK) return st;
    if (rows < 0 || requests < 0 || adapter_count < 0 || N < 0 || K < 0 || rank < 0 || workspace_bytes < 0 ||
        (type != LINEAR_F16 && type != LINEAR_BF16) || (offsets_type != 0 && offsets_type != 1) ||
        (o.tile == 256 && o.split > 0) || (o.tile != 0 && o.tile < 256 && o.split < 0)) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (N % 8 != 0 || K % 8 != 0 || rank % 8 != 0 || rank > kMaxRank || rows > kMaxDim || N > kMaxDim || K > kMaxDim ||
        adapter_count > kMaxDim || requests > GROUPED_MAX_GROUPS) {
        return GEMM_ERR_UNSUPPORTED_SHAPE;
    }
    if (rows == 0 || N == 0) return GEMM_OK;
    const bool some = requests > 0 && adapter_count > 0 && rank > 0 && K > 0;  // adapters at all
    Lora l = {{x, rows, K, ldx, 0, 0}, {W, N, K, ldw, 1, 0}, {down, rank, K, ld_down, adapter_count, down_stride},
              {up, N, rank, ld_up, adapter_count, up_stride}, {D, rows, N, ldd, 0, 0}, scales, offsets, adapters,
              rows, requests, adapter_count, N, K, rank, workspace};
    if (!D || (requests > 0 && (!offsets || !adapters))) return GEMM_ERR_INVALID_ARG;
    for (const Matrix *m : {&l.x, &l.W, &l.D}) {
        st = check_matrix(*m);
        if (st != GEMM_OK) return st;
    }
    if (some) {
        for (const Matrix *m : {&l.down, &l.up}) {
            st = check_matrix(*m);
            if (st != GEMM_OK) return st;
        }
        if (!workspace) return GEMM_ERR_INVALID_ARG;
        if (workspace_bytes < gemm_lora_workspace_size(rows, rank)) return GEMM_ERR_SCRATCH_LIMIT;
    }
    if (!aligned(offsets, offsets_type ? 8 : 4) || !aligned(adapters, 4) || !aligned(scales, 4) || !aligned(workspace, 16)) {
        return GEMM_ERR_MISALIGNED;
    }
    const struct {
        const void *p;
        int64_t bytes;
    } outs[2] = {{D, matrix_bytes(l.D)}, {workspace, some ? gemm_lora_workspace_size(rows, rank) : 0}},
      ins[6] = {{W, matrix_bytes(l.W)}, {down, some ? matrix_bytes(l.down) : 0},
                {up, some ? matrix_bytes(l.up) : 0}, {offsets, (requests + 1) * (offsets_type ? 8 : 4)},
                {adapters, requests * 4}, {scales, adapter_count * 4}};
    for (const auto &out : outs) {
        for (const auto &in : ins) {
            if (overlap(out.p, out.bytes, in.p, in.bytes)) return GEMM_ERR_INVALID_ARG;
        }
    }
    if (rows_shared(l.D, l.x) || overlap(workspace, outs[1].bytes, x, matrix_bytes(l.x)) ||
        overlap(outs[0].p, outs[0].bytes, outs[1].p, outs[1].bytes)) {
        return GEMM_ERR_INVALID_ARG;
    }
    Call c = {};
    st = gb300_sms(&c.sms);
    if (st != GEMM_OK) return st;
    if (!encoder()) return GEMM_ERR_CUDA;
    c.stream = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        const cudaError_t e = cudaMemset2DAsync(D, static_cast<size_t>(rows > 1 ? ldd : N) * 2, 0, static_cast<size_t>(N) * 2,
                                                static_cast<size_t>(rows), c.stream);
        return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
    }
    c.max_clusters = o.max_clusters;
    GroupParams &p = c.p;
    p.offsets = some ? offsets : nullptr;
    p.offsets_64 = offsets_type;
    p.out = D;
    p.out_row = rows > 1 ? ldd : 0;
    p.groups = some ? static_cast<int32_t>(requests) : 0;
    p.rows = static_cast<int32_t>(rows);
    p.I = static_cast<int32_t>(N);
    p.R = static_cast<int32_t>(K);
    p.bf16 = type == LINEAR_BF16;
    p.adapters = adapters;
    p.scales = scales;
    p.adapter_count = static_cast<int32_t>(adapter_count);
    p.rank = static_cast<int32_t>(rank);
    p.rank_pad = static_cast<int32_t>((rank + 63) / 64 * 64);
    if (some) {
        p.row_scale = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + rows * p.rank_pad * 4);
        p.some_scaled = reinterpret_cast<int32_t *>(p.row_scale + rows);
    }
    p.debug_flags = static_cast<uint32_t>(o.debug_flags);
    p.timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    if (rows == 1) l.x.stride = 0;
    const Choice how = choose_lora(p, c.sms, o);
    return lora(c, l, how);
}

int grouped_last_device_status(void *stream, uint64_t *info) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    int status = 0;
    unsigned long long where = 0;
    const int zero = 0;
    const unsigned long long zero64 = 0;
    if (cudaMemcpyFromSymbol(&status, g_group_status, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&where, g_group_info, sizeof(where)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_group_status, &zero, sizeof(int)) != cudaSuccess ||
        cudaMemcpyToSymbol(g_group_info, &zero64, sizeof(zero64)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    if (info) *info = where;
    return status;
}

}  // extern "C"
