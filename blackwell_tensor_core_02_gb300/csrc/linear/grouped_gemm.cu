// grouped_gemm.cu -- host side of the products grouped by rows: checks, tensor maps,
// the choice of a tile, launches (see grouped_ops.h).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

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
    GroupParams p;
    int max_clusters;
    int sms;
    cudaStream_t stream;
};

template <int CG, int TN, int MODE>
int launch_tile(const Call &c) {
    using C = GroupShape<CG, TN, MODE>;
    auto *kernel = grouped_kernel<CG, TN, MODE>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, C::SMEM_ALLOC, done)) return GEMM_ERR_CUDA;
    GroupParams p = c.p;
    const int64_t i_tiles = (static_cast<int64_t>(p.I) + 128 * CG - 1) / (128 * CG);
    const int64_t j_tiles = MODE == kGroupTN ? (static_cast<int64_t>(p.J) + TN - 1) / TN : 0;
    // every group's tiles, at most: each group may end in a part of a tile
    const int64_t some = p.groups < p.rows ? p.groups : p.rows;
    const int64_t most = MODE == kGroupTN ? p.groups * i_tiles * j_tiles : (static_cast<int64_t>(p.rows) / TN + some) * i_tiles;
    if (most > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    p.i_tiles = static_cast<int32_t>(i_tiles);
    p.j_tiles = static_cast<int32_t>(j_tiles);
    CUtensorMap tmP = {}, tmQ = {}, tmD = {};  // P's and Q's are not used by sums of nothing
    if (!encode(&tmD, c.D, 32)) return GEMM_ERR_CUDA;
    if (p.groups > 0 && c.P.rows > 0 && c.P.cols > 0 && c.Q.rows > 0 && c.Q.cols > 0) {
        if (!encode(&tmP, c.P, MODE == kGroupNT ? 128 : 64) || !encode(&tmQ, c.Q, MODE == kGroupTN ? 64 : TN / CG)) {
            return GEMM_ERR_CUDA;
        }
    }
    int64_t grid = c.sms / CG;
    if constexpr (CG == 2) {
        static std::atomic<int> fit[kMaxDevices];
        int dev = -1;
        if (cudaGetDevice(&dev) != cudaSuccess) return GEMM_ERR_CUDA;
        int clusters = fit[dev].load(std::memory_order_relaxed);
        if (clusters == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2);
            cfg.blockDim = dim3(C::THREADS);
            cfg.dynamicSmemBytes = C::SMEM_ALLOC;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters <= 0) {
                cudaGetLastError();
                return GEMM_ERR_CUDA;
            }
            fit[dev].store(clusters, std::memory_order_relaxed);
        }
        grid = clusters;
    }
    if (!(MODE != kGroupTN && p.zero_rest) && most < grid) grid = most;
    if (c.max_clusters > 0 && c.max_clusters < grid) grid = c.max_clusters;
    if (grid == 0) return GEMM_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(CG * grid));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM_ALLOC;
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, tmP, tmQ, tmD, static_cast<const GroupParams &>(p)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

// The tile's columns: of the ragged axis by the rows that a group has on average, of
// TN's by the columns.
int choose_tile(int mode, const GroupParams &p) {
    if (mode == kGroupTN) return p.J <= 64 ? 64 : (p.J <= 128 || p.I <= 128 ? 128 : 256);
    const int64_t some = p.groups < p.rows ? p.groups : p.rows;
    const int64_t each = some > 0 ? (p.rows + some - 1) / some : 0;
    return each <= 16 ? 32 : (each <= 32 ? 64 : (each <= 112 || p.I <= 128 ? 128 : 256));
}

template <int MODE>
int launch_mode(const Call &c, int tile) {
    switch (tile) {
        case 32:
            if constexpr (MODE != kGroupTN) return launch_tile<1, 32, MODE>(c);
            return GEMM_ERR_INVALID_ARG;
        case 64: return launch_tile<1, 64, MODE>(c);
        case 128: return launch_tile<1, 128, MODE>(c);
        default: return launch_tile<2, 256, MODE>(c);
    }
}

int check_options(const grouped_options *opts, grouped_options *o) {
    *o = opts ? *opts : grouped_options{};
    if ((o->tile != 0 && o->tile != 32 && o->tile != 64 && o->tile != 128 && o->tile != 256) || o->max_clusters < 0 ||
        (o->debug_flags & ~1) != 0 || o->timeout_ns < 0) {
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

// The checks that all three directions share, and the launch.
int grouped(int mode, Matrix ragged, Matrix other, Matrix out, const void *offsets, int32_t offsets_type, int64_t rows,
            int64_t groups, int64_t N, int64_t K, int32_t type, int32_t zero_rest, void *stream,
            const grouped_options *opts) {
    grouped_options o;
    int st = check_options(opts, &o);
    if (st != GEMM_OK) return st;
    if (rows < 0 || groups < 0 || N < 0 || K < 0 || (type != LINEAR_F16 && type != LINEAR_BF16) ||
        (offsets_type != 0 && offsets_type != 1) || (mode == kGroupTN && o.tile == 32)) {
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
    if (overlap(out.ptr, out_bytes, ragged.ptr, matrix_bytes(ragged)) ||
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
    const int tile = o.tile ? o.tile : choose_tile(mode, p);
    switch (mode) {
        case kGroupNT: return launch_mode<kGroupNT>(c, tile);
        case kGroupNN: return launch_mode<kGroupNN>(c, tile);
        default: return launch_mode<kGroupTN>(c, tile);
    }
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
