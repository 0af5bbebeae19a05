// gemm_fp4.cu -- host side of the product of microscaled 4-bit matrices: checks,
// tensor maps, the choice of a tile, launches (see linear_ops.h).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <mutex>

#include "gemm_fp4_kernel.cuh"

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

// Packed 4-bit rows, tiles of box_rows x 128 bytes, 128-byte swizzle, zeros past
// the edges.
bool encode_data(CUtensorMap *map, const void *ptr, int64_t rows, int64_t K, uint32_t box_rows) {
    const cuuint64_t bytes = static_cast<cuuint64_t>(fp4_padded_cols(K) / 2);
    const cuuint64_t dim[2] = {bytes, static_cast<cuuint64_t>(rows)}, stride[1] = {bytes};
    const cuuint32_t box[2] = {128u, box_rows}, step[2] = {1u, 1u};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dim, stride, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles of 512 bytes as [row tiles][tiles along K][128 words]; boxes of
// one stage's tiles of `row_tiles` row tiles.
bool encode_scales(CUtensorMap *map, const void *ptr, int64_t rows, int64_t K, bool nv, uint32_t row_tiles) {
    const cuuint64_t along = static_cast<cuuint64_t>(fp4_scale_tiles(K, nv));
    const cuuint64_t dim[3] = {128, along, static_cast<cuuint64_t>((rows + 127) / 128)};
    const cuuint64_t stride[2] = {kScaleTileBytes, along * kScaleTileBytes};
    const cuuint32_t box[3] = {128u, nv ? 4u : 2u, row_tiles}, step[3] = {1u, 1u, 1u};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, const_cast<void *>(ptr), dim, stride, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_d(CUtensorMap *map, void *ptr, int64_t M, int64_t N) {
    const cuuint64_t dim[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(N) * 2};
    const cuuint32_t box[2] = {64u, 32u}, step[2] = {1u, 1u};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, ptr, dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... P>
cudaError_t launch_cluster(void (*kernel)(P...), unsigned ctas, unsigned threads, unsigned cluster, size_t smem,
                           cudaStream_t stream, const P &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

struct Call {
    const void *A, *A_scales, *B, *B_scales;
    void *D;
    int64_t M, N, K;
    int32_t d_type;
    float first, alpha;  // of split_factor()
    cudaStream_t stream;
    gemm_fp4_options o;  // resolved: tile, cluster_k and swap set
};

template <int BN, int KS, bool NV>
int launch_single(const Call &c) {
    using C = Fp4Single<BN, KS, NV>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(fp4_single_kernel<BN, KS, NV>, C::SMEM_ALLOC, done)) return GEMM_ERR_CUDA;
    const bool swap = c.o.swap == 2;
    const void *P = swap ? c.B : c.A, *Q = swap ? c.A : c.B;
    const void *SP = swap ? c.B_scales : c.A_scales, *SQ = swap ? c.A_scales : c.B_scales;
    const int64_t p_rows = swap ? c.N : c.M, q_rows = swap ? c.M : c.N;
    CUtensorMap tmP, tmQ, tmSP, tmSQ;
    if (!encode_data(&tmP, P, p_rows, c.K, 128) || !encode_data(&tmQ, Q, q_rows, c.K, BN) ||
        !encode_scales(&tmSP, SP, p_rows, c.K, NV, 1) || !encode_scales(&tmSQ, SQ, q_rows, c.K, NV, 1)) {
        return GEMM_ERR_CUDA;
    }
    Fp4Params p = {};
    p.M = static_cast<int32_t>(c.M);
    p.N = static_cast<int32_t>(c.N);
    p.m_tiles = static_cast<int32_t>((p_rows + 127) / 128);
    p.n_tiles = static_cast<int32_t>((q_rows + BN - 1) / BN);
    p.k_tiles = static_cast<int32_t>((c.K + 255) / 256);
    p.d_type = c.d_type;
    p.swap = swap;
    p.wide_store = c.N % 4 == 0 && aligned(c.D, 4 * type_size(c.d_type));
    p.debug_flags = static_cast<uint32_t>(c.o.debug_flags);
    p.timeout_ns = static_cast<uint64_t>(c.o.timeout_ns);
    p.first = c.first;
    p.alpha = c.alpha;
    p.D = c.D;
    const int64_t ctas = static_cast<int64_t>(p.m_tiles) * p.n_tiles * KS;
    if (ctas > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return launch_cluster(fp4_single_kernel<BN, KS, NV>, static_cast<unsigned>(ctas), C::THREADS, KS, C::SMEM_ALLOC,
                          c.stream, tmP, tmQ, tmSP, tmSQ, p) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_LAUNCH;
}

template <bool NV>
int launch_pair(const Call &c) {
    using C = Fp4Pair<NV>;
    static std::atomic<uint64_t> done{0};
    static std::atomic<int> fit[kMaxDevices];
    if (!allow_smem(fp4_pair_kernel<NV>, C::SMEM_ALLOC, done)) return GEMM_ERR_CUDA;
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
        if (cudaOccupancyMaxActiveClusters(&clusters, fp4_pair_kernel<NV>, &cfg) != cudaSuccess || clusters <= 0) {
            cudaGetLastError();
            return GEMM_ERR_CUDA;
        }
        fit[dev].store(clusters, std::memory_order_relaxed);
    }
    Fp4Params p = {};
    p.M = static_cast<int32_t>(c.M);
    p.N = static_cast<int32_t>(c.N);
    const int64_t m_tiles = (c.M + 255) / 256, n_tiles = (c.N + 255) / 256;
    if (m_tiles * n_tiles > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    p.m_tiles = static_cast<int32_t>(m_tiles);
    p.n_tiles = static_cast<int32_t>(n_tiles);
    p.k_tiles = static_cast<int32_t>((c.K + 255) / 256);
    // a group's panel of A, a quarter of fp16's bytes, in 32 MiB of L2
    p.raster_group = gemm_f16::auto_raster_group(p.m_tiles, (c.K + 3) / 4, 256);
    p.d_type = c.d_type;
    p.tma_store = c.d_type != LINEAR_F32 && c.N % 8 == 0 && aligned(c.D, 16);
    p.debug_flags = static_cast<uint32_t>(c.o.debug_flags);
    p.timeout_ns = static_cast<uint64_t>(c.o.timeout_ns);
    p.first = c.first;
    p.alpha = c.alpha;
    p.D = c.D;
    CUtensorMap tmA, tmB, tmSA, tmSB, tmD;
    if (!encode_data(&tmA, c.A, c.M, c.K, 128) || !encode_data(&tmB, c.B, c.N, c.K, 128) ||
        !encode_scales(&tmSA, c.A_scales, c.M, c.K, NV, 1) || !encode_scales(&tmSB, c.B_scales, c.N, c.K, NV, 2)) {
        return GEMM_ERR_CUDA;
    }
    if (!p.tma_store) {
        tmD = tmA;  // not used
    } else if (!encode_d(&tmD, c.D, c.M, c.N)) {
        return GEMM_ERR_CUDA;
    }
    int64_t grid = m_tiles * n_tiles < clusters ? m_tiles * n_tiles : clusters;
    if (c.o.max_clusters > 0 && c.o.max_clusters < grid) grid = c.o.max_clusters;
    return launch_cluster(fp4_pair_kernel<NV>, static_cast<unsigned>(2 * grid), C::THREADS, 2, C::SMEM_ALLOC, c.stream,
                          tmA, tmB, tmSA, tmSB, tmD, p) == cudaSuccess
               ? GEMM_OK
               : GEMM_ERR_LAUNCH;
}

template <int BN, bool NV>
int launch_ks(const Call &c) {
    switch (c.o.cluster_k) {
        case 8: return launch_single<BN, 8, NV>(c);
        case 4: return launch_single<BN, 4, NV>(c);
        case 2: return launch_single<BN, 2, NV>(c);
        default: return launch_single<BN, 1, NV>(c);
    }
}

template <bool NV>
int launch_fp4(const Call &c) {
    switch (c.o.tile) {
        case 16: return launch_ks<16, NV>(c);
        case 32: return launch_ks<32, NV>(c);
        case 64: return launch_ks<64, NV>(c);
        case 128: return launch_ks<128, NV>(c);
        default: return launch_pair<NV>(c);
    }
}

int check_options(const gemm_fp4_options *opts, gemm_fp4_options *o) {
    *o = opts ? *opts : gemm_fp4_options{};
    if ((o->tile != 0 && o->tile != 16 && o->tile != 32 && o->tile != 64 && o->tile != 128 && o->tile != 256) ||
        (o->cluster_k != 0 && o->cluster_k != 1 && o->cluster_k != 2 && o->cluster_k != 4 && o->cluster_k != 8) ||
        o->swap < 0 || o->swap > 2 || o->max_clusters < 0 || o->exponent < -1000 || o->exponent > 1000 || (o->debug_flags & ~1) != 0 || o->timeout_ns < 0 ||
        (o->tile == 256 && (o->cluster_k > 1 || o->swap != 0))) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (o->timeout_ns == 0) o->timeout_ns = kDefaultTimeoutNs;
    return GEMM_OK;
}

// The result's factor f = alpha * 2^exponent as the kernels take it: the sum times
// `first`, a power of two, times `alpha`.  first is 1 where f is a normal fp32
// number, a zero or not finite.  Beyond, a sum of FP4_NV codes times scales is 0 or in
// [2^-20, 2^51] (K < 2^28), so the sum times first stays exact and the one rounding is
// the second product's; where alpha ends at its largest, or with fewer bits, the
// result is an infinity or 0 whatever the sum.
void split_factor(double f, float *first, float *alpha) {
    constexpr double kLeast = 0x1p-126, kMost = 0x1.fffffep127;
    const double size = std::fabs(f);
    int shift = 0;
    if (std::isfinite(f) && size > kMost) shift = 64;
    if (size < kLeast && size > 0.0) shift = -100;
    *first = std::ldexp(1.f, shift);
    *alpha = static_cast<float>(shift ? std::copysign(std::fmin(std::ldexp(size, -shift), kMost), f) : f);
}

// CTAs that share a single-CTA tile's K: the most of 8, 4 and 2 that keep two CTAs
// an SM, where the stages that it saves outweigh the cluster's start and the sums'
// way through distributed shared memory, which grow with the tile and the clusters
// at work.  Microseconds, FP4_MX:
//   1 x 4096 x 2048:    1: 3.48   2: 3.51   4: 3.24   8: 3.38
//   1 x 4096 x 14336:   1: 14.7   2: 9.7    4: 8.2    8: 7.3
//   64 x 2048 x 8192:   1: 8.6    2: 7.1    4: 5.2    8: 6.2
//   64 x 2048 x 14336:  1: 17.3   2: 11.7   4: 7.9    8: 7.3
//   64 x 1000 x 8192:   1: 8.5    2: 7.1    4: 5.1    8: 4.9     (8 tiles)
//   64 x 1000 x 2048:   1: 4.5    2: 5.1    4: 4.1    8: 4.5     (8 tiles)
//   64 x 8192 x 2048:   1: 5.0    2: 5.7    4: 5.5    8: 11.0    (64 tiles)
//   100 x 14336 x 2048: 1: 7.6    2: 8.0
//   100 x 14336 x 4096: 1: 11.4   2: 10.4
// More than two CTAs an SM is a second turn (1 x 28672 x 4096, 224 tiles: 11.3, and
// 14.0 with two CTAs a tile).
int split_of(int64_t tiles, int64_t k_tiles, int tile, int sms) {
    const bool wide = tile >= 64;
    if (tiles * 8 <= 2 * sms && k_tiles >= (wide && tiles * 16 > sms ? 48 : 32)) return 8;
    if (tiles * 4 <= 2 * sms && k_tiles >= (wide && tiles * 8 > sms ? 16 : 8)) return 4;
    if (tiles * 2 <= 2 * sms && k_tiles >= 16) return 2;
    return 1;
}

// The tile, side and K split of a call; false where the options cannot serve the
// shape (a tile narrower than 128 with more rows than that on that side).
//
// With more than 128 rows on both sides a CTA pair takes 256 x 256, unless 128 x 128
// tiles leave enough SMs free for a split of a long K.  Microseconds, FP4_MX, pairs
// and then 128 x 128 tiles with their best split:
//   512 x 2048 x 1024 5.1, 5.7     512 x 1024 x 2048 6.2, 6.2     256 x 512 x 2048  6.1, 4.9
//   500 x 1529 x 256  5.4, 7.0     500 x 1529 x 2048 7.2, 7.7     500 x 1529 x 4096 9.4, 8.5
//   512 x 2048 x 4096 8.3, 8.3     512 x 2048 x 8192 13.0, 10.2
//   384 x 4096 x 4096 8.5, 9.0     384 x 4096 x 8192 13.5, 12.8   2048 x 4096 x 4096 14.9, 21.4
bool resolve(int64_t M, int64_t N, int64_t K, int sms, gemm_fp4_options *o) {
    const int64_t k_tiles = (K + 255) / 256;
    if (o->tile == 0 && o->swap == 0 && o->cluster_k == 0 && M > 128 && N > 128) {
        const int split = split_of((M + 127) / 128 * ((N + 127) / 128), k_tiles, 128, sms);
        if (split < 4 && (split == 1 || k_tiles < 32)) o->tile = 256;
    }
    if (o->tile == 256) {
        o->cluster_k = 1;
        o->swap = 1;
        return true;
    }
    // the side with more rows, the weights of a few tokens, streams through the tile's
    // 128 rows; the other side's tile is the narrowest MMA that holds it
    if (o->swap == 0) o->swap = M < N ? 2 : 1;
    const int64_t p_rows = o->swap == 2 ? N : M, q_rows = o->swap == 2 ? M : N;
    if (o->tile == 0) o->tile = q_rows <= 16 ? 16 : (q_rows <= 32 ? 32 : (q_rows <= 64 ? 64 : 128));
    if (o->tile < 128 && q_rows > o->tile) return false;
    if (o->cluster_k == 0) {
        o->cluster_k = split_of((p_rows + 127) / 128 * ((q_rows + o->tile - 1) / o->tile), k_tiles, o->tile, sms);
    }
    while (o->cluster_k > k_tiles) o->cluster_k /= 2;
    return true;
}

int zero_fill(void *D, int64_t bytes, cudaStream_t stream) {
    return cudaMemsetAsync(D, 0, static_cast<size_t>(bytes), stream) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int gemm_fp4_nt(const void *A, const void *A_scales, const void *B, const void *B_scales, void *D, int64_t M, int64_t N,
                int64_t K, int32_t format, int32_t d_type, float alpha, void *stream, const gemm_fp4_options *opts) {
    Call c = {A, A_scales, B, B_scales, D, M, N, K, d_type, 1.f, alpha, static_cast<cudaStream_t>(stream), {}};
    int st = check_options(opts, &c.o);
    if (st != GEMM_OK) return st;
    if (M < 0 || N < 0 || K < 0 || (format != FP4_MX && format != FP4_NV) || !type_ok(d_type) ||
        (format == FP4_MX && c.o.exponent != 0)) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (format == FP4_NV) split_factor(std::ldexp(static_cast<double>(alpha), c.o.exponent), &c.first, &c.alpha);
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!D || (K > 0 && (!A || !A_scales || !B || !B_scales))) return GEMM_ERR_INVALID_ARG;
    if (!aligned(A, 16) || !aligned(A_scales, 16) || !aligned(B, 16) || !aligned(B_scales, 16) ||
        !aligned(D, type_size(d_type))) {
        return GEMM_ERR_MISALIGNED;
    }
    const int64_t d_bytes = M * N * type_size(d_type);
    if (K > 0) {
        const int64_t a = fp4_data_bytes(M, K), b = fp4_data_bytes(N, K);
        const int64_t as = fp4_scale_bytes(M, K, format), bs = fp4_scale_bytes(N, K, format);
        if (a < 0 || b < 0 || as < 0 || bs < 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
        if (overlap(D, d_bytes, A, a) || overlap(D, d_bytes, B, b) || overlap(D, d_bytes, A_scales, as) ||
            overlap(D, d_bytes, B_scales, bs)) {
            return GEMM_ERR_INVALID_ARG;
        }
    }
    int sms = 0;
    st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    if (K == 0) return zero_fill(D, d_bytes, c.stream);
    if (!resolve(M, N, K, sms, &c.o)) return GEMM_ERR_INVALID_ARG;
    if (!encoder()) return GEMM_ERR_CUDA;
    return format == FP4_NV ? launch_fp4<true>(c) : launch_fp4<false>(c);
}

int gemm_fp4_nt_describe(int64_t M, int64_t N, int64_t K, int32_t format, const gemm_fp4_options *opts,
                         int32_t sm_count, gemm_fp4_launch_info *out) {
    gemm_fp4_options o;
    const int st = check_options(opts, &o);
    if (st != GEMM_OK) return st;
    if (M < 0 || N < 0 || K < 0 || (format != FP4_MX && format != FP4_NV) || sm_count < 2 || !out) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    *out = gemm_fp4_launch_info{};
    if (M == 0 || N == 0 || K == 0) return GEMM_OK;
    if (!resolve(M, N, K, sm_count, &o)) return GEMM_ERR_INVALID_ARG;
    out->tile = o.tile;
    out->cluster_k = o.cluster_k;
    out->swap = o.swap;
    if (o.tile == 256) {
        const int64_t tiles = (M + 255) / 256 * ((N + 255) / 256);
        int64_t pairs = tiles < sm_count / 2 ? tiles : sm_count / 2;
        if (o.max_clusters > 0 && o.max_clusters < pairs) pairs = o.max_clusters;
        out->ctas = 2 * pairs;
    } else {
        const int64_t p_rows = o.swap == 2 ? N : M, q_rows = o.swap == 2 ? M : N;
        out->ctas = (p_rows + 127) / 128 * ((q_rows + o.tile - 1) / o.tile) * o.cluster_k;
    }
    return GEMM_OK;
}

int gemm_fp4_last_device_status(void *stream, uint64_t *info) {
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
    if (cudaMemcpyFromSymbol(&status, gemm_f16::g_status, sizeof(int)) != cudaSuccess ||
        cudaMemcpyFromSymbol(&where, gemm_f16::g_info, sizeof(where)) != cudaSuccess ||
        cudaMemcpyToSymbol(gemm_f16::g_status, &zero, sizeof(int)) != cudaSuccess ||
        cudaMemcpyToSymbol(gemm_f16::g_info, &zero64, sizeof(zero64)) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_CUDA;
    }
    if (info) *info = where;
    return status;
}

}  // extern "C"
