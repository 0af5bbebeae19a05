// layer_norm.cu -- layer norm and its gradient (see linear_ops.h).
//
// Both are bound by memory: forward reads a row and writes one, its gradient
// reads two and writes one, at 8 and 14 operations an element.  So each
// element is read from memory once: a row is held in registers, 16 bytes a
// load, by one warp to 32 of them, while its sums are formed (the variance
// from the centred values, as E[x^2] - mean^2 loses what an offset of the
// row costs).
#include <cmath>

#include "common.cuh"

namespace linear_ops {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;

// ---------------------------------------------------------------- forward --

struct NormArgs {
    const void *x, *weight, *bias;
    void *y;
    float *mean, *rstd;
    int64_t x_stride, y_stride;
    int32_t rows, cols;
    float eps, inv_cols;
};

// The threads of threadIdx.x hold one row, threadIdx.y counts rows of the CTA:
// thread t holds units t, t + blockDim.x, ... of VEC elements, NV of them.
template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(1024) norm_forward_kernel(const NormArgs a) {
    __shared__ float slots[2][4][32];  // two sums of each row of the CTA (at most 4)
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + (live ? row : 0) * a.x_stride;
    ptx::griddep_wait();

    Pack<T, VEC> raw[NV];
    float v[NV][VEC];
    float sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * VEC;
        if (live && col < a.cols) raw[i] = load_once<T, VEC>(x + col);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * VEC;
        const bool in = live && col < a.cols;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            v[i][j] = in ? to_f32(raw[i].v[j]) : 0.f;
            sum[0] += v[i][j];
        }
    }
    row_sum<1>(sum, slots[0][threadIdx.y]);
    const float mean = sum[0] * a.inv_cols;
    float var[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * VEC;
        if (live && col < a.cols) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i][j] -= mean;
                var[0] += v[i][j] * v[i][j];
            }
        }
    }
    row_sum<1>(var, slots[1][threadIdx.y]);
    const float rstd = 1.f / sqrtf(var[0] * a.inv_cols + a.eps);
    if (!live) return;
    if (threadIdx.x == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    T *y = static_cast<T *>(a.y) + row * a.y_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * VEC;
        if (col < a.cols) {
            float w[VEC], b[VEC], out[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = 1.f, b[j] = 0.f;
            if (a.weight) load_f32<W, VEC>(static_cast<const W *>(a.weight) + col, w);
            if (a.bias) load_f32<W, VEC>(static_cast<const W *>(a.bias) + col, b);
#pragma unroll
            for (int j = 0; j < VEC; ++j) out[j] = v[i][j] * rstd * w[j] + b[j];
            store_f32<T, VEC>(y + col, out);
        }
    }
}

// Rows too long for registers: one CTA of 1024 threads passes over its row
// three times (sum, centred squares, output), the second and third from L2.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_forward_long_kernel(const NormArgs a) {
    __shared__ float slots[2][32];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    T *y = static_cast<T *>(a.y) + row * a.y_stride;
    ptx::griddep_wait();
    float sum[1] = {0.f}, var[1] = {0.f};
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) sum[0] += to_f32(x[c]);
    row_sum<1>(sum, slots[0]);
    const float mean = sum[0] * a.inv_cols;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        var[0] += d * d;
    }
    row_sum<1>(var, slots[1]);
    const float rstd = 1.f / sqrtf(var[0] * a.inv_cols + a.eps);
    if (threadIdx.x == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        const float w = a.weight ? to_f32(static_cast<const W *>(a.weight)[c]) : 1.f;
        const float b = a.bias ? to_f32(static_cast<const W *>(a.bias)[c]) : 0.f;
        y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * w + b);
    }
}

// --------------------------------------------------------------- gradient --

struct GradArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void *dx;
    float *partial;  // [parts][2][cols]: sums over some rows of dy * h, then of dy
    int64_t dy_stride, x_stride, dx_stride;
    int32_t rows, cols;
    float inv_cols;
};

// A persistent grid: each CTA takes rows blockIdx.x * blockDim.y + threadIdx.y,
// then further ones a grid apart, loads the next row while it reduces this one,
// and keeps its columns' sums of dweight and dbias in registers until the end.
// (Where the next row would take more than 16 registers, it is loaded when its
// turn comes: with it the kernel would spill.)  Then the rows of a CTA are added up in shared memory and written as one part.
template <typename T, typename W, int VEC, int NV>
__global__ void __launch_bounds__(512) norm_backward_kernel(const GradArgs a) {
    __shared__ float slots[2][4][64];
    extern __shared__ float fold[];  // [2][cols], where a CTA has several rows
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    constexpr bool kAhead = NV * (VEC == 1 ? 8 : 2 * VEC * static_cast<int>(sizeof(T))) <= 64;
    const int tpr = static_cast<int>(blockDim.x);
    float w[NV][VEC], sw[NV][VEC], sb[NV][VEC];
    Pack<T, VEC> rx[NV], ry[NV];
    ptx::griddep_wait();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[i][j] = 1.f, sw[i][j] = 0.f, sb[i][j] = 0.f;
        if (a.weight && col < a.cols) load_f32<W, VEC>(static_cast<const W *>(a.weight) + col, w[i]);
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t r) {
        if (r >= a.rows) return;
        mean = a.mean[r];
        rstd = a.rstd[r];
        const T *x = static_cast<const T *>(a.x) + r * a.x_stride;
        const T *dy = static_cast<const T *>(a.dy) + r * a.dy_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
            if (col < a.cols) {
                rx[i] = load_once<T, VEC>(x + col);
                ry[i] = load_once<T, VEC>(dy + col);
            }
        }
    };
    if constexpr (kAhead) fetch(row);
    int flip = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.y; first < a.rows; first += step, row += step) {
        if constexpr (!kAhead) fetch(row);
        const bool live = row < a.rows;
        const float m = mean, rs = rstd;
        float h[NV][VEC], g[NV][VEC];
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
            const bool in = live && col < a.cols;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = in ? to_f32(ry[i].v[j]) : 0.f;
                h[i][j] = in ? (to_f32(rx[i].v[j]) - m) * rs : 0.f;
                g[i][j] = d * w[i][j];
                sw[i][j] += d * h[i][j];
                sb[i][j] += d;
                sums[0] += g[i][j];
                sums[1] += g[i][j] * h[i][j];
            }
        }
        if constexpr (kAhead) fetch(row + step);
        row_sum<2>(sums, slots[flip][threadIdx.y]);
        flip ^= 1;
        if (live) {
            const float c1 = sums[0] * a.inv_cols, c2 = sums[1] * a.inv_cols;
            T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
                if (col < a.cols) {
                    float out[VEC];
#pragma unroll
                    for (int j = 0; j < VEC; ++j) out[j] = rs * (g[i][j] - c1 - h[i][j] * c2);
                    store_f32<T, VEC>(dx + col, out);
                }
            }
        }
    }
    if (!a.partial) return;
    // the other rows' sums join those of the CTA's first row, one row after the other
    for (int r = 1; r < static_cast<int>(blockDim.y); ++r) {
        __syncthreads();
        if (static_cast<int>(threadIdx.y) == r) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
                if (col < a.cols) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) fold[col + j] = sw[i][j], fold[a.cols + col + j] = sb[i][j];
                }
            }
        }
        __syncthreads();
        if (threadIdx.y == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
                if (col < a.cols) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) sw[i][j] += fold[col + j], sb[i][j] += fold[a.cols + col + j];
                }
            }
        }
    }
    if (threadIdx.y == 0) {
        float *part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int col = (i * tpr + static_cast<int>(threadIdx.x)) * VEC;
            if (col < a.cols) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    part[col + j] = sw[i][j];
                    part[a.cols + col + j] = sb[i][j];
                }
            }
        }
    }
}

// Rows too long for registers: dx by one CTA per row in two passes, ...
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const GradArgs a) {
    __shared__ float slot[64];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
    ptx::griddep_wait();
    const float m = a.mean[row], rs = a.rstd[row];
    float sums[2] = {0.f, 0.f};
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        const float g = to_f32(dy[c]) * (a.weight ? to_f32(static_cast<const W *>(a.weight)[c]) : 1.f);
        sums[0] += g;
        sums[1] += g * ((to_f32(x[c]) - m) * rs);
    }
    row_sum<2>(sums, slot);
    const float c1 = sums[0] * a.inv_cols, c2 = sums[1] * a.inv_cols;
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        const float g = to_f32(dy[c]) * (a.weight ? to_f32(static_cast<const W *>(a.weight)[c]) : 1.f);
        dx[c] = from_f32<T>(rs * (g - c1 - (to_f32(x[c]) - m) * rs * c2));
    }
}

// ... and the weights' partial sums by columns: blockIdx.y takes every
// gridDim.y-th row.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const GradArgs a) {
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (col >= a.cols) return;
    float sw = 0.f, sb = 0.f;
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const float d = to_f32(static_cast<const T *>(a.dy)[r * a.dy_stride + col]);
        sw += d * ((to_f32(static_cast<const T *>(a.x)[r * a.x_stride + col]) - a.mean[r]) * a.rstd[r]);
        sb += d;
    }
    float *part = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * a.cols;
    part[col] = sw;
    part[a.cols + col] = sb;
}

// dweight (blockIdx.y 0) or dbias (1) of 32 columns: thread row y adds every
// 32nd part, then the 32 thread rows are added in order.
template <typename W>
__global__ void __launch_bounds__(1024) norm_join_kernel(const float *partial, int parts, int cols, W *dweight,
                                                         W *dbias) {
    __shared__ float s[32][33];
    ptx::griddep_wait();
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float sum = 0.f;
    if (col < cols) {
        const float *p = partial + static_cast<int64_t>(blockIdx.y) * cols + col;
#pragma unroll 4
        for (int i = threadIdx.y; i < parts; i += 32) sum += p[static_cast<int64_t>(i) * 2 * cols];
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    float t = s[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out < cols) (blockIdx.y ? dbias : dweight)[out] = from_f32<W>(t);
}

// ------------------------------------------------------------------- host --

// The shape of a CTA: threads per row (a power of two, whole warps) and rows.
struct RowShape {
    int nv = 0;  // units per thread; 0: the row does not fit
    int threads = 0, rows = 0;
};

// Few units a thread while that leaves the row at least a warp and at most
// `most` threads; short rows share a CTA of 128 threads.
RowShape row_shape(int64_t cols, int vec, const int *nvs, int count, int most) {
    const int64_t units = (cols + vec - 1) / vec;
    RowShape s;
    for (int i = 0; i < count; ++i) {
        int t = 32;
        while (t < most && static_cast<int64_t>(t) * nvs[i] < units) t *= 2;
        if (static_cast<int64_t>(t) * nvs[i] < units) continue;
        s.nv = nvs[i];
        s.threads = t;
        s.rows = t < 128 ? 128 / t : 1;
        // longer threads only for rows that would need more than 512 of them
        if (t <= 512 || i + 1 == count) break;
    }
    return s;
}

template <typename T, typename W, int VEC>
int forward_vec(const NormArgs &a, cudaStream_t stream) {
    static constexpr int kVec[3] = {1, 2, 4}, kOne[3] = {4, 8, 16};
    const RowShape s = row_shape(a.cols, VEC, VEC > 1 ? kVec : kOne, 3, 1024);
    const dim3 block(s.threads, s.rows);
    if (s.nv == 0) {
        return launch(norm_forward_long_kernel<T, W>, dim3(a.rows), dim3(1024), 0, stream, a);
    }
    const dim3 grid((a.rows + s.rows - 1) / s.rows);
    constexpr int k0 = VEC > 1 ? 1 : 4;
    if (s.nv == k0) return launch(norm_forward_kernel<T, W, VEC, k0>, grid, block, 0, stream, a);
    if (s.nv == 2 * k0) return launch(norm_forward_kernel<T, W, VEC, 2 * k0>, grid, block, 0, stream, a);
    return launch(norm_forward_kernel<T, W, VEC, 4 * k0>, grid, block, 0, stream, a);
}

template <typename T, typename W>
int forward_as(const NormArgs &a, cudaStream_t stream) {
    constexpr int U = kUnit<T>;
    const bool wide = a.cols % U == 0 && a.x_stride % U == 0 && a.y_stride % U == 0 && aligned(a.x, 16) &&
                      aligned(a.y, 16) && (!a.weight || aligned(a.weight, 16)) && (!a.bias || aligned(a.bias, 16));
    return wide ? forward_vec<T, W, U>(a, stream) : forward_vec<T, W, 1>(a, stream);
}

// Parts of the weights' gradient: at most two CTAs for each of 152 SMs.
constexpr int kMaxParts = 304;

int backward_parts(int64_t rows) { return static_cast<int>(rows < kMaxParts ? rows : kMaxParts); }

template <typename T, typename W, int VEC>
int backward_vec(const GradArgs &a, W *dweight, W *dbias, cudaStream_t stream) {
    static constexpr int kVec16[2] = {1, 2}, kVec32[2] = {2, 4}, kOne[2] = {8, 16};
    constexpr int k0 = VEC == 1 ? 8 : (VEC == 4 ? 2 : 1);
    const RowShape s = row_shape(a.cols, VEC, VEC == 1 ? kOne : (VEC == 4 ? kVec32 : kVec16), 2, 512);
    int parts = 0;
    int st = GEMM_OK;
    if (a.rows > 0 && s.nv != 0) {
        const dim3 block(s.threads, s.rows);
        const int64_t groups = (static_cast<int64_t>(a.rows) + s.rows - 1) / s.rows;
        parts = backward_parts(groups);
        const size_t smem = s.rows > 1 ? 2 * sizeof(float) * a.cols : 0;
        st = s.nv == k0 ? launch(norm_backward_kernel<T, W, VEC, k0>, dim3(parts), block, smem, stream, a)
                        : launch(norm_backward_kernel<T, W, VEC, 2 * k0>, dim3(parts), block, smem, stream, a);
    } else if (a.rows > 0) {
        st = launch(norm_backward_long_kernel<T, W>, dim3(a.rows), dim3(1024), 0, stream, a);
        if (st == GEMM_OK && dweight) {
            parts = backward_parts(a.rows);
            st = launch(norm_columns_kernel<T>, dim3((a.cols + 255) / 256, parts), dim3(256), 0, stream, a);
        }
    }
    if (st != GEMM_OK || !dweight) return st;
    return launch(norm_join_kernel<W>, dim3((a.cols + 31) / 32, 2), dim3(32, 32), 0, stream, a.partial, parts, a.cols,
                  dweight, dbias);
}

template <typename T, typename W>
int backward_as(const GradArgs &a, void *dweight, void *dbias, cudaStream_t stream) {
    constexpr int U = kUnit<T>;
    const bool wide = a.cols % U == 0 && a.x_stride % U == 0 && a.dy_stride % U == 0 && a.dx_stride % U == 0 &&
                      aligned(a.x, 16) && aligned(a.dy, 16) && aligned(a.dx, 16) &&
                      (!a.weight || aligned(a.weight, 16));
    W *dw = static_cast<W *>(dweight), *db = static_cast<W *>(dbias);
    return wide ? backward_vec<T, W, U>(a, dw, db, stream) : backward_vec<T, W, 1>(a, dw, db, stream);
}

// The element type and the weights' as template arguments.
#define LINEAR_BY_TYPE(type, weight_type, FN, ...)                                                              \
    ((type) == LINEAR_F32 ? FN<float, float>(__VA_ARGS__)                                                       \
     : (type) == LINEAR_F16                                                                                     \
         ? ((weight_type) == LINEAR_F32 ? FN<__half, float>(__VA_ARGS__) : FN<__half, __half>(__VA_ARGS__))     \
         : ((weight_type) == LINEAR_F32 ? FN<__nv_bfloat16, float>(__VA_ARGS__)                                 \
                                        : FN<__nv_bfloat16, __nv_bfloat16>(__VA_ARGS__)))

bool sizes_ok(int64_t rows, int64_t cols) { return rows >= 0 && cols >= 1; }

}  // namespace

int gb300_sms(int *sms) {
    static thread_local int last_dev = -1, last_sms = 0;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_NO_DEVICE;
    }
    if (dev != last_dev) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return GEMM_ERR_NO_DEVICE;
        }
        if (major != 10 || minor != 3) return GEMM_ERR_ARCH;
        last_dev = dev;
        last_sms = n;
    }
    *sms = last_sms;
    return GEMM_OK;
}

}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int layer_norm_forward(const void *x, int64_t x_stride, const void *weight, const void *bias, void *y, int64_t y_stride,
                       float *mean, float *rstd, int64_t rows, int64_t cols, float eps, int32_t type,
                       int32_t weight_type, void *stream) {
    if (!sizes_ok(rows, cols) || !type_ok(type) || (weight_type != type && weight_type != LINEAR_F32) ||
        !(eps >= 0.f) || std::isinf(eps) || x_stride < 0 || !mean != !rstd) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return GEMM_OK;
    if (!x || !y || (rows > 1 && y_stride < cols)) return GEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), wsize = type_size(weight_type);
    if (!aligned(x, size) || !aligned(y, size) || !aligned(weight, wsize) || !aligned(bias, wsize) || !aligned(mean, 4) ||
        !aligned(rstd, 4)) {
        return GEMM_ERR_MISALIGNED;
    }
    if (rows == 1) x_stride = y_stride = 0;
    const int64_t y_bytes = span_bytes(rows, cols, y_stride, size);
    if (overlap(y, y_bytes, x, span_bytes(rows, cols, x_stride, size)) || overlap(y, y_bytes, weight, cols * wsize) ||
        overlap(y, y_bytes, bias, cols * wsize) || overlap(y, y_bytes, mean, rows * 4) ||
        overlap(y, y_bytes, rstd, rows * 4)) {
        return GEMM_ERR_INVALID_ARG;
    }
    int sms = 0;
    const int st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    const NormArgs a = {x,    weight,   bias,     y,   mean, rstd, x_stride, y_stride, static_cast<int32_t>(rows),
                        static_cast<int32_t>(cols), eps, 1.f / static_cast<float>(cols)};
    return LINEAR_BY_TYPE(type, weight_type, forward_as, a, static_cast<cudaStream_t>(stream));
}

int64_t layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (!sizes_ok(rows, cols)) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return static_cast<int64_t>(backward_parts(rows)) * 2 * cols * 4;
}

int layer_norm_backward(const void *dy, int64_t dy_stride, const void *x, int64_t x_stride, const void *weight,
                        const float *mean, const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias,
                        int64_t rows, int64_t cols, int32_t type, int32_t weight_type, void *workspace,
                        int64_t workspace_bytes, void *stream) {
    if (!sizes_ok(rows, cols) || !type_ok(type) || (weight_type != type && weight_type != LINEAR_F32) ||
        dy_stride < 0 || x_stride < 0 || !dweight != !dbias || workspace_bytes < 0) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx || (rows > 1 && dx_stride < cols))) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 && !dweight) return GEMM_OK;
    const int64_t need = dweight ? layer_norm_backward_workspace_size(rows, cols) : 0;
    if (need > 0 && !workspace) return GEMM_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH_LIMIT;
    const int64_t size = type_size(type), wsize = type_size(weight_type);
    if (!aligned(dy, size) || !aligned(x, size) || !aligned(dx, size) || !aligned(weight, wsize) ||
        !aligned(dweight, wsize) || !aligned(dbias, wsize) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        (need > 0 && !aligned(workspace, 16))) {
        return GEMM_ERR_MISALIGNED;
    }
    if (rows <= 1) dy_stride = x_stride = dx_stride = 0;
    const struct {
        const void *p;
        int64_t bytes;
    } outs[4] = {{dx, span_bytes(rows, cols, dx_stride, size)}, {dweight, cols * wsize}, {dbias, cols * wsize},
                 {workspace, need}},
      ins[5] = {{dy, span_bytes(rows, cols, dy_stride, size)}, {x, span_bytes(rows, cols, x_stride, size)},
                {weight, cols * wsize}, {mean, rows * 4}, {rstd, rows * 4}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 5; ++j) {
            if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return GEMM_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j) {
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return GEMM_ERR_INVALID_ARG;
        }
    }
    int sms = 0;
    const int st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    const GradArgs a = {dy, x, weight, mean, rstd, dx, dweight ? static_cast<float *>(workspace) : nullptr,
                        dy_stride, x_stride, dx_stride, static_cast<int32_t>(rows), static_cast<int32_t>(cols),
                        1.f / static_cast<float>(cols)};
    return LINEAR_BY_TYPE(type, weight_type, backward_as, a, dweight, dbias, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
