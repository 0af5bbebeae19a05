// norm_forward.cu -- layer norm (see linear_ops.h and norm_rows.cuh).
#include <cmath>

#include "norm_rows.cuh"

namespace linear_ops {
namespace {

struct NormArgs {
    const void *x, *weight, *bias;
    void *y;
    float *mean, *rstd;
    int64_t x_stride, y_stride;
    int32_t rows, cols;
    float eps, inv_cols;
};

// Of the ring.  8192 x 4096 bf16: two 23.3 us, three 21.9, four 22.1; 20000 x 256
// fp16: 9.2, 6.3, 6.3; 8192 x 1024 fp16: 7.7, 7.4, 8.1.
constexpr int kStages = 3;

// Rows of a CTA: 128 threads' worth; CTAs of an SM: 512 threads (32 elements, their
// weights and biases take 100 registers) and what their rings leave room for.
//
// 8192 x 4096 bf16: 21.9 us, 6.1 TB/s, 90 % of the copy rate; 8192 x 8192 fp32 86.8
// (91 %); 2048 x 16384 fp16 24.4 (81 %).  Rows that start anywhere, 1023 x 5003 fp32:
// 10.9 us (55 %; the first rows' latency, 7 rows an SM); 8192 x 1021 fp16 10.3, element
// by element (8192 x 1024: 7.4).  One row
// of 4096: 1.9 us, a launch and one trip to memory.
template <typename T, int E, bool WIDE, int TPR>
struct NormShape {
    static constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;
    static constexpr int BYTES = ROWS * RowRing<T, E, WIDE, TPR, 1, kStages>::BYTES;
    static constexpr int BY_SMEM = 220 * 1024 / (BYTES + 2048), BY_THREADS = 512 / (ROWS * TPR);
    static constexpr int PER_SM = BY_SMEM < BY_THREADS ? BY_SMEM : BY_THREADS;
};

template <typename T, typename W, int E, bool WIDE, int TPR>
__global__ void __launch_bounds__(TPR *NormShape<T, E, WIDE, TPR>::ROWS, NormShape<T, E, WIDE, TPR>::PER_SM)
    norm_forward_ring_kernel(const NormArgs a) {
    constexpr int ROWS = NormShape<T, E, WIDE, TPR>::ROWS;
    using Ring = RowRing<T, E, WIDE, TPR, 1, kStages>;
    __shared__ __align__(16) float slots[2][ROWS][32];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    Ring ring(ring_mem, a.cols);
    int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.y;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;  // of this row
    T *y = static_cast<T *>(a.y) + row * a.y_stride;
    const int64_t x_step = step * a.x_stride, y_step = step * a.y_stride;
    ptx::griddep_wait();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        if (row + s * step < a.rows) ring.copy(s, 0, x + s * x_step);
        cp_async_commit();
    }
    float2 w[E / 2], b[E / 2];
    ring.gather(static_cast<const W *>(a.weight), 1.f, w);
    ring.gather(static_cast<const W *>(a.bias), 0.f, b);
    for (; row < a.rows; row += step, x += x_step, y += y_step) {
        cp_async_wait<kStages - 2>();
        if constexpr (!WIDE) row_barrier<TPR, ROWS>();
        float2 v[E / 2];
        ring.read(0, x, v);
        if (row + (kStages - 1) * step < a.rows) ring.copy(ring.slot_behind(), 0, x + (kStages - 1) * x_step);
        cp_async_commit();
        ring.next();
        float2 s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) s2 = add2(s2, v[i]);
        float sum[1] = {s2.x + s2.y};
        row_sum<1, TPR, ROWS>(sum, slots[0][threadIdx.y]);
        const float mean = sum[0] * a.inv_cols;
        s2 = both(0.f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            v[i] = add2(v[i], both(-mean));
            // elements past the row's end are no deviations
            if constexpr (WIDE) {
                if (ring.holds(2 * i)) s2 = fma2(v[i], v[i], s2);
            } else {
                if (ring.holds(2 * i)) s2.x += v[i].x * v[i].x;
                if (ring.holds(2 * i + 1)) s2.y += v[i].y * v[i].y;
            }
        }
        float var[1] = {s2.x + s2.y};
        row_sum<1, TPR, ROWS>(var, slots[1][threadIdx.y]);
        const float rstd = 1.f / sqrtf(var[0] * a.inv_cols + a.eps);
        if (threadIdx.x == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
#pragma unroll
        for (int i = 0; i < E / 2; ++i) v[i] = fma2(mul2(v[i], both(rstd)), w[i], b[i]);
        ring.scatter(y, v);
    }
}

// Rows past the ring's, of 16-bit elements in whole units, up to 32768 columns: a CTA
// of 256 threads a row, which holds it as it came from memory (pairs take half the
// registers of fp32 values).  2048 x 32768: 75.6 us; 2048 x 32776, by the next kernel,
// 115.5.
constexpr int kHeldUnits = 16;  // of a thread

template <typename T, typename W>
__global__ void __launch_bounds__(256) norm_forward_held_kernel(const NormArgs a) {
    constexpr int NV = kHeldUnits, U = kUnit<T>, step = 256 * U, P = Pair<T>::WORDS;
    __shared__ __align__(16) float slots[2][32];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const int first = static_cast<int>(threadIdx.x) * U;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride + first;
    ptx::griddep_wait();
    uint32_t raw[NV][4];
    float2 s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (first + i * step < a.cols) u = load_unit(x + i * step);
        raw[i][0] = u.x, raw[i][1] = u.y, raw[i][2] = u.z, raw[i][3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < U / 2; ++j) s2 = add2(s2, Pair<T>::widen(&raw[i][j * P]));
    }
    float sum[1] = {s2.x + s2.y};
    row_sum<1, 256, 1>(sum, slots[0]);
    const float mean = sum[0] * a.inv_cols;
    s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (first + i * step < a.cols) {
#pragma unroll
            for (int j = 0; j < U / 2; ++j) {
                const float2 d = add2(Pair<T>::widen(&raw[i][j * P]), both(-mean));
                s2 = fma2(d, d, s2);
            }
        }
    }
    float var[1] = {s2.x + s2.y};
    row_sum<1, 256, 1>(var, slots[1]);
    const float rstd = 1.f / sqrtf(var[0] * a.inv_cols + a.eps);
    if (threadIdx.x == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    T *y = static_cast<T *>(a.y) + row * a.y_stride + first;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (first + i * step < a.cols) {
            float2 w[U / 2], b[U / 2], out[U / 2];
#pragma unroll
            for (int j = 0; j < U / 2; ++j) w[j] = both(1.f), b[j] = both(0.f);
            if (a.weight) load_pairs<W, U / 2>(static_cast<const W *>(a.weight) + first + i * step, w);
            if (a.bias) load_pairs<W, U / 2>(static_cast<const W *>(a.bias) + first + i * step, b);
#pragma unroll
            for (int j = 0; j < U / 2; ++j) {
                out[j] = fma2(mul2(add2(Pair<T>::widen(&raw[i][j * P]), both(-mean)), both(rstd)), w[j], b[j]);
            }
            store_pairs<T, U / 2>(y + i * step, out);
        }
    }
}

// Rows too long for registers: one CTA of 1024 threads passes over its row three
// times (sum, centred squares, output), the second and third from L2.  2048 x 20480
// fp32: 96.6 us, 3.5 TB/s.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_forward_long_kernel(const NormArgs a) {
    __shared__ __align__(16) float slots[2][32];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    T *y = static_cast<T *>(a.y) + row * a.y_stride;
    ptx::griddep_wait();
    float sum[1] = {0.f}, var[1] = {0.f};
#pragma unroll 8
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) sum[0] += to_f32(x[c]);
    row_sum<1, 1024, 1>(sum, slots[0]);
    const float mean = sum[0] * a.inv_cols;
#pragma unroll 8
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        const float d = to_f32(x[c]) - mean;
        var[0] += d * d;
    }
    row_sum<1, 1024, 1>(var, slots[1]);
    const float rstd = 1.f / sqrtf(var[0] * a.inv_cols + a.eps);
    if (threadIdx.x == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        const float w = a.weight ? to_f32(static_cast<const W *>(a.weight)[c]) : 1.f;
        const float b = a.bias ? to_f32(static_cast<const W *>(a.bias)[c]) : 0.f;
        y[c] = from_f32<T>((to_f32(x[c]) - mean) * rstd * w + b);
    }
}

// ------------------------------------------------------------------- host --

template <typename T, typename W, int E, bool WIDE, int TPR>
int forward_ring(const NormArgs &a, int sms, cudaStream_t stream) {
    using S = NormShape<T, E, WIDE, TPR>;
    auto *kernel = norm_forward_ring_kernel<T, W, E, WIDE, TPR>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, S::BYTES, done)) return GEMM_ERR_CUDA;
    return launch(kernel, dim3(grid_of(a.rows, S::ROWS, S::PER_SM * sms)), dim3(TPR, S::ROWS), S::BYTES, stream, a);
}

template <typename T, typename W, bool WIDE>
int forward_rows(const NormArgs &a, int sms, cudaStream_t stream) {
#define LINEAR_CASE(E, TPR) return forward_ring<T, W, E, WIDE, TPR>(a, sms, stream)
    LINEAR_ROW_SHAPES(LINEAR_CASE)
#undef LINEAR_CASE
    if constexpr (WIDE && sizeof(T) == 2) {
        if (a.cols <= 256 * kHeldUnits * kUnit<T>) {
            return launch(norm_forward_held_kernel<T, W>, dim3(a.rows), dim3(256), 0, stream, a);
        }
    }
    return launch(norm_forward_long_kernel<T, W>, dim3(a.rows), dim3(1024), 0, stream, a);
}

template <typename T, typename W>
int forward_as(const NormArgs &a, int sms, cudaStream_t stream) {
    constexpr int U = kUnit<T>;
    const bool wide = a.cols % U == 0 && a.x_stride % U == 0 && a.y_stride % U == 0 && aligned(a.x, 16) &&
                      aligned(a.y, 16) && (!a.weight || aligned(a.weight, 16)) && (!a.bias || aligned(a.bias, 16));
    return wide ? forward_rows<T, W, true>(a, sms, stream) : forward_rows<T, W, false>(a, sms, stream);
}

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
    const struct {
        const void *p;
        int64_t bytes;
    } outs[3] = {{y, span_bytes(rows, cols, y_stride, size)}, {mean, rows * 4}, {rstd, rows * 4}},
      ins[3] = {{x, span_bytes(rows, cols, x_stride, size)}, {weight, cols * wsize}, {bias, cols * wsize}};
    if (rows_overlap(y, x, rows, cols * size, y_stride * size, x_stride * size)) return GEMM_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i) {
        for (int j = i == 0 ? 1 : 0; j < 3; ++j) {  // y and x above
            if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return GEMM_ERR_INVALID_ARG;
        }
        for (int j = 0; j < i; ++j) {
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return GEMM_ERR_INVALID_ARG;
        }
    }
    int sms = 0;
    const int st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    const NormArgs a = {x,    weight,   bias,     y,   mean, rstd, x_stride, y_stride, static_cast<int32_t>(rows),
                        static_cast<int32_t>(cols), eps, 1.f / static_cast<float>(cols)};
    return LINEAR_BY_TYPE(type, weight_type, forward_as, a, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
