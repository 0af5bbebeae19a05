// norm_backward.cu -- the gradient of layer norm (see linear_ops.h and
// norm_rows.cuh).
#include "norm_rows.cuh"

namespace linear_ops {
namespace {

// Floats from a fold's dweight to its dbias: whole units.
__host__ __device__ constexpr int fold_stride(int cols) { return (cols + 3) / 4 * 4; }

struct GradArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void *dx;
    float *partial;  // [parts][2][cols]: sums over some rows of dy * h, then of dy
    int64_t dy_stride, x_stride, dx_stride;
    int32_t rows, cols;
    float inv_cols;
};

// Stages of the ring; fp32 rows are larger, and three let two CTAs of 4096 columns
// share an SM.
template <typename T>
constexpr int kStages = sizeof(T) == 4 ? 3 : 4;

// A persistent grid: each CTA takes ROWS rows, then further ones a grid apart, and
// keeps its columns' sums of dweight and dbias in registers until the end.  Then
// the sums of its other rows join those of its first one, one row after the other
// through shared memory, and go out as one part.
template <typename T, typename W, int E, bool WIDE, int TPR, int THREADS, int PER_SM>
__global__ void __launch_bounds__(THREADS, PER_SM) norm_backward_ring_kernel(const GradArgs a) {
    constexpr int ROWS = THREADS / TPR, STAGES = kStages<T>;
    using Ring = RowRing<T, E, WIDE, TPR, 2, STAGES>;
    __shared__ __align__(16) float slots[2][ROWS][64];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    Ring ring(ring_mem, a.cols);
    int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.y;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride, *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
    const int64_t x_step = step * a.x_stride, dy_step = step * a.dy_stride, dx_step = step * a.dx_stride;
    ptx::griddep_wait();
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (row + s * step < a.rows) {
            ring.copy(s, 0, x + s * x_step);
            ring.copy(s, 1, dy + s * dy_step);
        }
        cp_async_commit();
    }
    float mean = 0.f, rstd = 0.f;
    if (row < a.rows) mean = a.mean[row], rstd = a.rstd[row];
    float2 w[E / 2], sw[E / 2], sb[E / 2];
    ring.gather(static_cast<const W *>(a.weight), 1.f, w);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) sw[i] = sb[i] = both(0.f);
    int flip = 0;
    for (; row < a.rows; row += step, x += x_step, dy += dy_step, dx += dx_step) {
        cp_async_wait<STAGES - 2>();
        if constexpr (!WIDE) row_barrier<TPR, ROWS>();
        const float2 m = both(-mean), rs = both(rstd);
        float2 h[E / 2], g[E / 2];
        ring.read(0, x, h);
        ring.read(1, dy, g);
        if (row + (STAGES - 1) * step < a.rows) {
            ring.copy(ring.slot_behind(), 0, x + (STAGES - 1) * x_step);
            ring.copy(ring.slot_behind(), 1, dy + (STAGES - 1) * dy_step);
        }
        cp_async_commit();
        ring.next();
        if (row + step < a.rows) mean = a.mean[row + step], rstd = a.rstd[row + step];
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            // past the row's end dy is 0, and so is what h there is multiplied with
            h[i] = mul2(add2(h[i], m), rs);
            sw[i] = fma2(g[i], h[i], sw[i]);
            sb[i] = add2(sb[i], g[i]);
            g[i] = mul2(g[i], w[i]);
            s0 = add2(s0, g[i]);
            s1 = fma2(g[i], h[i], s1);
        }
        float sums[2] = {s0.x + s0.y, s1.x + s1.y};
        row_sum<2, TPR, ROWS>(sums, slots[flip][threadIdx.y]);
        flip ^= 1;
        const float2 c1 = both(-sums[0] * a.inv_cols), c2 = both(-sums[1] * a.inv_cols);
#pragma unroll
        for (int i = 0; i < E / 2; ++i) g[i] = mul2(fma2(h[i], c2, add2(g[i], c1)), rs);
        ring.scatter(dx, g);
    }
    if (!a.partial) return;
    cp_async_wait<0>();
    float *fold = reinterpret_cast<float *>(ring_mem), *fold_b = fold + fold_stride(a.cols);  // the ring's memory
    for (int r = 1; r < ROWS; ++r) {
        __syncthreads();
        if (static_cast<int>(threadIdx.y) == r) {
            ring.scatter(fold, sw);
            ring.scatter(fold_b, sb);
        }
        __syncthreads();
        if (threadIdx.y == 0) {
            float2 o[E / 2];
            ring.gather(static_cast<const float *>(fold), 0.f, o);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) sw[i] = add2(sw[i], o[i]);
            ring.gather(static_cast<const float *>(fold_b), 0.f, o);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) sb[i] = add2(sb[i], o[i]);
        }
    }
    if (threadIdx.y != 0) return;
    float *part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * a.cols;
    ring.scatter(part, sw);
    ring.scatter(part + a.cols, sb);
}

// Rows too long for registers: dx by one CTA per row in two passes, ...
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const GradArgs a) {
    __shared__ __align__(16) float slot[64];
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
    row_sum<2, 1024, 1>(sums, slot);
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

// Parts of the weights' gradient: at most two CTAs for each of 152 SMs.
constexpr int kMaxParts = 304;

template <typename T, typename W, int E, bool WIDE, int TPR, int THREADS, int PER_SM>
int backward_ring(const GradArgs &a, int sms, int *parts, cudaStream_t stream) {
    constexpr int ROWS = THREADS / TPR;
    auto *kernel = norm_backward_ring_kernel<T, W, E, WIDE, TPR, THREADS, PER_SM>;
    constexpr int kBytes = ROWS * RowRing<T, E, WIDE, TPR, 2, kStages<T>>::BYTES;
    static_assert(kBytes >= 2 * 4 * TPR * E || ROWS == 1, "the ring's memory holds two rows of sums");
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, kBytes, done)) return GEMM_ERR_CUDA;
    *parts = grid_of(a.rows, ROWS, PER_SM * sms < kMaxParts ? PER_SM * sms : kMaxParts);
    return launch(kernel, dim3(*parts), dim3(TPR, ROWS), kBytes, stream, a);
}

template <typename T, typename W, bool WIDE>
int backward_rows(const GradArgs &a, int sms, int *parts, cudaStream_t stream) {
    if (a.cols <= 32 * 8) return backward_ring<T, W, 8, WIDE, 32, 256, 2>(a, sms, parts, stream);
    if (a.cols <= 32 * 16) return backward_ring<T, W, 16, WIDE, 32, 256, 2>(a, sms, parts, stream);
    if (a.cols <= 64 * 16) return backward_ring<T, W, 16, WIDE, 64, 256, 2>(a, sms, parts, stream);
    if (a.cols <= 128 * 16) return backward_ring<T, W, 16, WIDE, 128, 256, 2>(a, sms, parts, stream);
    if (a.cols <= 256 * 16) return backward_ring<T, W, 16, WIDE, 256, 256, 2>(a, sms, parts, stream);
    if (a.cols <= kRingCols) return backward_ring<T, W, 16, WIDE, 512, 512, 1>(a, sms, parts, stream);
    int st = launch(norm_backward_long_kernel<T, W>, dim3(a.rows), dim3(1024), 0, stream, a);
    if (st == GEMM_OK && a.partial) {
        *parts = grid_of(a.rows, 1, kMaxParts);
        st = launch(norm_columns_kernel<T>, dim3((a.cols + 255) / 256, *parts), dim3(256), 0, stream, a);
    }
    return st;
}

template <typename T, typename W>
int backward_as(const GradArgs &a, void *dweight, void *dbias, int sms, cudaStream_t stream) {
    constexpr int U = kUnit<T>;
    const bool wide = a.cols % U == 0 && a.x_stride % U == 0 && a.dy_stride % U == 0 && a.dx_stride % U == 0 &&
                      aligned(a.x, 16) && aligned(a.dy, 16) && aligned(a.dx, 16) &&
                      (!a.weight || aligned(a.weight, 16));
    int parts = 0;
    if (a.rows > 0) {
        const int st = wide ? backward_rows<T, W, true>(a, sms, &parts, stream)
                            : backward_rows<T, W, false>(a, sms, &parts, stream);
        if (st != GEMM_OK || !dweight) return st;
    }
    return launch(norm_join_kernel<W>, dim3((a.cols + 31) / 32, 2), dim3(32, 32), 0, stream, a.partial, parts, a.cols,
                  static_cast<W *>(dweight), static_cast<W *>(dbias));
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int64_t layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (!sizes_ok(rows, cols)) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return (rows < kMaxParts ? rows : kMaxParts) * 2 * cols * 4;
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
    return LINEAR_BY_TYPE(type, weight_type, backward_as, a, dweight, dbias, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
