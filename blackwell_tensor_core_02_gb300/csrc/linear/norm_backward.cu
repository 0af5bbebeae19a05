// norm_backward.cu -- the gradient of layer norm (see linear_ops.h and
// norm_rows.cuh).
#include "norm_rows.cuh"

namespace linear_ops {
namespace {

// Parts of the weights' gradient: a CTA for each of 152 SMs.
constexpr int kMaxParts = 152;

// Floats of a part's dweight, and of its dbias: whole 16-byte units.
__host__ __device__ constexpr int64_t part_stride(int64_t cols) { return (cols + 3) / 4 * 4; }

struct GradArgs {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    void *dx;
    float *partial;  // [parts][2][part_stride(cols)]: sums over some rows of dy * h, then of dy
    int64_t dy_stride, x_stride, dx_stride;
    int32_t rows, cols;
    float inv_cols;
};

// A persistent grid, one CTA an SM: each of its rows of threads takes a row, then
// further ones a grid apart, and keeps its columns' sums of dweight and dbias in
// registers until the end, when the CTA's are added up in shared memory and go
// out as one part.
//
// A row is read from the ring twice, once for its sums and once for dx: holding
// h and g in between takes 64 registers more a thread, which halves the rows at
// work on an SM, and a row's time is the latency of its sums.  8192 x 4096 bf16
// (the memory takes 29.6 us at the copy rate): 36.2 us, with them held 40.1; 32.1
// without the weights' gradient, the rest is the parts' way to the join.  4096 x
// 8192 fp16 41.9 us (parts twice as long), 4096 x 4096 fp32 34.7.  Of rows past 8192
// columns one is at work on an SM: 2048 x 12288 bf16 33.4 us, and past 12288 of 16
// bits the weights are read again with each row and the ring has two stages: 2048 x
// 16384 50.2.  Whole rows in a second pass over memory (norm_backward_long_kernel)
// took 84 and 93; fp32 rows past 12288 still do, their ring has no room.
// The second pass of a row behind the first pass of the next, with one barrier a
// row, gained nothing (8192 x 4096 36.9, 4096 x 8192 42.0, 8192 x 1024 16.4; 14.0 as
// it is).
template <typename T, int E, bool WIDE, int TPR>
struct GradShape {
    static constexpr int BUDGET = 200 * 1024;
    static constexpr int ROW = RowRing<T, E, WIDE, TPR, 2, 1>::BYTES;  // of dy and x
    static constexpr bool HELD = TPR <= 384;  // the weights, in registers
    // Two stages or three: 8192 x 512 fp16 8.8 and 9.4 us, 8192 x 1024 14.0 and 14.7, but
    // 4096 x 8192 42.6 and 41.9, and rows that start anywhere, 8192 x 1021, 20.7 and 18.4.
    static constexpr int STAGES = (WIDE && TPR <= 64) || !HELD || 3 * ROW > BUDGET ? 2 : 3;
    static constexpr int ROW_BYTES = STAGES * ROW;
    static constexpr int BY_SMEM = BUDGET / ROW_BYTES, BY_THREADS = E <= 16 ? 512 / TPR : (TPR < 384 ? 384 / TPR : 1);
    static constexpr int ROWS = BY_SMEM < BY_THREADS ? BY_SMEM : BY_THREADS;  // at most; 0: no room for a row
    static_assert(ROWS < 2 || ROW_BYTES >= 2 * 4 * TPR * E, "a row's ring holds its sums");
};

template <typename T, typename W, int E, bool WIDE, int TPR>
__global__ void __launch_bounds__(TPR *GradShape<T, E, WIDE, TPR>::ROWS, 1)
    norm_backward_ring_kernel(const GradArgs a) {
    constexpr int ROWS = GradShape<T, E, WIDE, TPR>::ROWS, STAGES = GradShape<T, E, WIDE, TPR>::STAGES;
    using Ring = RowRing<T, E, WIDE, TPR, 2, STAGES>;
    constexpr int U = Ring::U;
    __shared__ __align__(16) float slots[2][ROWS][64];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    Ring ring(ring_mem, a.cols);
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
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
    constexpr bool HELD = GradShape<T, E, WIDE, TPR>::HELD;
    float2 w[HELD ? E / 2 : U / 2], sw[E / 2], sb[E / 2];
    const W *weight = static_cast<const W *>(a.weight);
    if constexpr (HELD) ring.gather(weight, 1.f, w);
    // the weights of unit u: held, or read again
    auto weights = [&](int u) -> const float2 * {
        if constexpr (HELD) return w + u * U / 2;
        ring.gather_some(weight, 1.f, u, w);
        return w;
    };
#pragma unroll
    for (int i = 0; i < E / 2; ++i) sw[i] = sb[i] = both(0.f);
    int flip = 0;
    for (; row < a.rows; row += step, x += x_step, dy += dy_step, dx += dx_step) {
        cp_async_wait<STAGES - 2>();
        if constexpr (!WIDE) row_barrier<TPR, ROWS>();
        if (row + (STAGES - 1) * step < a.rows) {
            ring.copy(ring.slot_behind(), 0, x + (STAGES - 1) * x_step);
            ring.copy(ring.slot_behind(), 1, dy + (STAGES - 1) * dy_step);
        }
        cp_async_commit();
        const float2 m = both(-mean), rs = both(rstd);
        if (row + step < a.rows) mean = a.mean[row + step], rstd = a.rstd[row + step];
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int u = 0; u < Ring::NV; ++u) {
            float2 h[U / 2], g[U / 2];
            ring.read_some(0, x, u, h, -m.x);
            ring.read_some(1, dy, u, g);
            const float2 *wu = weights(u);
#pragma unroll
            for (int i = 0; i < U / 2; ++i) {
                // Past the row's end dy is 0, and so is its product with h if h is finite: it is
                // 0, or of WIDE rows -mean * rstd (which a row far from 0 with nearly no variance
                // takes past fp32's range) and kept out of the row's sum; no other sum of those
                // columns goes anywhere.  8192 x 512 fp16 8.6 us, 8192 x 1021 18.5 (18.3 without
                // the fill); the sum taken again by rows where it is NaN: 9.8 and 17.4.
                float2 &swi = sw[u * U / 2 + i], &sbi = sb[u * U / 2 + i];
                h[i] = mul2(add2(h[i], m), rs);
                swi = fma2(g[i], h[i], swi);
                sbi = add2(sbi, g[i]);
                g[i] = mul2(g[i], wu[i]);
                s0 = add2(s0, g[i]);
                if (!WIDE || ring.holds(u * U)) s1 = fma2(g[i], h[i], s1);
            }
        }
        float sums[2] = {s0.x + s0.y, s1.x + s1.y};
        row_sum<2, TPR, ROWS>(sums, slots[flip][threadIdx.y]);
        flip ^= 1;
        const float2 c1 = both(-sums[0] * a.inv_cols), c2 = both(-sums[1] * a.inv_cols);
#pragma unroll
        for (int u = 0; u < Ring::NV; ++u) {
            float2 h[U / 2], g[U / 2];
            ring.read_some(0, x, u, h);
            ring.read_some(1, dy, u, g);
            const float2 *wu = weights(u);
#pragma unroll
            for (int i = 0; i < U / 2; ++i) {
                h[i] = mul2(add2(h[i], m), rs);
                g[i] = mul2(fma2(h[i], c2, fma2(g[i], wu[i], c1)), rs);
            }
            ring.scatter_some(dx, u, g);
        }
        ring.next();
    }
    if (!a.partial) return;
    const int stride = static_cast<int>(part_stride(a.cols));
    float *part = a.partial + static_cast<int64_t>(blockIdx.x) * 2 * stride;
    if (ROWS == 1 || blockDim.y == 1) {
        ring.scatter(part, sw);
        ring.scatter(part + stride, sb);
        return;
    }
    // each row of threads puts its sums where its ring was, then all threads add them up
    cp_async_wait<0>();
    row_barrier<TPR, ROWS>();
    float *own = reinterpret_cast<float *>(ring_mem + threadIdx.y * Ring::BYTES);
    ring.scatter(own, sw);
    ring.scatter(own + stride, sb);
    __syncthreads();
    for (int u = static_cast<int>(threadIdx.y * TPR + threadIdx.x); u < stride / 2; u += static_cast<int>(blockDim.y) * TPR) {
        float4 t = *(reinterpret_cast<const float4 *>(ring_mem) + u);
        for (int r = 1; r < static_cast<int>(blockDim.y); ++r) {
            const float4 o = *(reinterpret_cast<const float4 *>(ring_mem + r * Ring::BYTES) + u);
            t.x += o.x, t.y += o.y, t.z += o.z, t.w += o.w;
        }
        *(reinterpret_cast<float4 *>(part) + u) = t;
    }
}

// Rows too long for registers: dx by one CTA per row in two passes, the second
// from L2 (2048 x 20480 fp16 with the weights' gradient 114 us, 2.2 TB/s), ...
template <typename T, typename W, bool WIDE>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const GradArgs a) {
    constexpr int VEC = WIDE ? kUnit<T> : 2;  // of a thread and step; odd rows by pairs of any alignment
    __shared__ __align__(16) float slot[64];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
    const W *weight = static_cast<const W *>(a.weight);
    ptx::griddep_wait();
    const float2 m = both(-a.mean[row]), rs = both(a.rstd[row]);
    // h and g of VEC columns from c on
    auto fetch = [&](int64_t c, float2 (&h)[VEC / 2], float2 (&g)[VEC / 2]) {
        if constexpr (WIDE) {
            load_pairs<T, VEC / 2>(x + c, h);
            load_pairs<T, VEC / 2>(dy + c, g);
        } else {
            const bool two = c + 1 < a.cols;
            h[0] = make_float2(to_f32(x[c]), two ? to_f32(x[c + 1]) : 0.f);
            g[0] = make_float2(to_f32(dy[c]), two ? to_f32(dy[c + 1]) : 0.f);
        }
        float2 w[VEC / 2];
        if constexpr (WIDE) {
            if (weight) load_pairs<W, VEC / 2>(weight + c, w);
        } else {
            if (weight) w[0] = make_float2(to_f32(weight[c]), c + 1 < a.cols ? to_f32(weight[c + 1]) : 0.f);
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            h[i] = mul2(add2(h[i], m), rs);
            if (weight) g[i] = mul2(g[i], w[i]);
        }
        // past the row's end, where -mean * rstd may not be finite
        if (!WIDE && c + 1 >= a.cols) h[0].y = 0.f;
    };
    float2 s0 = both(0.f), s1 = both(0.f);
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * VEC; c < a.cols; c += 1024 * VEC) {
        float2 h[VEC / 2], g[VEC / 2];
        fetch(c, h, g);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) s0 = add2(s0, g[i]), s1 = fma2(g[i], h[i], s1);
    }
    float sums[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sum<2, 1024, 1>(sums, slot);
    const float2 c1 = both(-sums[0] * a.inv_cols), c2 = both(-sums[1] * a.inv_cols);
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * VEC; c < a.cols; c += 1024 * VEC) {
        float2 h[VEC / 2], g[VEC / 2];
        fetch(c, h, g);
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) g[i] = mul2(fma2(h[i], c2, add2(g[i], c1)), rs);
        if constexpr (WIDE) {
            store_pairs<T, VEC / 2>(dx + c, g);
        } else {
            dx[c] = from_f32<T>(g[0].x);
            if (c + 1 < a.cols) dx[c + 1] = from_f32<T>(g[0].y);
        }
    }
}

// ... and the weights' partial sums by columns: blockIdx.y takes every
// gridDim.y-th row, a thread VEC columns.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) norm_columns_kernel(const GradArgs a) {
    constexpr int VEC = WIDE ? kUnit<T> : 1;
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t col = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * VEC;
    if (col >= a.cols) return;
    const int64_t stride = part_stride(a.cols);
    float *part = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * stride + col;
    if constexpr (WIDE) {
        float2 sw[VEC / 2], sb[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) sw[i] = sb[i] = both(0.f);
#pragma unroll 4
        for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
            float2 h[VEC / 2], d[VEC / 2];
            load_pairs<T, VEC / 2>(static_cast<const T *>(a.x) + r * a.x_stride + col, h);
            load_pairs<T, VEC / 2>(static_cast<const T *>(a.dy) + r * a.dy_stride + col, d);
            const float2 m = both(-a.mean[r]), rs = both(a.rstd[r]);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                sw[i] = fma2(d[i], mul2(add2(h[i], m), rs), sw[i]);
                sb[i] = add2(sb[i], d[i]);
            }
        }
        store_pairs<float, VEC / 2>(part, sw);
        store_pairs<float, VEC / 2>(part + stride, sb);
    } else {
        float sw = 0.f, sb = 0.f;
#pragma unroll 4
        for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
            const float d = to_f32(static_cast<const T *>(a.dy)[r * a.dy_stride + col]);
            sw += d * ((to_f32(static_cast<const T *>(a.x)[r * a.x_stride + col]) - a.mean[r]) * a.rstd[r]);
            sb += d;
        }
        part[0] = sw;
        part[stride] = sb;
    }
}

// dweight (blockIdx.y 0) or dbias (1) of 32 columns: each thread adds four columns
// of every 32nd part (all its loads on their way at once), then the part lanes of
// a warp and the warps are added, in a fixed order.
constexpr int kPartLanes = 32;

template <typename W>
__global__ void __launch_bounds__(256) norm_join_kernel(const float *partial, int parts, int cols, W *dweight,
                                                        W *dbias) {
    __shared__ float4 s[8][8];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int quad = static_cast<int>(threadIdx.x) % 8, lane = static_cast<int>(threadIdx.x) / 8;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + quad * 4;
    const int64_t stride = part_stride(cols);
    const float *p = partial + static_cast<int64_t>(blockIdx.y) * stride + col;
    constexpr int kEach = (kMaxParts + kPartLanes - 1) / kPartLanes;
    float4 v[kEach];
    ptx::griddep_wait();
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int i = k * kPartLanes + lane;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < parts && col < cols) v[k] = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(i) * 2 * stride);
    }
    float4 t = v[0];
#pragma unroll
    for (int k = 1; k < kEach; ++k) t.x += v[k].x, t.y += v[k].y, t.z += v[k].z, t.w += v[k].w;
#pragma unroll
    for (int o = 8; o < 32; o *= 2) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
        t.z += __shfl_xor_sync(0xffffffffu, t.z, o);
        t.w += __shfl_xor_sync(0xffffffffu, t.w, o);
    }
    if (threadIdx.x % 32 < 8) s[threadIdx.x / 32][quad] = t;
    __syncthreads();
    const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    if (threadIdx.x < 32 && out < cols) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += reinterpret_cast<const float *>(s[w])[threadIdx.x];
        (blockIdx.y ? dbias : dweight)[out] = from_f32<W>(sum);
    }
}

// ------------------------------------------------------------------- host --

template <typename T, typename W, int E, bool WIDE, int TPR>
int backward_ring(const GradArgs &a, int sms, int *parts, cudaStream_t stream) {
    using S = GradShape<T, E, WIDE, TPR>;
    auto *kernel = norm_backward_ring_kernel<T, W, E, WIDE, TPR>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, S::ROWS * S::ROW_BYTES, done)) return GEMM_ERR_CUDA;
    // few rows: spread over the SMs before they share one
    const int ctas = sms < kMaxParts ? sms : kMaxParts;
    const int64_t each = (a.rows + static_cast<int64_t>(ctas) - 1) / ctas;
    const int rows = each < S::ROWS ? static_cast<int>(each) : S::ROWS;
    *parts = grid_of(a.rows, rows, ctas);
    return launch(kernel, dim3(*parts), dim3(TPR, rows), rows * S::ROW_BYTES, stream, a);
}

template <typename T, typename W, bool WIDE>
int backward_rows(const GradArgs &a, int sms, int *parts, cudaStream_t stream) {
#define LINEAR_CASE(E, TPR)                                                      \
    if constexpr (GradShape<T, E, WIDE, TPR>::ROWS > 0) {                        \
        return backward_ring<T, W, E, WIDE, TPR>(a, sms, parts, stream);         \
    }                                                                            \
    break
    LINEAR_ROW_SHAPES(LINEAR_CASE)
#undef LINEAR_CASE
    int st = launch(norm_backward_long_kernel<T, W, WIDE>, dim3(a.rows), dim3(1024), 0, stream, a);
    if (st == GEMM_OK && a.partial) {
        constexpr int kCols = 256 * (WIDE ? kUnit<T> : 1);
        *parts = grid_of(a.rows, 1, kMaxParts);
        st = launch(norm_columns_kernel<T, WIDE>, dim3((a.cols + kCols - 1) / kCols, *parts), dim3(256), 0, stream, a);
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
    return launch(norm_join_kernel<W>, dim3((a.cols + 31) / 32, 2), dim3(256), 0, stream, a.partial, parts, a.cols,
                  static_cast<W *>(dweight), static_cast<W *>(dbias));
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int64_t layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (!sizes_ok(rows, cols)) return GEMM_ERR_INVALID_ARG;
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    return (rows < kMaxParts ? rows : kMaxParts) * 2 * part_stride(cols) * 4;
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
    if (rows_overlap(dx, dy, rows, cols * size, dx_stride * size, dy_stride * size) ||
        rows_overlap(dx, x, rows, cols * size, dx_stride * size, x_stride * size)) {
        return GEMM_ERR_INVALID_ARG;
    }
    for (int i = 0; i < 4; ++i) {
        for (int j = i == 0 ? 2 : 0; j < 5; ++j) {  // dx with dy and x above
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
