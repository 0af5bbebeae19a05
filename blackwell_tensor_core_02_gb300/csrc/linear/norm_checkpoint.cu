// norm_checkpoint.cu -- layer norm that keeps 8 bits an element, and its result from
// them (its gradient: norm_checkpoint_backward.cu;
// see checkpoint_ops.h and norm_rows.cuh).
//
// Bound by memory: the forward pass is layer norm's with the kept rows beside y, 1.03
// bytes an element.
#include <cmath>

#include "checkpoint_ops.h"
#include "fp8_rows.cuh"
#include "norm_rows.cuh"

namespace linear_ops {
namespace {

struct KeepArgs {
    const void *x, *weight, *bias;
    void *y;
    uint8_t *codes, *scales;
    float *rstd;
    int64_t x_stride, y_stride;
    int32_t rows, cols, blocks;
    float eps, inv_cols;
};

// Rows of a CTA, CTAs of an SM and stages: as layer norm's (norm_forward.cu).
constexpr int kStages = 3;
template <typename T, int E, bool WIDE, int TPR>
struct KeepShape {
    static constexpr int ROWS = TPR < 128 ? 128 / TPR : 1;
    static constexpr int BYTES = ROWS * RowRing<T, E, WIDE, TPR, 1, kStages>::BYTES;
    static constexpr int BY_SMEM = 220 * 1024 / (BYTES + 2048), BY_THREADS = (sizeof(T) == 4 ? 448 : 512) / (ROWS * TPR);
    static constexpr int PER_SM = BY_SMEM < BY_THREADS ? BY_SMEM : (BY_THREADS > 0 ? BY_THREADS : 1);
};

// A thread's share of a normalised row (0 past the row's end) to codes and scales.
//   WIDE   a block is the units of 4 lanes (fp32: 8)
//   else   a block is one element of each of a warp's lanes.  Each block's scale made by one
//          lane and handed round: 4096 x 4099 fp16 27.1 us, 517 x 1021 3.8; made by every lane
//          45.5 and 6.0.  (Consecutive elements a thread, shifted in registers to where a row
//          starts within 16 bytes, for wide stores: 43 and 6.8.)
template <typename T, int E, bool WIDE, int TPR>
__device__ __forceinline__ void keep_row(const RowShare<T, E, WIDE, TPR> &share, const float2 (&h)[E / 2], uint8_t *codes,
                                         uint8_t *scales, int blocks) {
    constexpr int U = kUnit<T>;
    const int lane = static_cast<int>(threadIdx.x) % 32;
    if constexpr (WIDE) {
        constexpr int kLanes = kFp8Block / U;
#pragma unroll
        for (int i = 0; i < E / U; ++i) {
            const float2 *v = h + i * U / 2;
            float amax = max_magnitude(v[0].x, v[0].y);
#pragma unroll
            for (int j = 1; j < U / 2; ++j) amax = max_magnitude(amax, max_magnitude(v[j].x, v[j].y));
#pragma unroll
            for (int o = 1; o < kLanes; o *= 2) amax = max_magnitude(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const uint32_t code = scale_code(amax);
            const float by = scale_inverse(code);
            if (!share.holds(i * U)) continue;
            const int column = share.column(i * U);
            uint32_t w[U / 4];
#pragma unroll
            for (int j = 0; j < U / 4; ++j) {
                const float2 a = mul2(v[2 * j], both(by)), b = mul2(v[2 * j + 1], both(by));
                w[j] = to_e4m3x2(a.x, a.y) | to_e4m3x2(b.x, b.y) << 16;
            }
            if constexpr (U == 8) {
                *reinterpret_cast<uint2 *>(codes + column) = make_uint2(w[0], w[1]);
            } else {
                *reinterpret_cast<uint32_t *>(codes + column) = w[0];
            }
            if (lane % kLanes == 0) scales[column / kFp8Block] = static_cast<uint8_t>(code);
        }
    } else {
        // lane e has the scale of the warp's e-th block, and makes its code for all
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float v = e % 2 ? h[e / 2].y : h[e / 2].x;
            const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(v)));
            if (lane == e) top = __uint_as_float(t);
        }
        const uint32_t code = scale_code(top);
        const float by = scale_inverse(code);
        const int block = lane * (TPR / 32) + static_cast<int>(threadIdx.x) / 32;
        if (lane < E && block < blocks) scales[block] = static_cast<uint8_t>(code);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float first = __shfl_sync(0xffffffffu, by, e), second = __shfl_sync(0xffffffffu, by, e + 1);
            const uint32_t pair = to_e4m3x2(h[e / 2].x * first, h[e / 2].y * second);
            if (share.holds(e)) codes[share.column(e)] = static_cast<uint8_t>(pair);
            if (share.holds(e + 1)) codes[share.column(e + 1)] = static_cast<uint8_t>(pair >> 8);
        }
    }
}

template <typename T, typename W, int E, bool WIDE, int TPR>
__global__ void __launch_bounds__(TPR *KeepShape<T, E, WIDE, TPR>::ROWS, KeepShape<T, E, WIDE, TPR>::PER_SM)
    norm_keep_ring_kernel(const KeepArgs a) {
    constexpr int ROWS = KeepShape<T, E, WIDE, TPR>::ROWS;
    using Ring = RowRing<T, E, WIDE, TPR, 1, kStages>;
    __shared__ __align__(16) float slots[2][ROWS][32];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    Ring ring(ring_mem, a.cols);
    int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.y;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
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
            // past the row's end there is nothing
            if (!ring.holds(2 * i)) v[i].x = 0.f;
            if (!ring.holds(WIDE ? 2 * i : 2 * i + 1)) v[i].y = 0.f;
            s2 = fma2(v[i], v[i], s2);
        }
        float var[1] = {s2.x + s2.y};
        row_sum<1, TPR, ROWS>(var, slots[1][threadIdx.y]);
        const float rstd = 1.f / sqrtf(var[0] * a.inv_cols + a.eps);
        if (threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            v[i] = mul2(v[i], both(rstd));
            // 0 * an infinite rstd (a row of one value, eps 0) past the end as well
            if (!ring.holds(2 * i)) v[i].x = 0.f;
            if (!ring.holds(WIDE ? 2 * i : 2 * i + 1)) v[i].y = 0.f;
        }
        keep_row<T, E, WIDE, TPR>(ring, v, a.codes + row * a.cols, a.scales + row * a.blocks, a.blocks);
        if (!a.y) continue;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) v[i] = fma2(v[i], w[i], b[i]);
        ring.scatter(y, v);
    }
}

// Rows too long for registers: one CTA of 1024 threads passes over its row three times;
// in the last a warp's 32 columns are a block.
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_keep_long_kernel(const KeepArgs a) {
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
    if (threadIdx.x == 0) a.rstd[row] = rstd;
    const int64_t end = (static_cast<int64_t>(a.cols) + 31) / 32 * 32;  // whole warps
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < end; c += 1024) {
        const float h = c < a.cols ? (to_f32(x[c]) - mean) * rstd : 0.f;
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(h)));
        const uint32_t code = scale_code(__uint_as_float(top));
        if (threadIdx.x % 32 == 0) a.scales[row * a.blocks + c / 32] = static_cast<uint8_t>(code);
        if (c >= a.cols) continue;
        a.codes[row * a.cols + c] = static_cast<uint8_t>(to_e4m3x2(h * scale_inverse(code), 0.f));
        if (!a.y) continue;
        const float w = a.weight ? to_f32(static_cast<const W *>(a.weight)[c]) : 1.f;
        const float b = a.bias ? to_f32(static_cast<const W *>(a.bias)[c]) : 0.f;
        y[c] = from_f32<T>(h * w + b);
    }
}

// --------------------------------------------------------------- restore --

struct RestoreArgs {
    const uint8_t *codes, *scales;
    const void *weight, *bias;
    void *y;
    int64_t y_stride;
    int32_t rows, cols, blocks;
};

// Whole units: a thread has the same 16 columns of every gridDim.y-th row (blockDim.y rows
// a CTA), whose weights it keeps.  Codes come ahead of time through shared memory, four
// rows at a time and two such batches on their way (a thread copies and reads its own, so
// there is no barrier); scales, bytes, a batch ahead in registers.  8192 x 4096 bf16
// 14.0 us; with a thread's codes in registers alone 21.8, 8 columns a thread 29.1.
template <typename T, typename W>
__global__ void __launch_bounds__(256) norm_restore_kernel(const RestoreArgs a) {
    constexpr int N = 16, R = 4, BATCHES = 3;
    __shared__ __align__(16) uint8_t ring[BATCHES * R][256 * 16];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t column = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * N;
    if (column >= a.cols) return;
    const uint32_t own = ptx::smem_u32(ring) + (threadIdx.y * blockDim.x + threadIdx.x) * 16u;
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.y) * blockDim.y + threadIdx.y;
    const uint8_t *codes = a.codes + row * a.cols + column, *scales = a.scales + row * a.blocks + column / kFp8Block;
    T *y = static_cast<T *>(a.y) + row * a.y_stride + column;
    const bool sectors = a.y_stride % 16 == 0 && reinterpret_cast<uintptr_t>(a.y) % 32 == 0;
    const int64_t code_step = step * a.cols, scale_step = step * a.blocks, y_step = step * a.y_stride;
    const uint8_t *ahead = codes;  // of the next batch to copy
    int64_t ahead_row = row;
    auto copy = [&](int batch) {
#pragma unroll
        for (int r = 0; r < R; ++r, ahead_row += step, ahead += code_step) {
            if (ahead_row < a.rows) cp_async_16(own + static_cast<uint32_t>(batch * R + r) * (256u * 16u), ahead);
        }
        cp_async_commit();
    };
    uint32_t next[R];
    auto load_scales = [&](int64_t first) {
#pragma unroll
        for (int r = 0; r < R; ++r, scales += scale_step) next[r] = first + r * step < a.rows ? *scales : 0u;
    };
    copy(0);
    copy(1);
    load_scales(row);
    float2 w[N / 2], b[N / 2];
#pragma unroll
    for (int j = 0; j < N / 2; ++j) w[j] = both(1.f), b[j] = both(0.f);
    if (a.weight) load_pairs<W, N / 2>(static_cast<const W *>(a.weight) + column, w);
    if (a.bias) load_pairs<W, N / 2>(static_cast<const W *>(a.bias) + column, b);
    for (int batch = 0; row < a.rows; batch = batch == BATCHES - 1 ? 0 : batch + 1) {
        copy(batch == 0 ? BATCHES - 1 : batch - 1);
        uint32_t scale[R];
#pragma unroll
        for (int r = 0; r < R; ++r) scale[r] = next[r];
        load_scales(row + R * step);
        cp_async_wait<BATCHES - 1>();
#pragma unroll
        for (int r = 0; r < R; ++r, row += step, y += y_step) {
            if (row >= a.rows) break;
            const uint4 u = ptx::ld_shared_v4(own + static_cast<uint32_t>(batch * R + r) * (256u * 16u));
            const uint32_t code[4] = {u.x, u.y, u.z, u.w};
            const float2 s = both(scale_value(scale[r]));
            float2 v[N / 2];
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const uint32_t pair = from_e4m3x2(code[j / 2] >> (j % 2 * 16) & 0xffffu);
                v[j] = fma2(mul2(__half22float2(*reinterpret_cast<const __half2 *>(&pair)), s), w[j], b[j]);
            }
            if (sectors) {  // a whole sector in one store, not two halves (8192 x 4096 to fp32 27.4 us, else 41.4)
                constexpr int kPairs = 8 / Pair<T>::WORDS;  // of a sector
#pragma unroll
                for (int i = 0; i < N / 2; i += kPairs) {
                    uint32_t t[8];
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) Pair<T>::narrow(v[i + j], t + j * Pair<T>::WORDS);
                    store_32(y + 2 * i, t);
                }
                continue;
            }
            store_pairs<T, N / 2>(y, v);
        }
    }
}

// Rows that start anywhere: a thread has the same four columns of every gridDim.y-th row,
// R at once.  Its codes lie in one or two aligned words (which hold a byte of the row each,
// so of its allocation), and go out in words of two where the row's address allows it.
template <typename T, typename W>
__global__ void __launch_bounds__(256) norm_restore_any_kernel(const RestoreArgs a) {
    constexpr int R = 4;
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t column = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 4;
    if (column >= a.cols) return;
    const int valid = a.cols - column < 4 ? static_cast<int>(a.cols - column) : 4;
    float w[4], b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = a.weight && j < valid ? to_f32(static_cast<const W *>(a.weight)[column + j]) : 1.f;
        b[j] = a.bias && j < valid ? to_f32(static_cast<const W *>(a.bias)[column + j]) : 0.f;
    }
    const int64_t step = static_cast<int64_t>(gridDim.y) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.y) * blockDim.y + threadIdx.y;
    const uint8_t *codes = a.codes + row * a.cols + column, *scales = a.scales + row * a.blocks + column / kFp8Block;
    T *y = static_cast<T *>(a.y) + row * a.y_stride + column;
    const int64_t code_step = step * a.cols, scale_step = step * a.blocks, y_step = step * a.y_stride;
    while (row < a.rows) {
        uint32_t low[R], high[R], head[R], scale[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            low[r] = high[r] = head[r] = scale[r] = 0u;
            if (row + r * step < a.rows) {
                head[r] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(codes) % 4);
                const uint32_t *word = reinterpret_cast<const uint32_t *>(codes - head[r]);
                low[r] = word[0];
                if (head[r] + valid > 4) high[r] = word[1];
                scale[r] = *scales;
            }
            codes += code_step, scales += scale_step;
        }
#pragma unroll
        for (int r = 0; r < R; ++r, row += step, y += y_step) {
            if (row >= a.rows) break;
            const uint32_t code = __funnelshift_r(low[r], high[r], head[r] * 8u);
            const float s = scale_value(scale[r]);
            const uint32_t first = from_e4m3x2(code & 0xffffu), second = from_e4m3x2(code >> 16);
            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&first)),
                         q = __half22float2(*reinterpret_cast<const __half2 *>(&second));
            const float v[4] = {fmaf(p.x * s, w[0], b[0]), fmaf(p.y * s, w[1], b[1]), fmaf(q.x * s, w[2], b[2]),
                                fmaf(q.y * s, w[3], b[3])};
            if constexpr (sizeof(T) == 2) {
                if (valid == 4) {
                    if (reinterpret_cast<uintptr_t>(y) % 4 == 0) {
                        uint32_t t[2];
                        Pair<T>::narrow(make_float2(v[0], v[1]), t);
                        Pair<T>::narrow(make_float2(v[2], v[3]), t + 1);
                        reinterpret_cast<uint32_t *>(y)[0] = t[0];
                        reinterpret_cast<uint32_t *>(y)[1] = t[1];
                    } else {
                        uint32_t t;
                        Pair<T>::narrow(make_float2(v[1], v[2]), &t);
                        y[0] = from_f32<T>(v[0]);
                        *reinterpret_cast<uint32_t *>(y + 1) = t;
                        y[3] = from_f32<T>(v[3]);
                    }
                    continue;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j < valid) y[j] = from_f32<T>(v[j]);
            }
        }
    }
}

// ------------------------------------------------------------------- host --

template <typename T, typename W, int E, bool WIDE, int TPR>
int keep_ring(const KeepArgs &a, int sms, cudaStream_t stream) {
    using S = KeepShape<T, E, WIDE, TPR>;
    auto *kernel = norm_keep_ring_kernel<T, W, E, WIDE, TPR>;
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(kernel, S::BYTES, done)) return GEMM_ERR_CUDA;
    return launch(kernel, dim3(grid_of(a.rows, S::ROWS, S::PER_SM * sms)), dim3(TPR, S::ROWS), S::BYTES, stream, a);
}

template <typename T, typename W, bool WIDE>
int keep_rows(const KeepArgs &a, int sms, cudaStream_t stream) {
#define LINEAR_CASE(E, TPR) return keep_ring<T, W, E, WIDE, TPR>(a, sms, stream)
    LINEAR_ROW_SHAPES(LINEAR_CASE)
#undef LINEAR_CASE
    return launch(norm_keep_long_kernel<T, W>, dim3(a.rows), dim3(1024), 0, stream, a);
}

template <typename T, typename W>
int keep_as(const KeepArgs &a, int sms, cudaStream_t stream) {
    constexpr int U = kUnit<T>;
    const bool wide = a.cols % U == 0 && a.x_stride % U == 0 && a.y_stride % U == 0 && aligned(a.x, 16) &&
                      aligned(a.y, 16) && aligned(a.codes, U) && (!a.weight || aligned(a.weight, 16)) &&
                      (!a.bias || aligned(a.bias, 16));
    return wide ? keep_rows<T, W, true>(a, sms, stream) : keep_rows<T, W, false>(a, sms, stream);
}

template <typename T, typename W>
int restore_as(const RestoreArgs &a, int sms, cudaStream_t stream) {
    const bool wide = a.cols % 16 == 0 && a.y_stride % 8 == 0 && aligned(a.y, 16) && aligned(a.codes, 16) &&
                      (!a.weight || aligned(a.weight, 16)) && (!a.bias || aligned(a.bias, 16));
    const int64_t units = wide ? a.cols / 16 : (static_cast<int64_t>(a.cols) + 3) / 4;
    // Threads of a row, of which an eighth at most has no unit: 4096 x 4099 fp16 18.2 us, 4096 x 4160 8.4;
    // 256 at most, but for short rows, 19.9 and 10.5.  fp32 rows that start anywhere take those:
    // 8192 x 333 4.3, 7.3 with the former.
    unsigned x = 256;
    if (wide || sizeof(T) == 2) {
        while (x > 8 && (units + x - 1) / x * x * 8 > units * 9) x /= 2;
    } else {
        while (x > 8 && x / 2 >= units) x /= 2;
    }
    const unsigned y = 256 / x;
    const int64_t across = (units + x - 1) / x;
    // CTAs of four rows a thread, as far as they run at once
    int64_t down = (static_cast<int64_t>(a.rows) + 4 * y - 1) / (4 * y);
    const int64_t most = (static_cast<int64_t>(sms) * (wide ? 3 : 6) + across - 1) / across;
    if (down > most) down = most;
    if (down > 65535) down = 65535;
    auto *kernel = wide ? norm_restore_kernel<T, W> : norm_restore_any_kernel<T, W>;
    return launch(kernel, dim3(static_cast<unsigned>(across), static_cast<unsigned>(down)), dim3(x, y), 0, stream, a);
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int norm_checkpoint_forward(const void *x, int64_t x_stride, const void *weight, const void *bias, void *y,
                            int64_t y_stride, void *codes, void *scales, float *rstd, int64_t rows, int64_t cols,
                            float eps, int32_t type, int32_t weight_type, void *stream) {
    if (!sizes_ok(rows, cols) || !type_ok(type) || (weight_type != type && weight_type != LINEAR_F32) || !(eps >= 0.f) ||
        std::isinf(eps) || x_stride < 0) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return GEMM_OK;
    if (!x || !codes || !scales || !rstd || (y && rows > 1 && y_stride < cols)) return GEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), wsize = type_size(weight_type), blocks = fp8_blocks(cols);
    if (!aligned(x, size) || !aligned(y, size) || !aligned(weight, wsize) || !aligned(bias, wsize) || !aligned(rstd, 4)) {
        return GEMM_ERR_MISALIGNED;
    }
    if (rows == 1) x_stride = 0;
    if (rows == 1 || !y) y_stride = 0;
    const Span outs[4] = {{y, y ? span_bytes(rows, cols, y_stride, size) : 0}, {codes, rows * cols}, {scales, rows * blocks}, {rstd, rows * 4}},
               ins[3] = {{x, span_bytes(rows, cols, x_stride, size)}, {weight, cols * wsize}, {bias, cols * wsize}};
    if (rows_overlap(y, x, rows, cols * size, y_stride * size, x_stride * size) || any_overlap(outs, ins)) return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    const int st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    const KeepArgs a = {x, weight, bias, y, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales), rstd, x_stride,
                        y_stride, static_cast<int32_t>(rows), static_cast<int32_t>(cols), static_cast<int32_t>(blocks), eps,
                        1.f / static_cast<float>(cols)};
    return LINEAR_BY_TYPE(type, weight_type, keep_as, a, sms, static_cast<cudaStream_t>(stream));
}

int norm_checkpoint_restore(const void *codes, const void *scales, const void *weight, const void *bias, void *y,
                            int64_t y_stride, int64_t rows, int64_t cols, int32_t type, int32_t weight_type,
                            void *stream) {
    if (!sizes_ok(rows, cols) || !type_ok(type) || (weight_type != type && weight_type != LINEAR_F32)) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return GEMM_OK;
    if (!codes || !scales || !y || (rows > 1 && y_stride < cols)) return GEMM_ERR_INVALID_ARG;
    const int64_t size = type_size(type), wsize = type_size(weight_type), blocks = fp8_blocks(cols);
    if (!aligned(y, size) || !aligned(weight, wsize) || !aligned(bias, wsize)) return GEMM_ERR_MISALIGNED;
    if (rows == 1) y_stride = 0;
    const Span outs[1] = {{y, span_bytes(rows, cols, y_stride, size)}},
               ins[4] = {{codes, rows * cols}, {scales, rows * blocks}, {weight, cols * wsize}, {bias, cols * wsize}};
    if (overlap(y, outs[0].bytes, codes, rows * cols) || any_overlap(outs, ins)) return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    const int st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    const RestoreArgs a = {static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), weight, bias, y, y_stride,
                           static_cast<int32_t>(rows), static_cast<int32_t>(cols), static_cast<int32_t>(blocks)};
    return LINEAR_BY_TYPE(type, weight_type, restore_as, a, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
