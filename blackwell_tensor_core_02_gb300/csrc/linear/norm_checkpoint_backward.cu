// norm_checkpoint_backward.cu -- the gradient of layer norm from 8 bits an element (see
// checkpoint_ops.h, norm_rows.cuh and norm_parts.cuh).
//
// Bound by memory: it reads the kept rows in place of x, at 16 bits an element 5.03
// bytes in all where layer norm's own gradient reads and writes 6.
#include "checkpoint_ops.h"
#include "fp8_rows.cuh"
#include "norm_parts.cuh"
#include "norm_rows.cuh"

namespace linear_ops {
namespace {

// -------------------------------------------------------------- gradient --

struct KeptGradArgs {
    const void *dy, *weight;
    const uint8_t *codes, *scales;
    const float *rstd;
    void *dx;
    float *partial;
    int64_t dy_stride, dx_stride;
    int32_t rows, cols, blocks;
    float inv_cols;
};

// U bytes (4 or 8) on their way to shared memory.
template <int U>
__device__ __forceinline__ void cp_async_few(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(U) : "memory");
}

// The kept rows on their way to shared memory, beside dy's ring (RowRing), a slot a stage.
//   WIDE   a thread copies and reads its own units' codes; it loads their scales itself,
//          a row ahead (they are few, and bytes)
//   else   the 16-byte units that hold a row's codes, and its scales, are copied, and
//          read by elements behind the ring's barrier; a warp's e-th elements are a
//          block, whose scale lane e has
template <typename T, int E, bool WIDE, int TPR>
struct KeptRing {
    static constexpr int U = kUnit<T>, NV = E / U;
    static constexpr uint32_t CODES = WIDE ? E * TPR : E * TPR + 16;
    static constexpr uint32_t SCALES = WIDE ? 0 : (E * TPR / 32 + 31) / 16 * 16;
    static constexpr uint32_t SLOT = CODES + SCALES;
    static_assert(SLOT % 16 == 0, "aligned slots");
    uint32_t base;
    int cols, blocks;

    static __device__ __forceinline__ void copy_units(uint32_t dst, const uint8_t *row, int bytes) {
        const uint32_t head = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) % 16);
        const int end = static_cast<int>(head) + bytes;
        for (int at = static_cast<int>(threadIdx.x) * 16; at < end; at += TPR * 16) {
            cp_async_16(dst + at, row - head + at, static_cast<uint32_t>(end - at < 16 ? end - at : 16));
        }
    }
    template <typename S>
    __device__ __forceinline__ void copy(const S &share, int s, const uint8_t *codes, const uint8_t *scales) const {
        const uint32_t dst = base + static_cast<uint32_t>(s) * SLOT;
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (share.holds(i * U)) cp_async_few<U>(dst + (i * TPR + threadIdx.x) * U, codes + share.column(i * U));
            }
        } else {
            copy_units(dst, codes, cols);
            copy_units(dst + CODES, scales, blocks);
        }
    }
    // this thread's units' scale codes (WIDE), 127 (1) past the row's end
    template <typename S>
    __device__ __forceinline__ void load_scales(const S &share, const uint8_t *scales, uint32_t (&code)[NV]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            code[i] = 127u;
            if (share.holds(i * U)) code[i] = scales[share.column(i * U) / kFp8Block];
        }
    }
    // (not WIDE) the scale of the warp's block `lane` in slot s, 1 past the row's end
    __device__ __forceinline__ float lane_scale(int s, const uint8_t *scales) const {
        const int lane = static_cast<int>(threadIdx.x) % 32, block = lane * (TPR / 32) + static_cast<int>(threadIdx.x) / 32;
        uint32_t t = 127u;
        if (lane < E && block < blocks) {
            const uint32_t at = base + static_cast<uint32_t>(s) * SLOT + CODES + static_cast<uint32_t>(reinterpret_cast<uintptr_t>(scales) % 16);
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(t) : "r"(at + block) : "memory");
        }
        return scale_value(t);
    }
    // the values of unit i of this thread in slot s, 0 past the row's end, without a WIDE unit's
    // scale if not SCALED; all of a warp's threads call it
    template <bool SCALED, typename S>
    __device__ __forceinline__ void read(const S &share, int s, int i, const uint8_t *codes, float scale_of_lane,
                                         const uint32_t (&code)[NV], float2 *h) const {
        const uint32_t src = base + static_cast<uint32_t>(s) * SLOT;
        if constexpr (WIDE) {
            uint32_t w[2] = {0, 0};
            if (share.holds(i * U)) {
                const uint32_t at = src + (i * TPR + threadIdx.x) * U;
                if constexpr (U == 8) {
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
                } else {
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
                }
            }
            const float2 scale = both(scale_value(code[i]));
#pragma unroll
            for (int j = 0; j < U / 2; ++j) {
                const uint32_t pair = from_e4m3x2(w[j / 2] >> (j % 2 * 16) & 0xffffu);
                h[j] = __half22float2(*reinterpret_cast<const __half2 *>(&pair));
                if constexpr (SCALED) h[j] = mul2(h[j], scale);
            }
        } else {
            const uint32_t at = src + static_cast<uint32_t>(reinterpret_cast<uintptr_t>(codes) % 16);
#pragma unroll
            for (int j = 0; j < U; j += 2) {
                const int e = i * U + j;
                uint32_t c = 0, d = 0;
                if (share.holds(e)) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(c) : "r"(at + share.column(e)) : "memory");
                if (share.holds(e + 1)) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(d) : "r"(at + share.column(e + 1)) : "memory");
                const uint32_t pair = from_e4m3x2(c | d << 8);
                const float first = __shfl_sync(0xffffffffu, scale_of_lane, e), second = __shfl_sync(0xffffffffu, scale_of_lane, e + 1);
                h[j / 2] = mul2(__half22float2(*reinterpret_cast<const __half2 *>(&pair)), make_float2(first, second));
                // a block of no element has no scale
                if (!share.holds(e)) h[j / 2].x = 0.f;
                if (!share.holds(e + 1)) h[j / 2].y = 0.f;
            }
        }
    }
};

template <typename T, int E, bool WIDE, int TPR>
struct KeptGradShape {
    // Threads of a CTA, one a SM: rows that start anywhere took, with a row of 160 threads and
    // with two, 4096 x 4099 fp16 84 and 55 us; of one warp, 8 rows and 12, 8192 x 1021 28.6 and 30.3.
    // (Their scales a lane each, since, not an element each: 38.2 and 16.0.)
    static constexpr int BUDGET = 200 * 1024;
    static constexpr int ROW = RowRing<T, E, WIDE, TPR, 1, 1>::BYTES + KeptRing<T, E, WIDE, TPR>::SLOT;
    static constexpr bool HELD = TPR <= 384;  // the weights, in registers
    static constexpr int STAGES = (WIDE && TPR <= 64) || !HELD || 3 * ROW > BUDGET ? 2 : 3;
    static constexpr int ROW_BYTES = STAGES * ROW > 2 * 4 * TPR * E ? STAGES * ROW : 2 * 4 * TPR * E;  // a row's sums go there
    static constexpr int BY_SMEM = BUDGET / ROW_BYTES, BY_THREADS = E <= 16 ? 512 / TPR : (TPR >= 384 ? 1 : (WIDE || TPR > 32 ? 384 : 256) / TPR);
    static constexpr int ROWS = BY_SMEM < BY_THREADS ? BY_SMEM : BY_THREADS;  // at most; 0: no room for a row
};

// As norm_backward_ring_kernel (norm_backward.cu), with h from the kept rows.
template <typename T, typename W, int E, bool WIDE, int TPR>
__global__ void __launch_bounds__(TPR *KeptGradShape<T, E, WIDE, TPR>::ROWS, 1)
    norm_kept_backward_kernel(const KeptGradArgs a) {
    using S = KeptGradShape<T, E, WIDE, TPR>;
    constexpr int ROWS = S::ROWS, STAGES = S::STAGES;
    using Ring = RowRing<T, E, WIDE, TPR, 1, STAGES>;
    using Kept = KeptRing<T, E, WIDE, TPR>;
    constexpr int U = Ring::U;
    __shared__ __align__(16) float slots[2][ROWS][64];
    extern __shared__ __align__(16) uint8_t ring_mem[];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    uint8_t *own = ring_mem + threadIdx.y * S::ROW_BYTES;
    Ring ring(ring_mem, a.cols);
    ring.base = ptx::smem_u32(own);
    const Kept kept{ptx::smem_u32(own) + Ring::BYTES, a.cols, a.blocks};
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
    const uint8_t *codes = a.codes + row * a.cols, *scales = a.scales + row * a.blocks;
    const int64_t dy_step = step * a.dy_stride, dx_step = step * a.dx_stride, code_step = step * a.cols,
                  scale_step = step * a.blocks;
    ptx::griddep_wait();
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (row + s * step < a.rows) {
            ring.copy(s, 0, dy + s * dy_step);
            kept.copy(ring, s, codes + s * code_step, scales + s * scale_step);
        }
        cp_async_commit();
    }
    float rstd = 0.f;
    uint32_t next[Kept::NV], code[Kept::NV];
    if (row < a.rows) {
        rstd = a.rstd[row];
        if constexpr (WIDE) kept.load_scales(ring, scales, next);
    }
    constexpr bool HELD = S::HELD;
    float2 w[HELD ? E / 2 : U / 2], sw[E / 2], sb[E / 2];
    const W *weight = static_cast<const W *>(a.weight);
    if constexpr (HELD) ring.gather(weight, 1.f, w);
    auto weights = [&](int u) -> const float2 * {
        if constexpr (HELD) return w + u * U / 2;
        ring.gather_some(weight, 1.f, u, w);
        return w;
    };
#pragma unroll
    for (int i = 0; i < E / 2; ++i) sw[i] = sb[i] = both(0.f);
    int flip = 0;
    for (; row < a.rows; row += step, dy += dy_step, dx += dx_step, codes += code_step, scales += scale_step) {
        cp_async_wait<STAGES - 2>();
        if constexpr (!WIDE) row_barrier<TPR, ROWS>();
        if (row + (STAGES - 1) * step < a.rows) {
            ring.copy(ring.slot_behind(), 0, dy + (STAGES - 1) * dy_step);
            kept.copy(ring, ring.slot_behind(), codes + (STAGES - 1) * code_step, scales + (STAGES - 1) * scale_step);
        }
        cp_async_commit();
        const float2 rs = both(rstd);
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < Kept::NV; ++i) code[i] = next[i];
        }
        if (row + step < a.rows) {
            rstd = a.rstd[row + step];
            if constexpr (WIDE) kept.load_scales(ring, scales + scale_step, next);
        }
        float scale_of_lane = 1.f;
        if constexpr (!WIDE) scale_of_lane = kept.lane_scale(ring.slot, scales);
        float2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
        for (int u = 0; u < Ring::NV; ++u) {
            float2 h[U / 2], g[U / 2];
            kept.template read<true>(ring, ring.slot, u, codes, scale_of_lane, code, h);
            ring.read_some(0, dy, u, g);
            const float2 *wu = weights(u);
#pragma unroll
            for (int i = 0; i < U / 2; ++i) {
                float2 &swi = sw[u * U / 2 + i], &sbi = sb[u * U / 2 + i];
                swi = fma2(g[i], h[i], swi);
                sbi = add2(sbi, g[i]);
                g[i] = mul2(g[i], wu[i]);
                s0 = add2(s0, g[i]);
                s1 = fma2(g[i], h[i], s1);
            }
        }
        float sums[2] = {s0.x + s0.y, s1.x + s1.y};
        row_sum<2, TPR, ROWS>(sums, slots[flip][threadIdx.y]);
        flip ^= 1;
        const float2 c1 = both(-sums[0] * a.inv_cols), c2 = both(-sums[1] * a.inv_cols);
        auto c2_of = [&](int u) {  // with a unit's scale, a power of two, where h comes without
            if constexpr (WIDE) return mul2(c2, both(scale_value(code[u])));
            return c2;
        };
#pragma unroll
        for (int u = 0; u < Ring::NV; ++u) {
            float2 h[U / 2], g[U / 2];
            kept.template read<false>(ring, ring.slot, u, codes, scale_of_lane, code, h);
            ring.read_some(0, dy, u, g);
            const float2 *wu = weights(u);
            const float2 cu = c2_of(u);
#pragma unroll
            for (int i = 0; i < U / 2; ++i) g[i] = mul2(fma2(h[i], cu, fma2(g[i], wu[i], c1)), rs);
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
    ring.scatter(reinterpret_cast<float *>(own), sw);
    ring.scatter(reinterpret_cast<float *>(own) + stride, sb);
    __syncthreads();
    for (int u = static_cast<int>(threadIdx.y * TPR + threadIdx.x); u < stride / 2; u += static_cast<int>(blockDim.y) * TPR) {
        float4 t = *(reinterpret_cast<const float4 *>(ring_mem) + u);
        for (int r = 1; r < static_cast<int>(blockDim.y); ++r) {
            const float4 o = *(reinterpret_cast<const float4 *>(ring_mem + r * S::ROW_BYTES) + u);
            t.x += o.x, t.y += o.y, t.z += o.z, t.w += o.w;
        }
        *(reinterpret_cast<float4 *>(part) + u) = t;
    }
}

// Rows without room in the ring: dx by one CTA per row in two passes, ...
template <typename T, typename W>
__global__ void __launch_bounds__(1024) norm_kept_backward_long_kernel(const KeptGradArgs a) {
    __shared__ __align__(16) float slot[64];
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    const int64_t row = blockIdx.x;
    const T *dy = static_cast<const T *>(a.dy) + row * a.dy_stride;
    T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
    const W *weight = static_cast<const W *>(a.weight);
    ptx::griddep_wait();
    const float rstd = a.rstd[row];
    auto fetch = [&](int64_t c, float *h, float *g) {
        const uint32_t pair = from_e4m3x2(a.codes[row * a.cols + c]);
        *h = __low2float(*reinterpret_cast<const __half2 *>(&pair)) * scale_value(a.scales[row * a.blocks + c / kFp8Block]);
        *g = to_f32(dy[c]) * (weight ? to_f32(weight[c]) : 1.f);
    };
    float sums[2] = {0.f, 0.f};
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        float h, g;
        fetch(c, &h, &g);
        sums[0] += g;
        sums[1] = fmaf(g, h, sums[1]);
    }
    row_sum<2, 1024, 1>(sums, slot);
    const float c1 = -sums[0] * a.inv_cols, c2 = -sums[1] * a.inv_cols;
#pragma unroll 4
    for (int64_t c = threadIdx.x; c < a.cols; c += 1024) {
        float h, g;
        fetch(c, &h, &g);
        dx[c] = from_f32<T>(fmaf(h, c2, g + c1) * rstd);
    }
}

// ... and the weights' partial sums by columns: blockIdx.y takes every gridDim.y-th row.
template <typename T>
__global__ void __launch_bounds__(256) norm_kept_columns_kernel(const KeptGradArgs a) {
    if (threadIdx.x == 0) ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (col >= a.cols) return;
    float sw = 0.f, sb = 0.f;
#pragma unroll 4
    for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y) {
        const uint32_t pair = from_e4m3x2(a.codes[r * a.cols + col]);
        const float h = __low2float(*reinterpret_cast<const __half2 *>(&pair)) * scale_value(a.scales[r * a.blocks + col / kFp8Block]);
        const float d = to_f32(static_cast<const T *>(a.dy)[r * a.dy_stride + col]);
        sw = fmaf(d, h, sw);
        sb += d;
    }
    const int64_t stride = part_stride(a.cols);
    float *part = a.partial + static_cast<int64_t>(blockIdx.y) * 2 * stride + col;
    part[0] = sw;
    part[stride] = sb;
}

// ------------------------------------------------------------------- host --

template <typename T, typename W, int E, bool WIDE, int TPR>
int kept_ring(const KeptGradArgs &a, int sms, int *parts, cudaStream_t stream) {
    using S = KeptGradShape<T, E, WIDE, TPR>;
    auto *kernel = norm_kept_backward_kernel<T, W, E, WIDE, TPR>;
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
int kept_rows(const KeptGradArgs &a, int sms, int *parts, cudaStream_t stream) {
#define LINEAR_CASE(E, TPR)                                                      \
    if constexpr (KeptGradShape<T, E, WIDE, TPR>::ROWS > 0) {                    \
        return kept_ring<T, W, E, WIDE, TPR>(a, sms, parts, stream);             \
    }                                                                            \
    break
    LINEAR_ROW_SHAPES(LINEAR_CASE)
#undef LINEAR_CASE
    int st = launch(norm_kept_backward_long_kernel<T, W>, dim3(a.rows), dim3(1024), 0, stream, a);
    if (st == GEMM_OK && a.partial) {
        *parts = grid_of(a.rows, 1, kMaxParts);
        st = launch(norm_kept_columns_kernel<T>, dim3((a.cols + 255) / 256, *parts), dim3(256), 0, stream, a);
    }
    return st;
}

template <typename T, typename W>
int kept_as(const KeptGradArgs &a, void *dweight, void *dbias, int sms, cudaStream_t stream) {
    constexpr int U = kUnit<T>;
    const bool wide = a.cols % U == 0 && a.dy_stride % U == 0 && a.dx_stride % U == 0 && aligned(a.dy, 16) &&
                      aligned(a.dx, 16) && aligned(a.codes, U) && (!a.weight || aligned(a.weight, 16));
    int parts = 0;
    if (a.rows > 0) {
        const int st = wide ? kept_rows<T, W, true>(a, sms, &parts, stream) : kept_rows<T, W, false>(a, sms, &parts, stream);
        if (st != GEMM_OK || !dweight) return st;
    }
    return launch(norm_join_kernel<W>, dim3((a.cols + 31) / 32, 2), dim3(256), 0, stream, a.partial, parts, a.cols,
                  static_cast<W *>(dweight), static_cast<W *>(dbias));
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int norm_checkpoint_backward(const void *dy, int64_t dy_stride, const void *codes, const void *scales, const void *weight,
                             const float *rstd, void *dx, int64_t dx_stride, void *dweight, void *dbias, int64_t rows,
                             int64_t cols, int32_t type, int32_t weight_type, void *workspace, int64_t workspace_bytes,
                             void *stream) {
    if (!sizes_ok(rows, cols) || !type_ok(type) || (weight_type != type && weight_type != LINEAR_F32) || dy_stride < 0 ||
        !dweight != !dbias || workspace_bytes < 0) {
        return GEMM_ERR_INVALID_ARG;
    }
    if (rows > kMaxDim || cols > kMaxDim) return GEMM_ERR_UNSUPPORTED_SHAPE;
    if (rows > 0 && (!dy || !codes || !scales || !rstd || !dx || (rows > 1 && dx_stride < cols))) return GEMM_ERR_INVALID_ARG;
    if (rows == 0 && !dweight) return GEMM_OK;
    const int64_t need = dweight ? layer_norm_backward_workspace_size(rows, cols) : 0;
    if (need > 0 && !workspace) return GEMM_ERR_INVALID_ARG;
    if (workspace_bytes < need) return GEMM_ERR_SCRATCH_LIMIT;
    const int64_t size = type_size(type), wsize = type_size(weight_type), blocks = fp8_blocks(cols);
    if (!aligned(dy, size) || !aligned(dx, size) || !aligned(weight, wsize) || !aligned(dweight, wsize) ||
        !aligned(dbias, wsize) || !aligned(rstd, 4) || (need > 0 && !aligned(workspace, 16))) {
        return GEMM_ERR_MISALIGNED;
    }
    if (rows <= 1) dy_stride = dx_stride = 0;
    const Span outs[4] = {{dx, span_bytes(rows, cols, dx_stride, size)}, {dweight, cols * wsize}, {dbias, cols * wsize},
                          {workspace, need}},
               ins[5] = {{dy, span_bytes(rows, cols, dy_stride, size)}, {codes, rows * cols}, {scales, rows * blocks},
                         {weight, cols * wsize}, {rstd, rows * 4}};
    if (rows_overlap(dx, dy, rows, cols * size, dx_stride * size, dy_stride * size) || any_overlap(outs, ins)) return GEMM_ERR_INVALID_ARG;
    int sms = 0;
    const int st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    const KeptGradArgs a = {dy, weight, static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), rstd, dx,
                            dweight ? static_cast<float *>(workspace) : nullptr, dy_stride, dx_stride,
                            static_cast<int32_t>(rows), static_cast<int32_t>(cols), static_cast<int32_t>(blocks),
                            1.f / static_cast<float>(cols)};
    return LINEAR_BY_TYPE(type, weight_type, kept_as, a, dweight, dbias, sms, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
