// norm_rows.cuh -- rows of layer norm and its gradient: their sizes, and a ring of
// rows on their way into shared memory.
//
// Both operators are bound by memory: forward reads a row and writes one, its
// gradient reads two and writes one, at 8 and 14 operations an element.  So each
// element is read from memory once and held in registers while its row's sums
// are formed (the variance from the centred values: E[x^2] - mean^2 loses what
// an offset of the row costs), and a persistent grid keeps the next rows on
// their way meanwhile.
#pragma once

#include "common.cuh"

namespace linear_ops {

// Elements of a row that a thread holds, and the threads: a sum over a row costs
// each warp some 50 instructions and a barrier, so few warps with many elements
// are faster (8192 x 4096 bf16 when it was chosen, us: 8 elements 36.6, 16 25.4,
// 32 23.7; gradient 66, 41.4, 41.7).  Whole warps up to 8 serve the widths up to
// 8192 and 12 and 16 those up to 16384; short rows of one warp take fewer elements
// (4976 x 639: 32 each 6.8 us, 24 each 5.2).
constexpr int kEach = 32;

// The columns of a row that the TPR threads of threadIdx.x hold, E each, as pairs.
//   WIDE   rows are whole 16-byte units: thread t holds units t, t + TPR, ...
//   else   rows start anywhere: thread t holds columns t, t + TPR, ...
template <typename T, int E, bool WIDE, int TPR>
struct RowShare {
    static constexpr int U = kUnit<T>;
    static constexpr int NV = E / U;  // units of a thread
    static_assert(E % U == 0, "whole units");
    int cols;
    // Columns of the narrowest row of this shape, less one (LINEAR_ROW_SHAPES); for
    // WIDE rows of one warp it is not used: the gradient of 8192 x 1024 took 18.3 us
    // with it and 14.8 with the comparisons.
    static constexpr int kFewest = TPR > 256 ? (TPR - 128) * E : (TPR > 32 ? (TPR - 32) * E : (WIDE ? 0 : (E - 8) * 32));
    // the column of element e (a constant after unrolling), and whether it is one of
    // the row's: known without a comparison for what the narrowest row has
    __device__ __forceinline__ int column(int e) const {
        return WIDE ? (e / U * TPR + static_cast<int>(threadIdx.x)) * U + e % U : e * TPR + static_cast<int>(threadIdx.x);
    }
    __device__ __forceinline__ bool holds(int e) const {
        const int past = WIDE ? (e / U + 1) * U * TPR : (e + 1) * TPR;  // every thread's element e lies before this
        return past <= kFewest || column(WIDE ? e / U * U : e) < cols;
    }

    // U of this thread's values (the i-th U of its E) of a vector by columns, `fill`
    // past its end and without a vector
    template <typename W>
    __device__ __forceinline__ void gather_some(const W *from, float fill, int i, float2 *v) const {
#pragma unroll
        for (int j = 0; j < U / 2; ++j) v[j] = both(fill);
        if (!from) return;
        if constexpr (WIDE) {
            if (holds(i * U)) load_pairs<W, U / 2>(from + column(i * U), v);
        } else {
#pragma unroll
            for (int j = 0; j < U / 2; ++j) {
                const int e = i * U + 2 * j;
                if (holds(e)) v[j].x = to_f32(from[column(e)]);
                if (holds(e + 1)) v[j].y = to_f32(from[column(e + 1)]);
            }
        }
    }
    template <typename W>
    __device__ __forceinline__ void gather(const W *from, float fill, float2 (&v)[E / 2]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) gather_some(from, fill, i, v + i * U / 2);
    }
    // U of this thread's values (the i-th U of its E) to a vector by columns
    template <typename W>
    __device__ __forceinline__ void scatter_some(W *to, int i, const float2 *v) const {
        if constexpr (WIDE) {
            if (holds(i * U)) store_pairs<W, U / 2>(to + column(i * U), v);
        } else {
#pragma unroll
            for (int j = 0; j < U / 2; ++j) {
                const int e = i * U + 2 * j;
                if (holds(e)) to[column(e)] = from_f32<W>(v[j].x);
                if (holds(e + 1)) to[column(e + 1)] = from_f32<W>(v[j].y);
            }
        }
    }
    template <typename W>
    __device__ __forceinline__ void scatter(W *to, const float2 (&v)[E / 2]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) scatter_some(to, i, v + i * U / 2);
    }
};

// Some rows of OPS operands on their way from global to shared memory: STAGES
// slots for each row of a CTA.
//   WIDE   a thread copies and reads its own units, so no barrier guards the ring
//   else   the 16-byte units that hold the row are copied (the first may start
//          with bytes that lie before the row; they share an aligned 16 bytes
//          with it, so its allocation; the last is cut at the row's end), and a
//          barrier is due between copying and reading, and between reading and
//          the next copy into that slot
template <typename T, int E, bool WIDE, int TPR, int OPS, int STAGES>
struct RowRing : RowShare<T, E, WIDE, TPR> {
    using Share = RowShare<T, E, WIDE, TPR>;
    using Share::cols;
    using Share::NV;
    using Share::U;
    static constexpr uint32_t SLOT = (NV * TPR + (WIDE ? 0 : 1)) * 16;
    static constexpr uint32_t BYTES = STAGES * OPS * SLOT;  // of one row's ring
    uint32_t base;
    int slot = 0;

    __device__ __forceinline__ RowRing(void *ring, int cols_) : Share{cols_} {
        base = ptx::smem_u32(ring) + threadIdx.y * BYTES;
    }
    __device__ __forceinline__ void copy(int s, int op, const T *row) const {
        const uint32_t dst = base + static_cast<uint32_t>(s * OPS + op) * SLOT;
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (this->holds(i * U)) cp_async_16(dst + (i * TPR + threadIdx.x) * 16u, row + this->column(i * U));
            }
        } else {
            const uint32_t head = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) % 16);
            const char *from = reinterpret_cast<const char *>(row) - head;
            const int end = static_cast<int>(head) + cols * static_cast<int>(sizeof(T));
#pragma unroll
            for (int i = 0; i <= NV; ++i) {
                const int at = (i * TPR + static_cast<int>(threadIdx.x)) * 16;
                if (at < end) cp_async_16(dst + at, from + at, static_cast<uint32_t>(end - at < 16 ? end - at : 16));
            }
        }
    }
    // U of this thread's elements (the i-th U of its E) of the current slot; past the
    // row's end `fill`, of WIDE rows 0
    __device__ __forceinline__ void read_some(int op, const T *row, int i, float2 *v, float fill = 0.f) const {
        const uint32_t src = base + static_cast<uint32_t>(slot * OPS + op) * SLOT;
        if constexpr (WIDE) {
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (this->holds(i * U)) raw = ptx::ld_shared_v4(src + (i * TPR + threadIdx.x) * 16u);
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int j = 0; j < U / 2; ++j) v[j] = Pair<T>::widen(w + j * Pair<T>::WORDS);
        } else {
            const uint32_t at = src + static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) % 16) +
                                threadIdx.x * static_cast<uint32_t>(sizeof(T));
            float f[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int e = i * U + j;
                f[j] = fill;
                if (this->holds(e)) {
                    if constexpr (sizeof(T) == 4) {
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[j]) : "r"(at + e * TPR * 4u) : "memory");
                    } else {
                        uint16_t u;
                        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at + e * TPR * 2u) : "memory");
                        f[j] = to_f32(*reinterpret_cast<const T *>(&u));
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < U / 2; ++j) v[j] = make_float2(f[2 * j], f[2 * j + 1]);
        }
    }
    __device__ __forceinline__ void read(int op, const T *row, float2 (&v)[E / 2]) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) read_some(op, row, i, v + i * U / 2);
    }
    __device__ __forceinline__ void next() { slot = slot + 1 == STAGES ? 0 : slot + 1; }
    __device__ __forceinline__ int slot_behind() const { return slot == 0 ? STAGES - 1 : slot - 1; }
};

// ------------------------------------------------------------------- host --

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;

// CASE(E, threads) of the first shape that holds a.cols; a warp's rows come in steps
// of 256 columns, longer ones in steps of 1024 and, past 8192, of 4096.
#define LINEAR_ROW_SHAPES(CASE)          \
    switch ((a.cols + 255) / 256) {      \
        case 1: CASE(8, 32);             \
        case 2: CASE(16, 32);            \
        case 3: CASE(24, 32);            \
        case 4: CASE(32, 32);            \
    }                                    \
    switch ((a.cols + 1023) / 1024) {    \
        case 2: CASE(kEach, 64);         \
        case 3: CASE(kEach, 96);         \
        case 4: CASE(kEach, 128);        \
        case 5: CASE(kEach, 160);        \
        case 6: CASE(kEach, 192);        \
        case 7: CASE(kEach, 224);        \
        case 8: CASE(kEach, 256);        \
        case 9:                          \
        case 10:                         \
        case 11:                         \
        case 12: CASE(kEach, 384);       \
        case 13:                         \
        case 14:                         \
        case 15:                         \
        case 16: CASE(kEach, 512);       \
    }

inline int grid_of(int64_t rows, int per_cta, int ctas) {
    const int64_t groups = (rows + per_cta - 1) / per_cta;
    return static_cast<int>(groups < ctas ? groups : ctas);
}

// The element type and the weights' as template arguments.
#define LINEAR_BY_TYPE(type, weight_type, FN, ...)                                                              \
    ((type) == LINEAR_F32 ? FN<float, float>(__VA_ARGS__)                                                       \
     : (type) == LINEAR_F16                                                                                     \
         ? ((weight_type) == LINEAR_F32 ? FN<__half, float>(__VA_ARGS__) : FN<__half, __half>(__VA_ARGS__))     \
         : ((weight_type) == LINEAR_F32 ? FN<__nv_bfloat16, float>(__VA_ARGS__)                                 \
                                        : FN<__nv_bfloat16, __nv_bfloat16>(__VA_ARGS__)))

inline bool sizes_ok(int64_t rows, int64_t cols) { return rows >= 0 && cols >= 1; }

}  // namespace linear_ops
