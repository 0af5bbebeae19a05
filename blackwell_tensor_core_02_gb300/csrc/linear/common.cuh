// common.cuh -- what the kernels of the linear layer's operators share: element
// types, vector loads and stores, reductions over the threads of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../ptx.cuh"
#include "linear_ops.h"

namespace linear_ops {

namespace ptx = gemm_f16::ptx;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// One rounding, to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
    return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// VEC elements as they lie in memory: one 16-byte unit, or one element where
// rows are not aligned to that.
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Pack {
    T v[VEC];
};

// Elements of a 16-byte unit.
template <typename T>
constexpr int kUnit = 16 / static_cast<int>(sizeof(T));

// Two values to and from the 32-bit words that hold them (two for fp32), one
// rounding each.  Words, not the 16-bit pair classes: arrays of those are copied
// one by one, and a 16-byte store becomes four.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
    static constexpr int WORDS = 2;
    static __device__ __forceinline__ float2 widen(const uint32_t *w) {
        return make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    }
    static __device__ __forceinline__ void narrow(float2 v, uint32_t *w) {
        w[0] = __float_as_uint(v.x);
        w[1] = __float_as_uint(v.y);
    }
};
template <>
struct Pair<__half> {
    static constexpr int WORDS = 1;
    static __device__ __forceinline__ float2 widen(const uint32_t *w) {
        return __half22float2(*reinterpret_cast<const __half2 *>(w));
    }
    static __device__ __forceinline__ void narrow(float2 v, uint32_t *w) {
        const __half2 h = __floats2half2_rn(v.x, v.y);
        *w = *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Pair<__nv_bfloat16> {
    static constexpr int WORDS = 1;
    static __device__ __forceinline__ float2 widen(const uint32_t *w) {
        return make_float2(__uint_as_float(*w << 16), __uint_as_float(*w & 0xffff0000u));
    }
    static __device__ __forceinline__ void narrow(float2 v, uint32_t *w) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        *w = *reinterpret_cast<const uint32_t *>(&h);
    }
};

// N pairs from and to consecutive memory in 16-byte units (N pairs fill whole ones).
template <typename T, int N>
__device__ __forceinline__ void load_pairs(const T *p, float2 *v) {
    constexpr int kWords = N * Pair<T>::WORDS;
    static_assert(kWords % 4 == 0, "whole units");
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
        const uint4 u = *(reinterpret_cast<const uint4 *>(p) + i / 4);
        w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = Pair<T>::widen(w + i * Pair<T>::WORDS);
}
template <typename T, int N>
__device__ __forceinline__ void store_pairs(T *p, const float2 *v) {
    constexpr int kWords = N * Pair<T>::WORDS;
    static_assert(kWords % 4 == 0, "whole units");
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < N; ++i) Pair<T>::narrow(v[i], w + i * Pair<T>::WORDS);
#pragma unroll
    for (int i = 0; i < kWords; i += 4) {
        *(reinterpret_cast<uint4 *>(p) + i / 4) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

// 16 bytes that are read once: they leave the L1 cache to what is read again.
__device__ __forceinline__ uint4 load_unit(const void *p) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p)
                 : "memory");
    return u;
}

// 32 bytes at a 32-byte boundary: one access fills whole sectors.
__device__ __forceinline__ void load_32(const void *p, uint32_t (&w)[8]) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store_32(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// OUT words from `bytes` (0 to 16) on in a run, zeros past it.  All threads of a row
// shift alike, so this branches on the words: with selects in its place 4096 x 4099
// fp16 takes 12.4 us to mx and 12.8 back, so 11.2 and 11.5.
template <int FROM, int OUT, int IN>
__device__ __forceinline__ void shift_from(const uint32_t (&in)[IN], uint32_t bits, uint32_t (&out)[OUT]) {
#pragma unroll
    for (int i = 0; i < OUT; ++i) {
        const int k = i + FROM;
        out[i] = __funnelshift_r(k < IN ? in[k < IN ? k : 0] : 0u, k + 1 < IN ? in[k + 1 < IN ? k + 1 : 0] : 0u, bits);
    }
}
template <int OUT, int IN>
__device__ __forceinline__ void shift_words(const uint32_t (&in)[IN], uint32_t bytes, uint32_t (&out)[OUT]) {
    const uint32_t bits = (bytes & 3u) * 8u;
    switch (bytes / 4) {
        case 0: return shift_from<0>(in, bits, out);
        case 1: return shift_from<1>(in, bits, out);
        case 2: return shift_from<2>(in, bits, out);
        case 3: return shift_from<3>(in, bits, out);
        default: return shift_from<4>(in, bits, out);
    }
}

// W words of a row of T that starts anywhere, from `p` on, of which `left` elements
// are the row's (the others come as zeros): by the aligned 16-byte units that hold
// them.  The first may start before p; it shares an aligned 16 bytes with *p, so
// its allocation.  The last may go past the row's end, but not past the matrix's,
// `all` elements from p on: that one unit is read by elements.
template <typename T, int W>
__device__ __forceinline__ void load_shifted(const T *p, int left, int64_t all, uint32_t (&w)[W]) {
    constexpr int U = kUnit<T>, kElements = W * 4 / static_cast<int>(sizeof(T));
    const uint32_t head = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) % 16);
    const T *from = p - head / sizeof(T);
    const int end = left + static_cast<int>(head / sizeof(T));  // of the row, from `from` on
    const int64_t last = all + static_cast<int64_t>(head / sizeof(T));
    uint32_t raw[W + 4];
#pragma unroll
    for (int i = 0; i < W + 4; i += 4) {
        const int first = i / 4 * U;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (left > 0 && first < end && first + U <= last) {
            if (first < kElements || head > 0) u = *reinterpret_cast<const uint4 *>(from + first);
        } else if (left > 0 && first < end) {
            uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (first + j < end && (i > 0 || j * sizeof(T) >= head)) {
                    if constexpr (sizeof(T) == 4) {
                        e[j] = reinterpret_cast<const uint32_t *>(from)[first + j];
                    } else {
                        e[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(from)[first + j]) << (j % 2 * 16);
                    }
                }
            }
            u = make_uint4(e[0], e[1], e[2], e[3]);
        }
        raw[i] = u.x, raw[i + 1] = u.y, raw[i + 2] = u.z, raw[i + 3] = u.w;
    }
    shift_words(raw, head, w);
    if (left < kElements) {
        constexpr int kPer = 4 / static_cast<int>(sizeof(T));  // elements of a word
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i * kPer >= left) w[i] = 0u;
            if (kPer == 2 && i * kPer + 1 >= left) w[i] &= 0xffffu;
        }
    }
}

// The other way: a thread's run of W words of a row of T, `valid` elements of it
// the row's, to `p`, anywhere.  w: the four words before the run, then the run.
// The 16-byte unit that the run shares with the one before belongs to this thread
// if `before` (w then has that run's end), and the one it shares with the next run
// to that one's thread if `after`; else each stores its own elements of it, in
// aligned words of 8, 4 and 2 bytes (values of 5461 x 375: 3.4 us, element by
// element 4.2).
template <typename T, int N>
__device__ __forceinline__ void store_shifted(T *p, int valid, bool before, bool after, const uint32_t (&w)[N]) {
    constexpr int W = N - 4, U = kUnit<T>;
    const uint32_t head = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) % 16);
    const int skip = static_cast<int>(head / sizeof(T));  // elements of the first unit before p
    T *to = p - skip;
    uint32_t out[W + 4];  // the words of the aligned units
    shift_words(w, 16u - head, out);
    const int start = before ? 0 : skip, end = skip + valid;
#pragma unroll
    for (int i = 0; i < W + 4; i += 4) {
        const int at = i / 4 * U;
        if (at >= start && at + U <= end) {
            *reinterpret_cast<uint4 *>(to + at) = make_uint4(out[i], out[i + 1], out[i + 2], out[i + 3]);
        }
    }
    const int tail = end / U * U;  // of the last unit, if it is not whole
    if (start > 0 && end < U) {
        // the first unit and the last: [start, end) of it
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (j < start || j >= end) continue;
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<uint32_t *>(to)[j] = out[j];
            } else {
                reinterpret_cast<uint16_t *>(to)[j] = static_cast<uint16_t>(out[j / 2] >> (j % 2 * 16));
            }
        }
        return;
    }
    if (start > 0) {
        if constexpr (sizeof(T) == 4) {
            if (start & 1) reinterpret_cast<uint32_t *>(to)[start] = start == 1 ? out[1] : out[3];
            if (start <= 2) *reinterpret_cast<uint2 *>(to + 2) = make_uint2(out[2], out[3]);
        } else {
            const int even = start + (start & 1);
            const uint32_t low = start & 2 ? out[1] : out[0], high = start & 2 ? out[3] : out[2];
            if (start & 1) reinterpret_cast<uint16_t *>(to)[start] = static_cast<uint16_t>((start & 4 ? high : low) >> 16);
            if (even & 2) *reinterpret_cast<uint32_t *>(to + even) = even & 4 ? out[3] : out[1];
            if (start <= 4) *reinterpret_cast<uint2 *>(to + 4) = make_uint2(out[2], out[3]);
        }
    }
    if (tail < end && !after) {
        uint32_t t[4] = {out[0], out[1], out[2], out[3]};
#pragma unroll
        for (int i = 4; i < W + 4; i += 4) {
            if (tail == i / 4 * U) t[0] = out[i], t[1] = out[i + 1], t[2] = out[i + 2], t[3] = out[i + 3];
        }
        const int n = end - tail;
        T *d = to + tail;
        if constexpr (sizeof(T) == 4) {
            if (n & 2) *reinterpret_cast<uint2 *>(d) = make_uint2(t[0], t[1]);
            if (n & 1) *reinterpret_cast<uint32_t *>(d + (n & 2)) = n & 2 ? t[2] : t[0];
        } else {
            const uint32_t low = n & 2 ? t[1] : t[0], high = n & 2 ? t[3] : t[2];
            if (n & 4) *reinterpret_cast<uint2 *>(d) = make_uint2(t[0], t[1]);
            if (n & 2) *reinterpret_cast<uint32_t *>(d + (n & 4)) = n & 4 ? t[2] : t[0];
            if (n & 1) *reinterpret_cast<uint16_t *>(d + (n & 6)) = static_cast<uint16_t>(n & 4 ? high : low);
        }
    }
}

// Two fp32 values in one 64-bit register pair: Blackwell adds, multiplies and
// fuses both in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
          "l"(reinterpret_cast<uint64_t &>(c)));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// N sums over the TPR threads of one row (threadIdx.x; whole warps), every
// thread getting them, in a fixed order.  ROWS rows (threadIdx.y) share the CTA
// and each has a barrier of its own; `slot` is this row's own N * 32 floats of
// shared memory, 16-byte aligned.  A second call on the same slot needs a call
// on another slot, or a barrier, between.
template <int TPR, int ROWS>
__device__ __forceinline__ void row_barrier() {
    if constexpr (TPR == 32) {
        __syncwarp();
    } else if constexpr (ROWS == 1) {
        __syncthreads();
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1u), "n"(TPR) : "memory");
    }
}

template <int N, int TPR, int ROWS>
__device__ __forceinline__ void row_sum(float (&v)[N], float *slot) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    constexpr int kWarps = TPR / 32;
    if constexpr (kWarps > 1) {
        const int warp = static_cast<int>(threadIdx.x) / 32;
        if (threadIdx.x % 32 == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) slot[i * 32 + warp] = v[i];
        }
        row_barrier<TPR, ROWS>();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            constexpr int kPer = kWarps % 4 == 0 ? 4 : (kWarps % 2 == 0 ? 2 : 1);
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w += kPer) {
                const Pack<float, kPer> p = *reinterpret_cast<const Pack<float, kPer> *>(slot + i * 32 + w);
#pragma unroll
                for (int j = 0; j < kPer; ++j) t += p.v[j];
            }
            v[i] = t;
        }
    }
}

// 16 bytes of global memory on their way to shared memory; or `bytes` of them, the
// rest zeroed.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------- host --

inline bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline bool overlap(const void *p, int64_t p_bytes, const void *q, int64_t q_bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && p_bytes > 0 && q_bytes > 0 && a < b + static_cast<uintptr_t>(q_bytes) &&
           b < a + static_cast<uintptr_t>(p_bytes);
}

inline int64_t type_size(int32_t type) { return type == LINEAR_F32 ? 4 : 2; }

inline bool type_ok(int32_t type) { return type >= LINEAR_F16 && type <= LINEAR_F32; }

// Bytes from the first to the last element of rows x cols at that stride.
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t stride, int64_t size) {
    return rows <= 0 || cols <= 0 ? 0 : ((rows - 1) * stride + cols) * size;
}

// Whether rows of `bytes` bytes, `stride` bytes apart, share memory between p and q.
// Rows of one stride may lie between each other's (two slices of a wider matrix).
inline bool rows_overlap(const void *p, const void *q, int64_t rows, int64_t bytes, int64_t p_stride, int64_t q_stride) {
    if (!overlap(p, span_bytes(rows, bytes, p_stride, 1), q, span_bytes(rows, bytes, q_stride, 1))) return false;
    if (p_stride != q_stride || p_stride < bytes) return true;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const int64_t apart = static_cast<int64_t>((a < b ? b - a : a - b) % static_cast<uintptr_t>(p_stride));
    return apart < bytes || p_stride - apart < bytes;
}

// The current device is a GB300 (checked once per device); its SM count.
int gb300_sms(int *sms);

constexpr int kMaxDevices = 64;

// The kernel's dynamic shared memory, allowed once per device.
template <typename K>
inline bool allow_smem(K *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
    const uint64_t bit = uint64_t(1) << dev;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// A grid of CTAs that may start while the previous kernel of the stream ends
// (every kernel here waits for it, griddepcontrol.wait, before its first
// access to memory that another kernel may write).
template <typename... P, typename... A>
inline int launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace linear_ops
