// common.cuh -- what the kernels of the linear layer's operators share: element
// types, vector loads and stores, reductions over the threads of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

// A load of data that is read once: it leaves the L1 cache to what is read
// again (the weights, which every row reads).
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_once(const T *p) {
    Pack<T, VEC> r;
    if constexpr (VEC * sizeof(T) == 16) {
        uint4 u;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(p)
                     : "memory");
        *reinterpret_cast<uint4 *>(&r) = u;
    } else {
        r = *reinterpret_cast<const Pack<T, VEC> *>(p);
    }
    return r;
}

template <typename T, int VEC>
__device__ __forceinline__ void load_f32(const T *p, float (&out)[VEC]) {
    // VEC elements of T may be two 16-byte units (fp32 weights beside 16-bit rows)
    constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
    constexpr int kPer = kBytes > 16 ? kUnit<T> : VEC;
#pragma unroll
    for (int i = 0; i < VEC / kPer; ++i) {
        const Pack<T, kPer> u = *reinterpret_cast<const Pack<T, kPer> *>(p + i * kPer);
#pragma unroll
        for (int j = 0; j < kPer; ++j) out[i * kPer + j] = to_f32(u.v[j]);
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_f32(T *p, const float (&in)[VEC]) {
    constexpr int kBytes = VEC * static_cast<int>(sizeof(T));
    constexpr int kPer = kBytes > 16 ? kUnit<T> : VEC;
#pragma unroll
    for (int i = 0; i < VEC / kPer; ++i) {
        Pack<T, kPer> u;
#pragma unroll
        for (int j = 0; j < kPer; ++j) u.v[j] = from_f32<T>(in[i * kPer + j]);
        *reinterpret_cast<Pack<T, kPer> *>(p + i * kPer) = u;
    }
}

// N sums over the threads of one row, every thread getting them.  The row's
// threads are the x dimension of the CTA (a power of two of at least 32, whole
// warps); `slot` is this row's own N * 32 floats of shared memory.  The order
// of the additions is fixed.  Rows that share a CTA call it together (it holds
// CTA barriers when a row has several warps); a second call on the same slot
// needs other shared memory or a barrier between.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float *slot) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    const int warps = static_cast<int>(blockDim.x) / 32;
    if (warps == 1) return;
    const int warp = static_cast<int>(threadIdx.x) / 32, lane = static_cast<int>(threadIdx.x) % 32;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) slot[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // a power of two of warps: lanes beyond repeat the first ones' values
        float t = slot[i * 32 + (lane & (warps - 1))];
        for (int o = warps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        v[i] = t;
    }
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

// The current device is a GB300 (checked once per device); its SM count.
int gb300_sms(int *sms);

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
