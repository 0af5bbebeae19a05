// norm_parts.cuh -- the weights' gradient of a norm: sums over some rows, left as parts
// by the CTAs that had the rows, and the kernel that joins them.
#pragma once

#include "common.cuh"

namespace linear_ops {
namespace {

// Parts of the weights' gradient: a CTA for each of 152 SMs.
constexpr int kMaxParts = 152;

// Floats of a part's dweight, and of its dbias: whole 16-byte units.
__host__ __device__ constexpr int64_t part_stride(int64_t cols) { return (cols + 3) / 4 * 4; }

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

}  // namespace
}  // namespace linear_ops
