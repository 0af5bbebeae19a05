// fp4_quantize.cu -- microscaled 4-bit floats: from and to ordinary ones (see
// linear_ops.h).
//
// Bound by memory: 2 or 4 bytes an element on one side, 0.53 to 0.56 on the
// other, which at 16 bits an element leaves some ten instructions for each.  A
// thread owns a unit of 16 consecutive elements of a row, which is a block of
// FP4_NV and half of one of FP4_MX, and 8 bytes of data; a scale word (4 blocks
// of a row) is gathered from 4 or 8 lanes and stored once.
#include "common.cuh"
#include "fp4.cuh"

namespace linear_ops {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
constexpr int kThreads = 256;

// 8 pairs of floats to E2M1, to nearest with ties to the even code, magnitudes past 6
// to 6: element 2i in the low nibble of byte i.
__device__ __forceinline__ uint2 to_e2m1(const float2 (&v)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 *f = v + 4 * i;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(w[i])
            : "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y));
    }
    return make_uint2(w[0], w[1]);
}

// The 4 pairs of values of 4 bytes of E2M1 codes.
__device__ __forceinline__ void from_e2m1(uint32_t w, float2 *v) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
}

// E4M3 code of t (finite, 0 <= t <= 448), to nearest even.
__device__ __forceinline__ uint32_t to_e4m3(float t) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(t));
    return r & 0xffu;
}

__device__ __forceinline__ float from_e4m3(uint32_t code) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
    return __low2float(*reinterpret_cast<const __half2 *>(&h));
}

// 2^(code - 127); NaN for 255.
__device__ __forceinline__ float from_e8m0(uint32_t code) {
    return __uint_as_float(code == 255u ? 0x7fffffffu : (code == 0u ? 0x00400000u : code << 23));
}

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// A row's units along threadIdx.x (8 to 256 of them, so a scale word's lanes are
// neighbours) and blockIdx.y, rows along threadIdx.y and blockIdx.x.
struct Grid {
    dim3 grid, block;
};

Grid grid_for(int64_t rows, int64_t units) {
    int x = 8;
    while (x < kThreads && x < units) x *= 2;
    const int y = kThreads / x;
    const int64_t chunks = (units + x - 1) / x;
    return {dim3(static_cast<unsigned>((rows + y - 1) / y), static_cast<unsigned>(chunks < 65535 ? chunks : 65535)),
            dim3(x, y)};
}

// The 16 elements of each lane's unit, where rows start anywhere: the lanes of a
// row read its elements one after the other and meet in shared memory.
// `group`: lanes of a row in the warp; `seg`: their elements, from the first of
// lane 0's unit on; `left`: how many there are.
template <typename T>
__device__ __forceinline__ void read_scattered(const T *seg, int left, int group, T *stage, float (&v)[16]) {
    const int lane = static_cast<int>(threadIdx.x) % group;
    T *own = stage + ((threadIdx.y * blockDim.x + threadIdx.x) % 32 - lane) * 16;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int e = i * group + lane;
        own[e] = e < left ? seg[e] : from_f32<T>(0.f);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; i += kUnit<T>) {
        const Pack<T, kUnit<T>> p = *reinterpret_cast<const Pack<T, kUnit<T>> *>(own + lane * 16 + i);
#pragma unroll
        for (int j = 0; j < kUnit<T>; ++j) v[i + j] = to_f32(p.v[j]);
    }
    __syncwarp();
}

struct QuantArgs {
    const void *x;
    uint8_t *data, *scales;
    int64_t x_stride;
    int32_t rows, cols;
    int32_t units, data_units;  // units of a row: with the scale tiles' rest, and of data
    int32_t tiles;              // scale tiles along a row
    int32_t exponent;
};

template <typename T, bool NV, bool WIDE>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantArgs a) {
    __shared__ __align__(16) T stage[WIDE ? 1 : kThreads * 16];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool inside = row < a.rows;
    const T *x = static_cast<const T *>(a.x) + (inside ? row : 0) * a.x_stride;
    const bool padded = row < (static_cast<int64_t>(a.rows) + kScaleTileRows - 1) / kScaleTileRows * kScaleTileRows;
    ptx::griddep_wait();
    for (int base = static_cast<int>(blockIdx.y * blockDim.x); base < a.units; base += static_cast<int>(gridDim.y * blockDim.x)) {
        // units is a multiple of 4 (FP4_NV) or 8: the lanes of a scale word agree on `live`
        const int unit = base + static_cast<int>(threadIdx.x), col = unit * 16;
        const bool live = padded && unit < a.units;
        float v[16];
        if constexpr (WIDE) {
            constexpr int U = kUnit<T>;
            uint4 raw[16 / U];
#pragma unroll
            for (int i = 0; i < 16 / U; ++i) {
                raw[i] = make_uint4(0, 0, 0, 0);
                if (inside && col + i * U < a.cols) raw[i] = load_unit(x + col + i * U);
            }
#pragma unroll
            for (int i = 0; i < 16 / U; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int j = 0; j < U / 2; ++j) {
                    const float2 f = Pair<T>::widen(w + j * Pair<T>::WORDS);
                    v[i * U + 2 * j] = f.x;
                    v[i * U + 2 * j + 1] = f.y;
                }
            }
        } else {
            const int group = blockDim.x < 32 ? static_cast<int>(blockDim.x) : 32;
            const int first = (unit - unit % group) * 16;
            read_scattered<T>(x + first, inside ? a.cols - first : 0, group,
                              stage + (threadIdx.y * blockDim.x + threadIdx.x) / 32 * 512, v);
        }
        // the largest magnitude as bits: they order like the values, and an infinity or
        // NaN is above every finite one
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
        if constexpr (!NV) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const bool bad = amax >= 0x7f800000u;
        uint32_t code;
        float2 q[8];
        if constexpr (NV) {
            // A quotient has to be rounded as a quotient, ties included.  With a reciprocal
            // i of s within an ulp, q = x * i is off by a few ulps; one step with the exact
            // remainder x - q * s leaves an error far below half an ulp before its rounding.
            // That gives a quotient that is a tie of E2M1 (or E4M3; they have few bits)
            // exactly, and no other quotient of fp32 numbers lies within half an ulp of one.
            const float m = __uint_as_float(amax);
            constexpr float sixth = 1.f / 6.f;
            const float t0 = m * sixth, t = fmaf(fmaf(-t0, 6.f, m), sixth, t0) * pow2(-a.exponent);
            code = to_e4m3(fminf(fmaxf(t, 0x1p-9f), 448.f));
            const float s = from_e4m3(code) * pow2(a.exponent);
            float inv;
            asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 xi = make_float2(v[2 * i], v[2 * i + 1]), q0 = mul2(xi, both(inv));
                q[i] = fma2(fma2(q0, both(-s), xi), both(inv), q0);
            }
            if (m > 8.f * s) {
                // the scale ended at its largest: quotients may overflow, and their
                // remainders with them, but past 8 the code is 6 either way
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (fabsf(v[2 * i] * inv) >= 8.f) q[i].x = copysignf(8.f, v[2 * i]);
                    if (fabsf(v[2 * i + 1] * inv) >= 8.f) q[i].y = copysignf(8.f, v[2 * i + 1]);
                }
            }
            if (bad) code = 0x7fu;
        } else {
            const uint32_t e = amax >> 23;  // floor(log2(amax)) + 127; 0 for zeros and subnormal values
            code = e > 2u ? e - 2u : 0u;
            const float inv = pow2(127 - static_cast<int>(code));  // code <= 252: 2^-125 .. 2^127
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = mul2(make_float2(v[2 * i], v[2 * i + 1]), both(inv));
            if (bad) code = 0xffu;
        }
        uint2 packed = to_e2m1(q);
        if (bad) packed = make_uint2(0u, 0u);
        if (inside && unit < a.data_units) {
            *reinterpret_cast<uint2 *>(a.data + (row * a.data_units + unit) * 8) = packed;
        }
        // rows and blocks past the matrix have scale 0
        if (!inside || unit >= a.data_units) code = 0u;
        if constexpr (NV) {
            uint32_t word = code | (__shfl_down_sync(0xffffffffu, code, 1) << 8);
            word |= __shfl_down_sync(0xffffffffu, word, 2) << 16;
            if (live && unit % 4 == 0) *reinterpret_cast<uint32_t *>(a.scales + fp4_scale_at(row, unit, a.tiles)) = word;
        } else {
            uint32_t word = code | (__shfl_down_sync(0xffffffffu, code, 2) << 8);
            word |= __shfl_down_sync(0xffffffffu, word, 4) << 16;
            if (live && unit % 8 == 0) {
                *reinterpret_cast<uint32_t *>(a.scales + fp4_scale_at(row, unit / 2, a.tiles)) = word;
            }
        }
    }
}

struct DequantArgs {
    const uint8_t *data, *scales;
    void *out;
    int64_t out_stride;
    int32_t rows, cols, data_units, tiles, exponent;
};

template <typename T, bool NV, bool WIDE>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantArgs a) {
    __shared__ __align__(16) T stage[WIDE ? 1 : kThreads * 16];
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool inside = row < a.rows;
    ptx::griddep_wait();
    for (int base = static_cast<int>(blockIdx.y * blockDim.x); base < a.data_units;
         base += static_cast<int>(gridDim.y * blockDim.x)) {
        const int unit = base + static_cast<int>(threadIdx.x), col = unit * 16;
        const bool live = inside && unit < a.data_units;
        uint2 packed = make_uint2(0u, 0u);
        uint32_t code = 0;
        if (live) {
            packed = *reinterpret_cast<const uint2 *>(a.data + (row * a.data_units + unit) * 8);
            code = a.scales[fp4_scale_at(row, NV ? unit : unit / 2, a.tiles)];
        }
        const float s = NV ? from_e4m3(code) * pow2(a.exponent) : from_e8m0(code);
        float2 v[8];
        from_e2m1(packed.x, v);
        from_e2m1(packed.y, v + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = mul2(v[i], both(s));
        T *out = static_cast<T *>(a.out) + row * a.out_stride;
        if constexpr (WIDE) {
            constexpr int U = kUnit<T>;
#pragma unroll
            for (int i = 0; i < 16 / U; ++i) {
                if (live && col + i * U < a.cols) store_pairs<T, U / 2>(out + col + i * U, v + i * U / 2);
            }
        } else {
            // rows start anywhere: through shared memory, one element a lane after the other
            const int group = blockDim.x < 32 ? static_cast<int>(blockDim.x) : 32, lane = static_cast<int>(threadIdx.x) % group;
            const int thread = static_cast<int>(threadIdx.y * blockDim.x + threadIdx.x);
            T *own = stage + (thread - lane) * 16;
            store_pairs<T, 8>(own + lane * 16, v);
            __syncwarp();
            const int first = (unit - lane) * 16;
            if (inside) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int e = i * group + lane;
                    if (first + e < a.cols) out[first + e] = own[e];
                }
            }
            __syncwarp();
        }
    }
}

template <typename T>
int quantize_as(const QuantArgs &a, bool nv, cudaStream_t stream) {
    const bool wide = a.cols % kUnit<T> == 0 && a.x_stride % kUnit<T> == 0 && aligned(a.x, 16);
    const Grid g = grid_for((static_cast<int64_t>(a.rows) + kScaleTileRows - 1) / kScaleTileRows * kScaleTileRows, a.units);
    if (nv) {
        return wide ? launch(quantize_kernel<T, true, true>, g.grid, g.block, 0, stream, a)
                    : launch(quantize_kernel<T, true, false>, g.grid, g.block, 0, stream, a);
    }
    return wide ? launch(quantize_kernel<T, false, true>, g.grid, g.block, 0, stream, a)
                : launch(quantize_kernel<T, false, false>, g.grid, g.block, 0, stream, a);
}

template <typename T>
int dequantize_as(const DequantArgs &a, bool nv, cudaStream_t stream) {
    const bool wide = a.cols % kUnit<T> == 0 && a.out_stride % kUnit<T> == 0 && aligned(a.out, 16);
    const Grid g = grid_for(a.rows, a.data_units);
    if (nv) {
        return wide ? launch(dequantize_kernel<T, true, true>, g.grid, g.block, 0, stream, a)
                    : launch(dequantize_kernel<T, true, false>, g.grid, g.block, 0, stream, a);
    }
    return wide ? launch(dequantize_kernel<T, false, true>, g.grid, g.block, 0, stream, a)
                : launch(dequantize_kernel<T, false, false>, g.grid, g.block, 0, stream, a);
}

int check_matrix(int64_t rows, int64_t cols, int32_t format, int32_t exponent) {
    if (rows < 0 || cols < 0 || (format != FP4_MX && format != FP4_NV) || exponent < -100 || exponent > 100 ||
        (format == FP4_MX && exponent != 0)) {
        return GEMM_ERR_INVALID_ARG;
    }
    return rows > kMaxDim || cols > kMaxDim ? GEMM_ERR_UNSUPPORTED_SHAPE : GEMM_OK;
}

}  // namespace
}  // namespace linear_ops

using namespace linear_ops;

extern "C" {

int64_t fp4_data_bytes(int64_t rows, int64_t cols) {
    const int st = check_matrix(rows, cols, FP4_MX, 0);
    return st != GEMM_OK ? st : rows * (fp4_padded_cols(cols) / 2);
}

int64_t fp4_scale_bytes(int64_t rows, int64_t cols, int32_t format) {
    const int st = check_matrix(rows, cols, format, 0);
    return st != GEMM_OK ? st
                         : (rows + kScaleTileRows - 1) / kScaleTileRows * fp4_scale_tiles(cols, format == FP4_NV) *
                               kScaleTileBytes;
}

int fp4_quantize(const void *x, int64_t x_stride, int64_t rows, int64_t cols, int32_t type, int32_t format,
                 int32_t exponent, void *data, void *scales, void *stream) {
    if (!type_ok(type) || x_stride < 0) return GEMM_ERR_INVALID_ARG;
    int st = check_matrix(rows, cols, format, exponent);
    if (st != GEMM_OK || rows == 0 || cols == 0) return st;
    if (!x || !data || !scales) return GEMM_ERR_INVALID_ARG;
    if (!aligned(x, type_size(type)) || !aligned(data, 16) || !aligned(scales, 16)) return GEMM_ERR_MISALIGNED;
    const bool nv = format == FP4_NV;
    if (rows == 1) x_stride = 0;
    const int64_t x_bytes = span_bytes(rows, cols, x_stride, type_size(type));
    const int64_t data_bytes = fp4_data_bytes(rows, cols), scale_bytes = fp4_scale_bytes(rows, cols, format);
    if (overlap(data, data_bytes, x, x_bytes) || overlap(scales, scale_bytes, x, x_bytes) ||
        overlap(data, data_bytes, scales, scale_bytes)) {
        return GEMM_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    QuantArgs a = {};
    a.x = x;
    a.data = static_cast<uint8_t *>(data);
    a.scales = static_cast<uint8_t *>(scales);
    a.x_stride = x_stride;
    a.rows = static_cast<int32_t>(rows);
    a.cols = static_cast<int32_t>(cols);
    a.tiles = static_cast<int32_t>(fp4_scale_tiles(cols, nv));
    a.units = a.tiles * (nv ? 4 : 8);
    a.data_units = static_cast<int32_t>(fp4_padded_cols(cols) / 16);
    a.exponent = exponent;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return type == LINEAR_F16    ? quantize_as<__half>(a, nv, s)
           : type == LINEAR_BF16 ? quantize_as<__nv_bfloat16>(a, nv, s)
                                 : quantize_as<float>(a, nv, s);
}

int fp4_dequantize(const void *data, const void *scales, int64_t rows, int64_t cols, int32_t format, int32_t exponent,
                   void *out, int64_t out_stride, int32_t type, void *stream) {
    if (!type_ok(type)) return GEMM_ERR_INVALID_ARG;
    int st = check_matrix(rows, cols, format, exponent);
    if (st != GEMM_OK || rows == 0 || cols == 0) return st;
    if (!data || !scales || !out || (rows > 1 && out_stride < cols)) return GEMM_ERR_INVALID_ARG;
    if (!aligned(out, type_size(type)) || !aligned(data, 16) || !aligned(scales, 16)) return GEMM_ERR_MISALIGNED;
    if (rows == 1) out_stride = 0;
    const int64_t out_bytes = span_bytes(rows, cols, out_stride, type_size(type));
    if (overlap(out, out_bytes, data, fp4_data_bytes(rows, cols)) ||
        overlap(out, out_bytes, scales, fp4_scale_bytes(rows, cols, format))) {
        return GEMM_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = gb300_sms(&sms);
    if (st != GEMM_OK) return st;
    DequantArgs a = {};
    a.data = static_cast<const uint8_t *>(data);
    a.scales = static_cast<const uint8_t *>(scales);
    a.out = out;
    a.out_stride = out_stride;
    a.cols = static_cast<int32_t>(cols);
    a.data_units = static_cast<int32_t>(fp4_padded_cols(cols) / 16);
    a.tiles = static_cast<int32_t>(fp4_scale_tiles(cols, format == FP4_NV));
    a.rows = static_cast<int32_t>(rows);
    a.exponent = exponent;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool nv = format == FP4_NV;
    return type == LINEAR_F16    ? dequantize_as<__half>(a, nv, s)
           : type == LINEAR_BF16 ? dequantize_as<__nv_bfloat16>(a, nv, s)
                                 : dequantize_as<float>(a, nv, s);
}

}  // extern "C"
