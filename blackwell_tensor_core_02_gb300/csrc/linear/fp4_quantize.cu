// fp4_quantize.cu -- microscaled 4-bit floats: from and to ordinary ones (see
// linear_ops.h).
//
// Bound by memory: 2 or 4 bytes an element on one side, 0.53 to 0.56 on the
// other, which at 16 bits an element leaves some ten instructions for each.  A
// thread owns a unit of 16 consecutive elements of a row, which is a block of
// FP4_NV and half of one of FP4_MX, and 8 bytes of data; a scale word (4 blocks
// of a row) is gathered from 4 or 8 lanes and stored once.
//
// 8192 x 4096 (share of the copy rate): fp16 to mx 15.7 us (80 %, with two thirds of
// the issue slots taken), bf16 to nv 17.5 (72 %), fp32 to mx 23.1 (97 %), back to bf16
// 13.7 (91 %).  Rows that start anywhere: 4096 x 4099 fp16 to mx 11.2 us (56 %), back
// 11.5.  One row of 8192: 2.0 us and 1.1.
#include "common.cuh"
#include "fp4.cuh"

namespace linear_ops {
namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;
constexpr int kThreads = 256;
// Columns that a grid's 65535 chunks of 256 units (grid_for, for wide rows) cover.
constexpr int64_t kMaxCols = int64_t(65535) * kThreads * 16;

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

// As many threads of a row as leave at most an eighth of them without a unit (of
// 257 units 256 threads would take two turns).
Grid grid_for(int64_t rows, int64_t units) {
    int x = kThreads;
    while (x > 8 && (units + x - 1) / x * x * 8 > units * 9) x /= 2;
    const int y = kThreads / x;
    const int64_t chunks = (units + x - 1) / x;
    return {dim3(static_cast<unsigned>((rows + y - 1) / y), static_cast<unsigned>(chunks)), dim3(x, y)};
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

// How rows lie in memory: elements anywhere, whole 16-byte units, or whole 16
// elements of which each 32 bytes are aligned (one access then fills sectors).
enum : int { kScattered = 0, kUnits = 1, kSectors = 2 };

// The largest magnitude of a thread's elements as fp32 bits.  Bits order like the
// magnitudes, and an infinity or NaN is above every finite one; 16-bit elements are
// compared two at a time.
template <typename T, int N>
__device__ __forceinline__ uint32_t largest(const uint32_t (&w)[N]) {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) m = max(m, w[i] & 0x7fffffffu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(m), "r"(w[i] & 0x7fff7fffu));
        m = max(m & 0xffffu, m >> 16);
        return __float_as_uint(Pair<T>::widen(&m).x);
    }
}

// FP4_NV, with the longer arithmetic, runs on a grid of the CTAs that fit at once: a
// thread takes rows a grid apart and loads its unit of the next row while it works
// on this one (8192 x 4096 bf16: 17.5 us, a CTA for each row 18.7; FP4_MX 15.6 and
// 15.4, so it takes a CTA for each row, and so do rows that start anywhere, whose
// loads take more registers).
template <typename T, bool NV, int LAYOUT>
constexpr bool kAhead = NV && LAYOUT != kScattered;
template <typename T, bool NV, int LAYOUT>
constexpr int kQuantizePerSm = kAhead<T, NV, LAYOUT> || sizeof(T) == 4 ? 4 : 5;

template <typename T, bool NV, int LAYOUT>
__global__ void __launch_bounds__(kThreads, kQuantizePerSm<T, NV, LAYOUT>) quantize_kernel(const QuantArgs a) {
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    const int64_t rows = (static_cast<int64_t>(a.rows) + kScaleTileRows - 1) / kScaleTileRows * kScaleTileRows;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    // units is a multiple of 4 (FP4_NV) or 8: the lanes of a scale word agree on `live`
    const int unit = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x), col = unit * 16;
    const bool live = unit < a.units;
    constexpr int W = 16 * sizeof(T) / 4;
    // this thread's unit of a row as it lies in memory, zeros past the matrix
    auto fetch = [&](int64_t row, uint32_t (&w)[W]) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
        if (row >= a.rows) return;
        const T *x = static_cast<const T *>(a.x) + row * a.x_stride + col;
        if constexpr (LAYOUT == kSectors) {
#pragma unroll
            for (int i = 0; i < W; i += 8) {
                if (col < a.cols) load_32(x + i * 4 / static_cast<int>(sizeof(T)), reinterpret_cast<uint32_t (&)[8]>(w[i]));
            }
        } else if constexpr (LAYOUT == kUnits) {
#pragma unroll
            for (int i = 0; i < W; i += 4) {
                const int c = i * 4 / static_cast<int>(sizeof(T));
                if (col + c < a.cols) {
                    const uint4 u = load_unit(x + c);
                    w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
                }
            }
        } else {
            load_shifted<T>(x, a.cols - col, (a.rows - 1 - row) * a.x_stride + a.cols - col, w);
        }
    };
    ptx::griddep_wait();
    uint32_t next[W];
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.y;  // whole CTAs take part in the shuffles
    if constexpr (kAhead<T, NV, LAYOUT>) fetch(first + threadIdx.y, next);
    for (int64_t base = first; base < rows; base += step) {
        const int64_t row = base + threadIdx.y;
        const bool inside = row < a.rows;
        uint32_t w[W];
        if constexpr (kAhead<T, NV, LAYOUT>) {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = next[i];
            if (base + step < rows) fetch(row + step, next);
        } else {
            fetch(row, w);
        }
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = Pair<T>::widen(w + i * Pair<T>::WORDS);
        uint32_t amax = largest<T>(w);
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
            // It is formed with its sign turned, which the codes then undo: for x = -0 every
            // step leaves the +0 that stands for -0 (x - q * s = +0, and +0 * -i + +0 = +0;
            // unturned the last step is +0 + -0, which loses the sign).
            const float m = __uint_as_float(amax);
            constexpr float sixth = 1.f / 6.f;
            const float t0 = m * sixth, t = fmaf(fmaf(-t0, 6.f, m), sixth, t0) * pow2(-a.exponent);
            code = to_e4m3(fminf(fmaxf(t, 0x1p-9f), 448.f));
            const float s = from_e4m3(code) * pow2(a.exponent);
            float inv;  // -i
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(-s));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 q0 = mul2(v[i], both(inv));
                q[i] = fma2(fma2(q0, both(s), v[i]), both(inv), q0);
            }
            if (!(m <= 8.f * s)) {
                // the scale ended at its largest: quotients may overflow, and their
                // remainders with them, but past 8 the code is 6 either way; an infinity or
                // NaN comes here too
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (fabsf(v[i].x * inv) >= 8.f) q[i].x = copysignf(8.f, -v[i].x);
                    if (fabsf(v[i].y * inv) >= 8.f) q[i].y = copysignf(8.f, -v[i].y);
                    if (bad) q[i] = both(-0.f);
                }
                if (bad) code = 0x7fu;
            }
        } else {
            const uint32_t e = amax >> 23;  // floor(log2(amax)) + 127; 0 for zeros and subnormal values
            code = e > 2u ? e - 2u : 0u;
            const float inv = pow2(127 - static_cast<int>(code));  // code <= 252: 2^-125 .. 2^127
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = mul2(v[i], both(inv));
            if (bad) code = 0xffu;
        }
        uint2 packed = to_e2m1(q);
        if constexpr (NV) {
            packed.x ^= 0x88888888u, packed.y ^= 0x88888888u;  // the signs turned back
        } else if (bad) {
            packed = make_uint2(0u, 0u);
        }
        if (inside && unit < a.data_units) {
            *reinterpret_cast<uint2 *>(a.data + (row * a.data_units + unit) * 8) = packed;
        }
        // rows and blocks past the matrix have scale 0
        if (!inside || unit >= a.data_units) code = 0u;
        if constexpr (NV) {
            uint32_t word = code | (__shfl_down_sync(0xffffffffu, code, 1) << 8);
            word |= __shfl_down_sync(0xffffffffu, word, 2) << 16;
            if (live && row < rows && unit % 4 == 0) {
                *reinterpret_cast<uint32_t *>(a.scales + fp4_scale_at(row, unit, a.tiles)) = word;
            }
        } else {
            uint32_t word = code | (__shfl_down_sync(0xffffffffu, code, 2) << 8);
            word |= __shfl_down_sync(0xffffffffu, word, 4) << 16;
            if (live && row < rows && unit % 8 == 0) {
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

template <typename T, bool NV, int LAYOUT>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const DequantArgs a) {
    if (threadIdx.x == 0 && threadIdx.y == 0) ptx::griddep_launch_dependents();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool inside = row < a.rows;
    ptx::griddep_wait();
    {
        const int unit = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x), col = unit * 16;
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
        if constexpr (LAYOUT == kSectors) {
            constexpr int P = Pair<T>::WORDS;
            uint32_t w[8 * P];
#pragma unroll
            for (int i = 0; i < 8; ++i) Pair<T>::narrow(v[i], w + i * P);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (live && col < a.cols) store_32(out + col + i * 8, reinterpret_cast<const uint32_t (&)[8]>(w[i * 8]));
            }
        } else if constexpr (LAYOUT == kUnits) {
            constexpr int U = kUnit<T>;
#pragma unroll
            for (int i = 0; i < 16 / U; ++i) {
                if (live && col + i * U < a.cols) store_pairs<T, U / 2>(out + col + i * U, v + i * U / 2);
            }
        } else {
            // Rows start anywhere: a lane's unit and the end of the lane before's give it the
            // aligned units of 16 bytes that begin in its unit or the one before; elements of
            // no whole one go by themselves.
            const int group = blockDim.x < 32 ? static_cast<int>(blockDim.x) : 32;  // lanes of this row
            const bool first = threadIdx.x % group == 0, final = threadIdx.x % group == group - 1;
            constexpr int P = Pair<T>::WORDS, W = 8 * P;
            uint32_t w[W + 4];  // four words of the lane before, then this lane's
#pragma unroll
            for (int i = 0; i < 8; ++i) Pair<T>::narrow(v[i], w + 4 + i * P);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[W + i], 1);
            if (live && col < a.cols) {
                store_shifted<T>(out + col, a.cols - col < 16 ? a.cols - col : 16, !first, !final && col + 16 < a.cols, w);
            }
        }
    }
}

// The layout of rows at `p` with that stride.
int layout_of(const void *p, int64_t stride, int64_t cols, int64_t size) {
    if (cols % 16 == 0 && stride * size % 32 == 0 && aligned(p, 32)) return kSectors;
    return cols * size % 16 == 0 && stride * size % 16 == 0 && aligned(p, 16) ? kUnits : kScattered;
}

template <typename T, bool NV, int LAYOUT>
int quantize_rows(const QuantArgs &a, int sms, cudaStream_t stream) {
    Grid g = grid_for((static_cast<int64_t>(a.rows) + kScaleTileRows - 1) / kScaleTileRows * kScaleTileRows, a.units);
    if (kAhead<T, NV, LAYOUT>) {
        const unsigned fit = (kQuantizePerSm<T, NV, LAYOUT> * static_cast<unsigned>(sms) + g.grid.y - 1) / g.grid.y;
        if (g.grid.x > fit) g.grid.x = fit;
    }
    return launch(quantize_kernel<T, NV, LAYOUT>, g.grid, g.block, 0, stream, a);
}

template <typename T, bool NV>
int quantize_as(const QuantArgs &a, int sms, cudaStream_t stream) {
    switch (layout_of(a.x, a.x_stride, a.cols, sizeof(T))) {
        case kSectors: return quantize_rows<T, NV, kSectors>(a, sms, stream);
        case kUnits: return quantize_rows<T, NV, kUnits>(a, sms, stream);
        default: return quantize_rows<T, NV, kScattered>(a, sms, stream);
    }
}

template <typename T, bool NV>
int dequantize_as(const DequantArgs &a, cudaStream_t stream) {
    const Grid g = grid_for(a.rows, a.data_units);
    switch (layout_of(a.out, a.out_stride, a.cols, sizeof(T))) {
        case kSectors: return launch(dequantize_kernel<T, NV, kSectors>, g.grid, g.block, 0, stream, a);
        case kUnits: return launch(dequantize_kernel<T, NV, kUnits>, g.grid, g.block, 0, stream, a);
        default: return launch(dequantize_kernel<T, NV, kScattered>, g.grid, g.block, 0, stream, a);
    }
}

// The element type and the format as template arguments.
#define LINEAR_BY_FORMAT(type, nv, FN, ...)                                                    \
    ((type) == LINEAR_F16    ? ((nv) ? FN<__half, true>(__VA_ARGS__) : FN<__half, false>(__VA_ARGS__)) \
     : (type) == LINEAR_BF16 ? ((nv) ? FN<__nv_bfloat16, true>(__VA_ARGS__) : FN<__nv_bfloat16, false>(__VA_ARGS__)) \
                             : ((nv) ? FN<float, true>(__VA_ARGS__) : FN<float, false>(__VA_ARGS__)))

int check_matrix(int64_t rows, int64_t cols, int32_t format, int32_t exponent) {
    if (rows < 0 || cols < 0 || (format != FP4_MX && format != FP4_NV) || exponent < -100 || exponent > 100 ||
        (format == FP4_MX && exponent != 0)) {
        return GEMM_ERR_INVALID_ARG;
    }
    return rows > kMaxDim || cols > kMaxCols ? GEMM_ERR_UNSUPPORTED_SHAPE : GEMM_OK;
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
    return LINEAR_BY_FORMAT(type, nv, quantize_as, a, sms, s);
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
    return LINEAR_BY_FORMAT(type, nv, dequantize_as, a, s);
}

}  // extern "C"
