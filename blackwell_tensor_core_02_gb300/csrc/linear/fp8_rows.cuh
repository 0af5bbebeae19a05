// fp8_rows.cuh -- rows of microscaled 8-bit floats (see checkpoint_ops.h): conversions,
// and the checks of memory that their calls share.
#pragma once

#include "common.cuh"

namespace linear_ops {

constexpr int kFp8Block = 32;  // elements of a row with one scale

inline int64_t fp8_blocks(int64_t cols) { return (cols + kFp8Block - 1) / kFp8Block; }

// Two floats to E4M3, to nearest even, magnitudes past 448 to 448; lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The two values of E4M3 codes (low byte first), which fp16 holds.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
    return h;
}

// The larger magnitude; NaN if either is.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// The E8M0 code of a block's scale from its largest magnitude, 2^(floor(log2(amax)) - 8) with
// the exponent at least -127; 255, NaN, where an element is an infinity or NaN.
__device__ __forceinline__ uint32_t scale_code(float amax) {
    const int e = static_cast<int>(__float_as_uint(amax) >> 23);
    return e == 255 ? 255u : static_cast<uint32_t>(e > 8 ? e - 8 : 0);
}

// What brings a block's elements to E4M3's range: 2^(127 - code); NaN for 255.
__device__ __forceinline__ float scale_inverse(uint32_t code) {
    return __uint_as_float(code == 255u ? 0x7fffffffu : (254u - code) << 23);
}

// 2^(code - 127); NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t code) {
    return __uint_as_float(code == 255u ? 0x7fffffffu : (code == 0u ? 0x00400000u : code << 23));
}

// ------------------------------------------------------------------- host --

struct Span {
    const void *p;
    int64_t bytes;
};

// Whether an output shares memory with an input or another output; not the first output with the first
// input, whose rows may lie between each other's (rows_overlap()).
template <int OUTS, int INS>
bool any_overlap(const Span (&outs)[OUTS], const Span (&ins)[INS]) {
    for (int i = 0; i < OUTS; ++i) {
        for (int j = i == 0 ? 1 : 0; j < INS; ++j) {
            if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
        }
        for (int j = 0; j < i; ++j) {
            if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
        }
    }
    return false;
}

}  // namespace linear_ops
