// Device building blocks of the 8-bit operators: element types, 16-byte
// pieces of byte matrices, e4m3 and int8 conversions.
#pragma once

#include "gemv_device.hpp"

namespace fp8dev {

using gemvdev::f32x4;
using gemvdev::quad;
using gemvdev::quad_any;
using gemvdev::TBF16;
using gemvdev::TF16;
using gemvdev::TF32;
using gemvdev::widen;

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr float kE4m3Max = 448.0f;
constexpr float kSmallestScale = 0x1p-126f;  // the smallest normal fp32: its reciprocal is finite

// 16 bytes at p of which `n` lie inside the row; what lies behind reads as
// zero and is never touched.
__device__ __forceinline__ quad load_bytes(const uint8_t* p, int n) {
    if (n >= 16) return *reinterpret_cast<const quad_any*>(p);
    quad v{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) v[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return v;
}

// The 16 bytes from column `at` of a row of K on, one load: near the row's end
// the row's last 16, moved down.
__device__ __forceinline__ quad load_end(const uint8_t* row, int64_t at, int K) {
    if (K < 16) return load_bytes(row + at, (int)(K - at));
    const int64_t from = at < K - 16 ? at : K - 16;
    const int down = (int)(at - from);
    quad v = *reinterpret_cast<const quad_any*>(row + from);
    if (down & 4) v = quad{v[1], v[2], v[3], 0u};
    if (down & 8) v = quad{v[2], v[3], 0u, 0u};
    if (down >= 16) v = quad{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_amdgcn_alignbyte(i < 3 ? v[i + 1] : 0u, v[i], down & 3);
    return v;
}

// What follows from v is not kept in registers from before a loop on.
__device__ __forceinline__ int worked_out_here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// Rounds an fp32 result to the output type (to nearest even).
__device__ __forceinline__ float narrow(TF32, float v) { return v; }
__device__ __forceinline__ uint16_t narrow(TF16, float v) {
    return __builtin_bit_cast(uint16_t, (_Float16)v);
}
__device__ __forceinline__ uint16_t narrow(TBF16, float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Four fp32 values rounded to e4m3 (nearest even) in one word.  Values past
// 448 by less than half a step round to 448; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// The bits of |v| as an unsigned number: ordered as the magnitudes are, with
// infinity above every number and NaN above infinity, so an integer maximum
// carries NaN along where fmaxf would drop it.
__device__ __forceinline__ uint32_t magnitude(float v) {
    return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
// Maximum over each 16-lane row, in every lane of it.
__device__ __forceinline__ uint32_t row_max16(uint32_t v) {
    v = max_u32(v, dpp_u32<gemvdev::kDppSwapAdjacent>(v));
    v = max_u32(v, dpp_u32<gemvdev::kDppSwapPairs>(v));
    v = max_u32(v, dpp_u32<gemvdev::kDppHalfRowMirror>(v));
    return max_u32(v, dpp_u32<gemvdev::kDppRowMirror>(v));
}
// ... and over the whole wavefront.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = row_max16(v);
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max_u32(r[0], r[1]);
    r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max_u32(r[0], r[1]);
}

}  // namespace fp8dev
