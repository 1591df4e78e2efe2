// device.hpp -- small device helpers of the layer kernels (norm.hip,
// proj_i8.hip, delta.hip): vector types, BF16 rounding, wave reductions and
// explicit waits.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace tp1 {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// FP32 -> BF16, round to nearest, ties to even; NaN -> quiet NaN.
__device__ __forceinline__ uint16_t round_bf16(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);
}
// Two floats rounded and packed (low half first).
__device__ __forceinline__ unsigned pack_bf16(float a, float b) {
    return (unsigned)round_bf16(a) | ((unsigned)round_bf16(b) << 16);
}

// Exact BF16 -> FP32 of the two halves of a packed pair, and of one value.
__device__ __forceinline__ float bf16_lo(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(unsigned u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((unsigned)v << 16); }

// Wave-uniform value, kept in a scalar register.
__device__ __forceinline__ int scalar(int v) { return __builtin_amdgcn_readfirstlane(v); }

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

// Sum over the 64 lanes in a fixed tree: DPP butterflies inside each 16-lane
// row, then the four row sums added in order.  Wave-uniform result.
__device__ __forceinline__ float sum64(float v) {
    v += dpp_move<0xB1>(v);   // quad_perm [1,0,3,2]
    v += dpp_move<0x4E>(v);   // quad_perm [2,3,0,1]
    v += dpp_move<0x141>(v);  // row_half_mirror
    v += dpp_move<0x140>(v);  // row_mirror
    return ((lane_value(v, 0) + lane_value(v, 16)) + lane_value(v, 32)) + lane_value(v, 48);
}

// Largest of the 64 lanes' unsigned values (wave-uniform).  On the bits of
// magnitudes this is the largest magnitude, with infinity above every finite
// value and NaN above infinity.
__device__ __forceinline__ unsigned max64(unsigned v) {
    auto step = [](unsigned a, unsigned b) { return a > b ? a : b; };
    v = step(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true));
    v = step(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true));
    v = step(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true));
    v = step(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true));
    const unsigned a = step(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
    const unsigned b = step(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48));
    return step(a, b);
}

// s_waitcnt vmcnt(N) leaving the other counters alone (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N <= 63, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

}  // namespace tp1
