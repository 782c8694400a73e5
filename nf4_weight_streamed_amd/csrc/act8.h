// The 8-bit checkpoint format of activations, on the device: 64 consecutive elements of a
// row share one step,
//   a = max |x|,  scale = RN32(a / 127),  code = 128 + rne(x RN32(127 / a)),
//   value = RN32((code - 128) scale),
// so that a value is off by at most half a step, a / 254, and 2^-23 of itself (a subnormal step's rounding adds up
// to 127 2^-150).
#pragma once

#include <type_traits>

#include "device.h"

namespace nf4 {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Magnitude bits of the largest of 8 bf16: as whole numbers they are in order of size, with
// infinities and NaNs above all finite ones.
__device__ __forceinline__ uint32_t top_bits(u32x4 x) {
    u16x2 t = __builtin_bit_cast(u16x2, x[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, x[i] & 0x7FFF7FFFu));
    return t[0] > t[1] ? t[0] : t[1];
}

// The largest over 8 neighbouring lanes: two steps within quads, one across them.
__device__ __forceinline__ uint32_t max_of_8_lanes(uint32_t v) {
    auto other = [](uint32_t w, auto c) {
        return uint32_t(__builtin_amdgcn_update_dpp(int(w), int(w), decltype(c)::value, 0xF, 0xF, false));
    };
    v = max(v, other(v, std::integral_constant<int, 0xB1>{}));   // quad_perm 1 0 3 2
    v = max(v, other(v, std::integral_constant<int, 0x4E>{}));   // quad_perm 2 3 0 1
    return max(v, other(v, std::integral_constant<int, 0x141>{}));  // row_half_mirror
}

struct Act8Step {
    float inv, lift, scale;  // code = 128 + rne(x * lift * inv)
    bool bad;                // the block holds an infinity or a NaN: all its values are NaN
};

// From the block's top_bits. 127 / a would pass fp32's range for a below 2^-121: blocks below
// 2^-64 are lifted by 2^64 first, which is exact.
__device__ __forceinline__ Act8Step act8_step(uint32_t top) {
    Act8Step s;
    const float a = __uint_as_float(top << 16);
    s.bad = top >= 0x7F80u;
    s.lift = a < 0x1p-64f ? 0x1p64f : 1.0f;
    s.inv = a > 0.0f ? 127.0f / (a * s.lift) : 0.0f;
    s.scale = s.bad ? __builtin_nanf("") : a / 127.0f;
    return s;
}

// 4 codes. Adding 1.5 * 2^23 leaves the rounded product (of at most 127 in size), plus 128, in
// the sum's low byte; the fused product is not rounded before.
__device__ __forceinline__ uint32_t act8_codes4(uint32_t w0, uint32_t w1, const Act8Step& s) {
    constexpr float kMagic = 12582912.0f + 128.0f;
    const uint32_t c0 = __float_as_uint(__builtin_fmaf(bf16_lo(w0) * s.lift, s.inv, kMagic));
    const uint32_t c1 = __float_as_uint(__builtin_fmaf(bf16_hi(w0) * s.lift, s.inv, kMagic));
    const uint32_t c2 = __float_as_uint(__builtin_fmaf(bf16_lo(w1) * s.lift, s.inv, kMagic));
    const uint32_t c3 = __float_as_uint(__builtin_fmaf(bf16_hi(w1) * s.lift, s.inv, kMagic));
    const uint32_t lo = __builtin_amdgcn_perm(c1, c0, 0x0C0C0400u), hi = __builtin_amdgcn_perm(c3, c2, 0x0C0C0400u);
    return s.bad ? 0x80808080u : lo | (hi << 16);
}

// 8 codes of 8 bf16; the 8 lanes of a block call it together, and any of them may store the scale.
__device__ __forceinline__ u32x2 act8_quantize8(u32x4 x, float& scale) {
    const Act8Step s = act8_step(max_of_8_lanes(top_bits(x)));
    scale = s.scale;
    return u32x2{act8_codes4(x[0], x[1], s), act8_codes4(x[2], x[3], s)};
}

// The values of 4 codes. (Folding the 128 into a fused operation on the byte would pass fp32's
// range for the largest bf16 value.)
__device__ __forceinline__ void act8_values4(uint32_t c, float scale, float (&v)[8], int at) {
    c ^= 0x80808080u;  // code - 128 as a signed byte
    v[at] = float(int8_t(c)) * scale;
    v[at + 1] = float(int8_t(c >> 8)) * scale;
    v[at + 2] = float(int8_t(c >> 16)) * scale;
    v[at + 3] = float(int8_t(c >> 24)) * scale;
}

__device__ __forceinline__ void act8_values8(u32x2 c, float scale, float (&v)[8]) {
    act8_values4(c.x, scale, v, 0);
    act8_values4(c.y, scale, v, 4);
}

__device__ __forceinline__ u32x4 pack_octet(const float (&v)[8]) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

__device__ __forceinline__ void unpack_octet(u32x4 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

}  // namespace nf4
