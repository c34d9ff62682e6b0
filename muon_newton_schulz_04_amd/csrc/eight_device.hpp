// Device helpers of 8-bit floating point with a scale for each block of 128:
// formats, block maxima, and the rounding of values to 8 bits.
#pragma once

#include "layer_device.hpp"

namespace muon {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A block's largest magnitude counts as kSmallest at least, which keeps the
// scale and its reciprocal normal numbers for a block of zeros too.
constexpr float kSmallest = 0x1p-110f;
template <int F>
constexpr float kLargest = F == EIGHT_E4M3 ? 448.f : 57344.f;

// |v| as bits: ordered as the magnitudes are, infinity and NaN last.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of 16 lanes' values (a row of the wave), in each of them.
template <int CTRL>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = umax(v, turned<0x128>(v));  // row_ror 8, 4, 2, 1
    v = umax(v, turned<0x124>(v));
    v = umax(v, turned<0x122>(v));
    return umax(v, turned<0x121>(v));
}

// A block's scale from its largest magnitude: a block that holds an infinity or
// a NaN gets it as its scale, and so stands for no number anywhere.
template <int F>
struct BlockScale {
    float amax, scale;
    __device__ __forceinline__ explicit BlockScale(uint32_t bits) {
        amax = __uint_as_float(umax(bits, __float_as_uint(kSmallest)));
        scale = amax / kLargest<F>;
    }
};

// Two values rounded to nearest even into the low or high half of a word.
template <int F, bool HI>
__device__ __forceinline__ uint32_t pack2(float a, float b, uint32_t old) {
    if constexpr (F == EIGHT_E4M3)
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
    else
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(a, b, (int)old, HI);
}
template <int F>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    return pack2<F, true>(c, d, pack2<F, false>(a, b, 0u));
}
template <int F>
__device__ __forceinline__ u32x2 pack8(const float (&v)[8]) {
    return u32x2{pack4<F>(v[0], v[1], v[2], v[3]), pack4<F>(v[4], v[5], v[6], v[7])};
}

// v kLargest / amax rounded once: values divided by one another often fall on the
// border between two 8-bit values, where an error of the quotient's last bit takes the
// wrong one. kLargest is 7/8 of a power of two: a = 7 v / 8, exact for 16-bit v and
// with the rest of its rounding in `low` for 32-bit ones (WIDE), t = a / amax is
// corrected by its exact remainder, and the power of two is exact again.
template <int F, bool WIDE>
struct ExactScale : BlockScale<F> {
    float rcp;
    __device__ __forceinline__ explicit ExactScale(uint32_t bits) : BlockScale<F>(bits) { rcp = 1.f / this->amax; }
    __device__ __forceinline__ float operator()(float v) const {
        constexpr float P = F == EIGHT_E4M3 ? 512.f : 65536.f;
        const float a = 0.875f * v, t = a * rcp;
        float rest = fmaf(-t, this->amax, a);
        if constexpr (WIDE) rest += fmaf(0.875f, v, -a);
        return fmaf(rest, rcp, t) * P;
    }
};

}  // namespace muon
