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

// v kLargest / amax of 16-bit v, rounded once to float32: values divided by one another
// often fall on the border between two 8-bit values, where an error of the quotient's last
// bit takes the wrong one. kLargest is 7/8 of a power of two: a = 7 v / 8 is exact, t =
// a / amax is corrected by its exact remainder, and the power of two is exact again. A
// quotient of 16-bit values that is no border is further from one than this rounding, so
// that the one to 8 bits takes the nearest value.
template <int F>
struct ExactScale : BlockScale<F> {
    float rcp;
    __device__ __forceinline__ explicit ExactScale(uint32_t bits) : BlockScale<F>(bits) { rcp = 1.f / this->amax; }
    // 8 values, 0 from the n-th on
    __device__ __forceinline__ void scale8(float (&v)[8], int n) const {
        constexpr float P = F == EIGHT_E4M3 ? 512.f : 65536.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = 0.875f * v[e], t = a * rcp;
            v[e] = e < n ? fmaf(fmaf(-t, this->amax, a), rcp, t) * P : 0.f;
        }
    }
};

// The same of float32 v, whose quotient may lie nearer to a border than float32's last
// bit. v times a factor just below and just above kLargest / amax: where both round to
// the same 8-bit values, so does the quotient between them. Else it is rounded to odd (an
// inexact one to the neighbour whose last bit is 1), which no border is, so that the
// rounding to 8 bits sees the side it lies on. (That for every value: 1600 x 6400 15.6 us
// in one order, not 13.1. The corrected division above, which rounds twice: 13.1 as well,
// rows of 16384 x 1600 25.6 against 26.2, a norm of them 39.2 against 38.6.)
template <int F>
struct OnceScale : BlockScale<F> {
    float below, above;
    __device__ __forceinline__ explicit OnceScale(uint32_t bits) : BlockScale<F>(bits) {
        // the scale 2^-24 of itself off, its reciprocal 2^-23 (both normal numbers; a NaN
        // beside an infinity), three more roundings of 2^-24 to come
        const float k = __builtin_amdgcn_rcpf(this->scale) + 0.f * this->amax;
        below = k * (1.f - 0x1p-21f);
        above = k * (1.f + 0x1p-21f);
    }
    __device__ __forceinline__ float odd(float v) const {
        constexpr float P = F == EIGHT_E4M3 ? 512.f : 65536.f;
        // blocks below 1 scaled up, so that the remainders of the smallest do not underflow
        const bool up = this->amax < 1.f;
        const float by = up ? 0.875f * 0x1p100f : 0.875f, of = up ? this->amax * 0x1p100f : this->amax, rcp = 1.f / of;
        const float a = by * v, low = fmaf(by, v, -a), t = a * rcp;
        const float q = fmaf(fmaf(-t, of, a) + low, rcp, t);  // one of the quotient's neighbours
        const float rest = fmaf(-q, of, a) + low;             // of its sign, and 0 for an exact one
        const int u = __float_as_int(q), toward = ((__float_as_int(rest) ^ u) >> 31) | 1;
        const bool off = fabsf(rest) > 0.f && fabsf(q) > 0.f;  // (of a NaN neither)
        return __int_as_float(off && !(u & 1) ? u + toward : u) * P;
    }
    __device__ __forceinline__ void scale8(float (&v)[8], int n) const {
        float lo[8], hi[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo[e] = v[e] * below;
            hi[e] = v[e] * above;
        }
        const u32x2 p = pack8<F>(lo), q = pack8<F>(hi);
        if (__builtin_expect(p[0] != q[0] || p[1] != q[1], 0)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) lo[e] = odd(v[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? lo[e] : 0.f;
    }
};
// What values of type T are scaled by.
template <int F, typename T>
using ScaleOf = std::conditional_t<sizeof(T) == 4, OnceScale<F>, ExactScale<F>>;

}  // namespace muon
