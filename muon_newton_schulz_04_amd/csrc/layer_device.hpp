// Device helpers of the layer operators: 16-bit type traits, chunks of 8
// elements, the activations and their derivatives, and the epilogue of a
// product.
#pragma once

#include "layers.hpp"
#include "ns_mfma_common.hpp"

namespace muon {

typedef _Float16 f16;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

// 8 elements as a vector, and the same in memory at any element's address (the
// hardware takes unaligned 16-byte accesses).
template <typename T>
struct V8;
template <>
struct V8<bf16> {
    typedef bf16x8 type;
    typedef bf16x8 mem __attribute__((aligned(2)));
};
template <>
struct V8<f16> {
    typedef f16x8 type;
    typedef f16x8 mem __attribute__((aligned(2)));
};
template <>
struct V8<float> {
    typedef f32x8 type;
    typedef f32x8 mem __attribute__((aligned(4)));
};
typedef u32x4 u32x4_mem __attribute__((aligned(2)));
typedef f32x4 f32x4_mem __attribute__((aligned(4)));

// 8 consecutive elements as float; n of them exist (the others read as 0).
template <typename T>
__device__ __forceinline__ void load8(const T* __restrict__ p, int n, float (&v)[8]) {
    if (n >= 8) {
        const typename V8<T>::type t = *reinterpret_cast<const typename V8<T>::mem*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? (float)p[e] : 0.f;
    }
}

// The same 8 elements rounded once (nearest even) to T.
template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, int n, const float (&v)[8]) {
    if (n >= 8) {
        f32x8 t;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = v[e];
        *reinterpret_cast<typename V8<T>::mem*>(p) = __builtin_convertvector(t, typename V8<T>::type);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (T)v[e];
    }
}

// The same, stored nontemporally: a product's outputs would push the operand
// panels that the workgroups share out of L2 (c_fc forward at 16384 x 1600 x
// 6400 with the pre-activation kept: 401 us with plain stores, 366 so).
template <typename T>
__device__ __forceinline__ void stream8(T* __restrict__ p, int n, const float (&v)[8]) {
    if (n >= 8) {
        f32x8 t;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = v[e];
        if constexpr (sizeof(T) == 2) {
            __builtin_nontemporal_store(__builtin_convertvector(t, typename V8<T>::type),
                                        reinterpret_cast<typename V8<T>::mem*>(p));
        } else {
            const f32x4 lo = {t[0], t[1], t[2], t[3]}, up = {t[4], t[5], t[6], t[7]};
            __builtin_nontemporal_store(lo, reinterpret_cast<f32x4_mem*>(p));
            __builtin_nontemporal_store(up, reinterpret_cast<f32x4_mem*>(p + 4));
        }
    } else {
        store8(p, n, v);
    }
}

enum { ACT_NONE = 0, ACT_RELU, ACT_RELU2, ACT_GELU, ACT_GELU_TANH, ACT_SILU };

// 1 / (1 + e^-x) from the hardware's exp2 and reciprocal (about 1 ulp each);
// an overflowing e^-x gives 0.
__device__ __forceinline__ float sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * x));
}

constexpr float kGeluTwoK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// gelu(z) = z Phi(z) with the normal distribution's lower tail as
// Phi(-a) = e^(-a^2/2) t p(t), t = 1 / (1 + a / 4), a >= 0: p of degree 9 fitted
// to the scaled complementary error function with equal relative error on
// t in (0, 1] (3.3e-8; 3.7e-7 evaluated in float32), so the tail keeps its
// digits. Half the instructions of the library's erfc. `e`: e^(-a^2/2).
__device__ __forceinline__ float normal_tail(float a, float& e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.25f, a, 1.f));
    e = __builtin_amdgcn_exp2f(-0.72134752044448170f * a * a);
    float p = 0.0198428007f;
    p = fmaf(p, t, -0.0811460938f);
    p = fmaf(p, t, 0.0960938974f);
    p = fmaf(p, t, -0.03221571f);
    p = fmaf(p, t, 0.0639933433f);
    p = fmaf(p, t, 0.0588711657f);
    p = fmaf(p, t, 0.0816244597f);
    p = fmaf(p, t, 0.0934640081f);
    p = fmaf(p, t, 0.0997365477f);
    p = fmaf(p, t, 0.099735565f);
    return p * t * e;
}
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float q = normal_tail(fabsf(z), e);
    return z > 0.f ? 1.f - q : q;
}

// gelu_tanh(z) = z/2 (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3):
// one exponential and one reciprocal, and no cancellation in the tail, where
// 1 + tanh u loses its bits.
template <int act>
__device__ __forceinline__ float act_value(float z) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? z : z * 0.f;
        case ACT_RELU2: {
            const float r = z > 0.f ? z : z * 0.f;
            return r * r;
        }
        case ACT_GELU: {
            float e;
            return z * normal_cdf(z, e);
        }
        case ACT_GELU_TANH: return z * sigmoid(kGeluTwoK * z * fmaf(kGeluCubic * z, z, 1.f));
        case ACT_SILU: return z * sigmoid(z);
        default: return z;
    }
}

// The derivative at z. relu'(0) = 0. Factors z times a vanishing term are
// taken at z clamped to +-30, where that term is 0 already, so that no
// inf * 0 comes up for a large finite z; a NaN stays one through the first term.
template <int act>
__device__ __forceinline__ float act_slope(float z) {
    const float zc = fminf(fmaxf(z, -30.f), 30.f);
    switch (act) {
        case ACT_RELU: return z > 0.f ? 1.f : z != z ? z : 0.f;
        case ACT_RELU2: return z > 0.f ? 2.f * z : z != z ? z : 0.f;
        case ACT_GELU: {
            float e;
            const float q = normal_cdf(z, e);
            return fmaf(zc * 0.3989422804014327f, e, q);
        }
        case ACT_GELU_TANH: {
            const float q = sigmoid(kGeluTwoK * z * fmaf(kGeluCubic * z, z, 1.f));
            return fmaf(zc * q * (1.f - q) * kGeluTwoK, fmaf(3.f * kGeluCubic * zc, zc, 1.f), q);
        }
        case ACT_SILU: {
            const float q = sigmoid(z);
            return fmaf(zc * q, 1.f - q, q);
        }
        default: return 1.f;
    }
}

// One uniform branch for a chunk of 8, not one an element.
#define MUON_ACT_CASE(A, F)                                 \
    case A:                                                 \
        _Pragma("unroll") for (int e = 0; e < 8; ++e) v[e] = F<A>(v[e]); \
        break;
__device__ __forceinline__ void act_values(int act, float (&v)[8]) {
    switch (act) {
        MUON_ACT_CASE(ACT_RELU, act_value)
        MUON_ACT_CASE(ACT_RELU2, act_value)
        MUON_ACT_CASE(ACT_GELU, act_value)
        MUON_ACT_CASE(ACT_GELU_TANH, act_value)
        MUON_ACT_CASE(ACT_SILU, act_value)
    }
}
__device__ __forceinline__ void act_slopes(int act, float (&v)[8]) {
    switch (act) {
        MUON_ACT_CASE(ACT_RELU, act_slope)
        MUON_ACT_CASE(ACT_RELU2, act_slope)
        MUON_ACT_CASE(ACT_GELU, act_slope)
        MUON_ACT_CASE(ACT_GELU_TANH, act_slope)
        MUON_ACT_CASE(ACT_SILU, act_slope)
    }
}
#undef MUON_ACT_CASE

// What the epilogue reads of a chunk of 8 outputs, fetched ahead of its use as
// 16-byte vectors: first8 is z on the way back through an activation, else
// add, or the lower half of a weight gradient to add to; second8 is add where
// first8 is z, or the upper half.
template <typename T>
__device__ __forceinline__ u32x4 first8(const Epilogue& E, int64_t r, int64_t c) {
    const void* p = nullptr;
    if (E.mode == EPI_GRAD_WEIGHT) {
        if (E.accumulate) p = static_cast<const float*>(E.y) + r * E.ld_y + c;
    } else if (E.mode == EPI_GRAD_INPUT && E.act != ACT_NONE) {
        p = static_cast<const T*>(E.z) + r * E.ld_z + c;
    } else if (E.add) {
        p = static_cast<const T*>(E.add) + r * E.ld_add + c;
    }
    return p ? __builtin_nontemporal_load(static_cast<const u32x4_mem*>(p)) : u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ bool has_second(const Epilogue& E) {
    return E.mode == EPI_GRAD_WEIGHT ? E.accumulate != 0 : E.mode == EPI_GRAD_INPUT && E.act != ACT_NONE && E.add;
}
template <typename T>
__device__ __forceinline__ u32x4 second8(const Epilogue& E, int64_t r, int64_t c) {
    const void* p = E.mode == EPI_GRAD_WEIGHT
                        ? static_cast<const void*>(static_cast<const float*>(E.y) + r * E.ld_y + c + 4)
                        : static_cast<const void*>(static_cast<const T*>(E.add) + r * E.ld_add + c);
    return __builtin_nontemporal_load(static_cast<const u32x4_mem*>(p));
}

template <typename T>
__device__ __forceinline__ void widen8(const u32x4& u, float (&v)[8]) {
    const typename V8<T>::type t = __builtin_bit_cast(typename V8<T>::type, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
}

// The epilogue of 8 consecutive accumulators of row r from column c on, n of
// them inside the matrix. bias: their bias values (forward). in, in2: first8's
// and second8's if n is 8 or more; a chunk at the matrix's edge is read in place.
template <typename T>
__device__ __forceinline__ void finish8(const Epilogue& E, int64_t r, int64_t c, int n, float (&v)[8],
                                        const float (&bias)[8], const u32x4& in, const u32x4& in2) {
    float t[8];
    if (E.mode == EPI_GRAD_WEIGHT) {
        float* y = static_cast<float*>(E.y) + r * E.ld_y + c;
        if (E.accumulate) {
            if (n >= 8) {
                const f32x4 lo = __builtin_bit_cast(f32x4, in), up = __builtin_bit_cast(f32x4, in2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    t[e] = lo[e];
                    t[4 + e] = up[e];
                }
            } else {
                load8(y, n, t);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += t[e];
        }
        stream8(y, n, v);
        return;
    }
    bool fetched = false;  // `in` was z, and add is in2
    if (E.mode == EPI_FORWARD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
        if (E.z) stream8(static_cast<T*>(E.z) + r * E.ld_z + c, n, v);
        act_values(E.act, v);
    } else if (E.act != ACT_NONE) {
        fetched = true;
        if (n >= 8)
            widen8<T>(in, t);
        else
            load8(static_cast<const T*>(E.z) + r * E.ld_z + c, n, t);
        act_slopes(E.act, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= t[e];
    }
    if (E.add) {
        if (n >= 8 && fetched)
            widen8<T>(in2, t);
        else if (n >= 8)
            widen8<T>(in, t);
        else
            load8(static_cast<const T*>(E.add) + r * E.ld_add + c, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    stream8(static_cast<T*>(E.y) + r * E.ld_y + c, n, v);
}

}  // namespace muon
