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
typedef float f32x8_a16 __attribute__((ext_vector_type(8), aligned(16)));  // in memory

template <typename T>
struct V8;
template <>
struct V8<bf16> {
    typedef bf16x8 type;
};
template <>
struct V8<f16> {
    typedef f16x8 type;
};
template <>
struct V8<float> {
    typedef f32x8_a16 type;
};

// 8 consecutive elements as float; `n` of them exist (the rest read as 0).
// vec: p is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* __restrict__ p, int n, bool vec, float (&v)[8]) {
    if (n >= 8 && vec) {
        const typename V8<T>::type t = *reinterpret_cast<const typename V8<T>::type*>(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? (float)p[e] : 0.f;
    }
}

// The same 8 elements rounded once (nearest even) to T.
template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, int n, bool vec, const float (&v)[8]) {
    if (n >= 8 && vec) {
        f32x8 t;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = v[e];
        *reinterpret_cast<typename V8<T>::type*>(p) = __builtin_convertvector(t, typename V8<T>::type);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (T)v[e];
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

// gelu_tanh(z) = z/2 (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3):
// one exponential and one reciprocal, and no cancellation in the tail, where
// 1 + tanh u loses its bits. gelu(z) = z erfc(-z / sqrt 2) / 2 for the same reason.
__device__ __forceinline__ float act_value(int act, float z) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? z : z * 0.f;
        case ACT_RELU2: {
            const float r = z > 0.f ? z : z * 0.f;
            return r * r;
        }
        case ACT_GELU: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        case ACT_GELU_TANH: return z * sigmoid(kGeluTwoK * z * fmaf(kGeluCubic * z, z, 1.f));
        case ACT_SILU: return z * sigmoid(z);
        default: return z;
    }
}

// The derivative at z. relu'(0) = 0. Factors z times a vanishing term are
// taken at z clamped to +-30, where that term is 0 already, so that no
// inf * 0 comes up for a large finite z; a NaN stays one through the first term.
__device__ __forceinline__ float act_slope(int act, float z) {
    const float zc = fminf(fmaxf(z, -30.f), 30.f);
    switch (act) {
        case ACT_RELU: return z > 0.f ? 1.f : z != z ? z : 0.f;
        case ACT_RELU2: return z > 0.f ? 2.f * z : z != z ? z : 0.f;
        case ACT_GELU:
            return fmaf(zc * 0.3989422804014327f, __builtin_amdgcn_exp2f(-0.72134752044448170f * zc * zc),
                        0.5f * erfcf(-0.70710678118654752f * z));
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

// The epilogue of 8 consecutive accumulators of row r from column c on, n of
// them inside the matrix. bias: their bias values (forward).
template <typename T>
__device__ __forceinline__ void epilogue8(const Epilogue& E, int64_t r, int c, int n, float (&v)[8],
                                          const float (&bias)[8]) {
    if (E.mode == EPI_GRAD_WEIGHT) {
        float* y = static_cast<float*>(E.y) + r * E.ld_y + c;
        if (E.accumulate) {
            float o[8];
            load8(y, n, E.vec_y, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        store8(y, n, E.vec_y, v);
        return;
    }
    if (E.mode == EPI_FORWARD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
        if (E.z) store8(static_cast<T*>(E.z) + r * E.ld_z + c, n, E.vec_z, v);
        if (E.act != ACT_NONE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_value(E.act, v[e]);
        }
    } else if (E.act != ACT_NONE) {
        float z[8];
        load8(static_cast<const T*>(E.z) + r * E.ld_z + c, n, E.vec_z, z);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= act_slope(E.act, z[e]);
    }
    if (E.add) {
        float a[8];
        load8(static_cast<const T*>(E.add) + r * E.ld_add + c, n, E.vec_add, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += a[e];
    }
    store8(static_cast<T*>(E.y) + r * E.ld_y + c, n, E.vec_y, v);
}

}  // namespace muon
