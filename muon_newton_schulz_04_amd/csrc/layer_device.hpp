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

// gelu_tanh's sigmoid(2u) = 1 / (1 + 2^(z (A + B z^2))), and 2u' = C + D z^2
constexpr float kGeluA = -2.3022081985f;   // -2 sqrt(2 / pi) log2 e
constexpr float kGeluB = -0.1029432397f;   // 0.044715 A
constexpr float kGeluC = 1.5957691216f;    // 2 sqrt(2 / pi)
constexpr float kGeluD = 0.2140644488f;    // 3 * 0.044715 C
__device__ __forceinline__ float gelu_gate(float z, float z2) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * fmaf(kGeluB, z2, kGeluA)));
}

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
        case ACT_RELU: return z < 0.f ? 0.f : z;  // a NaN stays one
        case ACT_RELU2: {
            const float r = z < 0.f ? 0.f : z;
            return r * r;
        }
        case ACT_GELU: {
            float e;
            return z * normal_cdf(z, e);
        }
        case ACT_GELU_TANH: return z * gelu_gate(z, z * z);
        case ACT_SILU: return z * sigmoid(z);
        default: return z;
    }
}

// The derivative at z. relu'(0) = 0. Products of z with a vanishing term are
// grouped, and z^2 bounded where the term is 0 already, so that no inf * 0 comes
// up for a large finite z.
template <int act>
__device__ __forceinline__ float act_slope(float z) {
    switch (act) {
        case ACT_RELU: return z > 0.f ? 1.f : z != z ? z : 0.f;
        case ACT_RELU2: return z > 0.f ? 2.f * z : z != z ? z : 0.f;
        case ACT_GELU: {
            float e;
            const float q = normal_cdf(z, e);
            return fmaf(z * e, 0.3989422804014327f, q);
        }
        case ACT_GELU_TANH: {
            const float z2 = fminf(z * z, 900.f), q = gelu_gate(z, z2);
            return fmaf(z * q, (1.f - q) * fmaf(kGeluD, z2, kGeluC), q);
        }
        case ACT_SILU: {
            const float q = sigmoid(z);
            return fmaf(z * q, 1.f - q, q);
        }
        default: return 1.f;
    }
}

// One uniform branch for all the values (8, a chunk, or more), not one an element.
#define MUON_ACT_CASE(A, F)                                 \
    case A:                                                 \
        _Pragma("unroll") for (int e = 0; e < N; ++e) v[e] = F<A>(v[e]); \
        break;
template <int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    switch (act) {
        MUON_ACT_CASE(ACT_RELU, act_value)
        MUON_ACT_CASE(ACT_RELU2, act_value)
        MUON_ACT_CASE(ACT_GELU, act_value)
        MUON_ACT_CASE(ACT_GELU_TANH, act_value)
        MUON_ACT_CASE(ACT_SILU, act_value)
    }
}
template <int N>
__device__ __forceinline__ void act_slopes(int act, float (&v)[N]) {
    switch (act) {
        MUON_ACT_CASE(ACT_RELU, act_slope)
        MUON_ACT_CASE(ACT_RELU2, act_slope)
        MUON_ACT_CASE(ACT_GELU, act_slope)
        MUON_ACT_CASE(ACT_GELU_TANH, act_slope)
        MUON_ACT_CASE(ACT_SILU, act_slope)
    }
}
#undef MUON_ACT_CASE

// Where a lane's chunk lies in each tensor from an element (row, column) that
// is the same for the whole wave: bytes, computed once, so that a chunk's
// address is a scalar one plus a register.
struct LaneAt {
    uint32_t y = 0, z = 0, add = 0;
    __device__ __forceinline__ LaneAt() {}
    // r rows down, c columns along
    __device__ __forceinline__ LaneAt(const Epilogue& E, int r, int c) {
        y = (uint32_t)(r * E.ld_y + c) * (E.mode == EPI_GRAD_WEIGHT ? 4u : 2u);
        z = (uint32_t)(r * E.ld_z + c) * 2u;
        add = (uint32_t)(r * E.ld_add + c) * 2u;
    }
};
template <typename U>
__device__ __forceinline__ U* chunk_at(const void* p, int64_t r, int ld, int64_t c, uint32_t lane) {
    return reinterpret_cast<U*>(const_cast<char*>(static_cast<const char*>(p)) + (r * ld + c) * (int64_t)sizeof(U) + lane);
}

// What the epilogue reads of a chunk of 8 outputs, fetched ahead of its use as
// 16-byte vectors: first8 is z on the way back through an activation, else
// add, or the lower half of a weight gradient to add to; second8 is add where
// first8 is z, or the upper half.
template <typename T>
__device__ __forceinline__ u32x4 first8(const Epilogue& E, int64_t r, int64_t c, const LaneAt& l) {
    const void* p = nullptr;
    if (E.mode == EPI_GRAD_WEIGHT) {
        if (E.accumulate) p = chunk_at<float>(E.y, r, E.ld_y, c, l.y);
    } else if (E.mode == EPI_GRAD_INPUT && E.act != ACT_NONE) {
        p = chunk_at<T>(E.z, r, E.ld_z, c, l.z);
    } else if (E.add) {
        p = chunk_at<T>(E.add, r, E.ld_add, c, l.add);
    }
    return p ? __builtin_nontemporal_load(static_cast<const u32x4_mem*>(p)) : u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ bool has_second(const Epilogue& E) {
    return E.mode == EPI_GRAD_WEIGHT ? E.accumulate != 0 : E.mode == EPI_GRAD_INPUT && E.act != ACT_NONE && E.add;
}
template <typename T>
__device__ __forceinline__ u32x4 second8(const Epilogue& E, int64_t r, int64_t c, const LaneAt& l) {
    const void* p = E.mode == EPI_GRAD_WEIGHT ? static_cast<const void*>(chunk_at<float>(E.y, r, E.ld_y, c, l.y) + 4)
                                              : static_cast<const void*>(chunk_at<T>(E.add, r, E.ld_add, c, l.add));
    return __builtin_nontemporal_load(static_cast<const u32x4_mem*>(p));
}

template <typename T>
__device__ __forceinline__ void widen8(const u32x4& u, float (&v)[8]) {
    const typename V8<T>::type t = __builtin_bit_cast(typename V8<T>::type, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)t[e];
}

// The epilogue of 8 consecutive accumulators from row r, column c (and the
// lane's place from there) on, n of them inside the matrix. bias: their bias
// values (forward). in, in2: first8's and second8's if n is 8 or more; a chunk at
// the matrix's edge is read in place.
template <typename T>
__device__ __forceinline__ void finish8(const Epilogue& E, int64_t r, int64_t c, const LaneAt& l, int n, float (&v)[8],
                                        const float (&bias)[8], const u32x4& in, const u32x4& in2) {
    float t[8];
    if (E.mode == EPI_GRAD_WEIGHT) {
        float* y = chunk_at<float>(E.y, r, E.ld_y, c, l.y);
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
        if (E.z) stream8(chunk_at<T>(E.z, r, E.ld_z, c, l.z), n, v);
        act_values(E.act, v);
    } else if (E.act != ACT_NONE) {
        fetched = true;
        if (n >= 8)
            widen8<T>(in, t);
        else
            load8(chunk_at<const T>(E.z, r, E.ld_z, c, l.z), n, t);
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
            load8(chunk_at<const T>(E.add, r, E.ld_add, c, l.add), n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += t[e];
    }
    stream8(chunk_at<T>(E.y, r, E.ld_y, c, l.y), n, v);
}

}  // namespace muon
