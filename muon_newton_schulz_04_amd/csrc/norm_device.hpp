// Device helpers of the norms: sums over the lanes that share a row, and chunks
// of 8 elements kept as they were loaded.
#pragma once

#include "layer_device.hpp"

namespace muon {

// One step of a wave sum: v + v moved by a DPP control, 0 from outside.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
}
// Wave-wide sum in the vector unit: within rows of 16 lanes by shifts, then
// across them by the row broadcasts; lane 63 holds it.
__device__ __forceinline__ float wave_total(float v) {
    v = dpp_add<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);  // row_bcast 15 into rows 1, 3
    v = dpp_add<0x143, 0xc>(v);  // row_bcast 31 into rows 2, 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums over the lanes that share a row: a wave, or WPR neighbouring waves of
// the workgroup, all of which call it. red: two floats a wave; calls in turn
// use two such buffers, so that one barrier a call orders them.
template <int WPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float* red) {
    a = wave_total(a);
    b = wave_total(b);
    if constexpr (WPR > 1) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        if (lane == 0) {
            red[2 * wave] = a;
            red[2 * wave + 1] = b;
        }
        __syncthreads();
        const float* r = red + wave / WPR * WPR * 2;
        a = r[0];
        b = r[1];
#pragma unroll
        for (int w = 1; w < WPR; ++w) {
            a += r[2 * w];
            b += r[2 * w + 1];
        }
    }
}
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
    float none = 0.f;
    row_sum2<WPR>(v, none, red);
    return v;
}

// A chunk of 8 elements as loaded.
template <typename T>
struct Raw {
    uint32_t w[sizeof(T) * 2];
    // n of the elements exist, the others are 0. VEC: n is 8 or more, or none
    template <bool VEC>
    __device__ __forceinline__ void load(const T* __restrict__ p, int n) {
        if (VEC && n <= 0) {
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) * 2; ++k) w[k] = 0;
        } else if (VEC || n >= 8) {
            const u32x4_mem* q = reinterpret_cast<const u32x4_mem*>(p);
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
                const u32x4 t = q[k];
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * k + e] = t[e];
            }
        } else {
            T t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = e < n ? p[e] : (T)0.f;
            __builtin_memcpy(w, t, sizeof(w));
        }
    }
    // the elements from n on become v
    __device__ __forceinline__ void fill(int n, T v) {
        constexpr int PER = 4 / sizeof(T);
        uint32_t u = 0;
        __builtin_memcpy(&u, &v, sizeof(T));
        if constexpr (PER == 2) u |= u << 16;
#pragma unroll
        for (int k = 0; k < 8 / PER; ++k) {
            if (PER * k >= n)
                w[k] = u;
            else if (PER * k + 1 >= n && PER == 2)
                w[k] = (w[k] & 0xffffu) | (u & 0xffff0000u);
        }
    }
    // the compiler takes the words as new: it widens them again rather than
    // keep the float values across
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) * 2; ++k) asm volatile("" : "+v"(w[k]));
    }
    // 8 values rounded once to T
    __device__ __forceinline__ void put(const float (&v)[8]) {
        f32x8 t;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = v[e];
        const typename V8<T>::type u = __builtin_convertvector(t, typename V8<T>::type);
        __builtin_memcpy(w, &u, sizeof(w));
    }
    // all 8 elements to p
    __device__ __forceinline__ void store(T* __restrict__ p) const {
        u32x4_mem* q = reinterpret_cast<u32x4_mem*>(p);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            __builtin_nontemporal_store(u32x4{w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]}, q + k);
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[e]);
        } else {
            T t;
            const uint16_t u = (uint16_t)(w[e / 2] >> (e % 2 * 16));
            __builtin_memcpy(&t, &u, 2);
            return (float)t;
        }
    }
};

}  // namespace muon
