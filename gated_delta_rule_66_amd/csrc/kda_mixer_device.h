// Device helpers of the mixer operators.
#pragma once

#include "kda_device.h"

namespace kda {

// V consecutive elements of T kept raw: one access of 16 or 8 bytes, or V = 1.
template <typename T, int V> struct Vec {
    static_assert(V == 1 || V * sizeof(T) == 16 || V * sizeof(T) == 8, "one access");
    T v[V];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V * sizeof(T) == 16)
            *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
        else if constexpr (V * sizeof(T) == 8)
            *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
        else
            v[0] = *p;
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (V * sizeof(T) == 16)
            *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
        else if constexpr (V * sizeof(T) == 8)
            *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(v);
        else
            *p = v[0];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (T)0.f;
    }
    __device__ __forceinline__ float f(int i) const { return (float)v[i]; }
    __device__ __forceinline__ void set(int i, float x) { v[i] = from_f32<T>(x); }
};

// sigmoid: bf16 results take the hardware exp2 and reciprocal (1 ulp each,
// far below half a bf16 step); fp32 results take expf and a full division.
template <typename T> __device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (sizeof(T) == 2)
        return sigmoidf_fast(v);
    else
        return 1.f / (1.f + expf(-v));
}
// activation and derivative; act: 0 none, 1 silu, 2 sigmoid
template <typename T> __device__ __forceinline__ float act_of(float v, int act) {
    if (act == 0) return v;
    const float s = sigmoid_of<T>(v);
    return act == 1 ? v * s : s;
}
template <typename T> __device__ __forceinline__ float dact_of(float v, int act) {
    if (act == 0) return 1.f;
    const float s = sigmoid_of<T>(v);
    return act == 1 ? s * (1.f + v * (1.f - s)) : s * (1.f - s);
}

}  // namespace kda
