// wq_logits.cuh -- reading logits of three element types, and the order of the top entries.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/wq.h"

namespace wq {

template <int TYPE> struct Logit;
template <> struct Logit<WQ_TYPE_F32> {
    using raw = float;
    static __device__ __forceinline__ float load(const raw* p) { return *p; }
};
template <> struct Logit<WQ_TYPE_F16> {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(const raw* p) { return __half2float(__ushort_as_half(*p)); }
};
template <> struct Logit<WQ_TYPE_BF16> {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(const raw* p) { return __uint_as_float((uint32_t)*p << 16); }
};

// Unsigned key in the order of the values; NaN orders as -inf and -0 as +0.
constexpr uint32_t KEY_NEG_INF = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(fmaxf(v, -INFINITY) + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// 2^v, v <= 0 here, to 2 units in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
constexpr float LOG2E = 1.4426950408889634f;

}  // namespace wq
