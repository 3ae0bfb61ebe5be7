// Element types, conversions and activations shared by the neural decoder's kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gsmi.h"

namespace gsmi {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float f16_to_f32(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
// rounds to nearest, ties to even
__device__ __forceinline__ uint16_t f32_to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t f32_to_f16(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

// 16 and 8 bytes at any address that is a multiple of the element: one wide access where the hardware has it.
__device__ __forceinline__ u32x4 load16(const void* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// Element i of an array whose type is known at run time (uniform over the launch).
__device__ __forceinline__ float load_elem(const void* p, int type, int64_t i) {
    if (type == GS_TYPE_F32) return static_cast<const float*>(p)[i];
    const uint16_t v = static_cast<const uint16_t*>(p)[i];
    return type == GS_TYPE_BF16 ? bf16_to_f32(v) : f16_to_f32(v);
}
__device__ __forceinline__ void store_elem(void* p, int type, int64_t i, float v) {
    if (type == GS_TYPE_F32)
        static_cast<float*>(p)[i] = v;
    else
        static_cast<uint16_t*>(p)[i] = type == GS_TYPE_BF16 ? f32_to_bf16(v) : f32_to_f16(v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, int type) {
    return type == GS_TYPE_BF16 ? (uint32_t)f32_to_bf16(a) | (uint32_t)f32_to_bf16(b) << 16
                                : (uint32_t)f32_to_f16(a) | (uint32_t)f32_to_f16(b) << 16;
}
// Four or eight consecutive elements from i on.
__device__ __forceinline__ f32x4 load_elem4(const void* p, int type, int64_t i) {
    if (type == GS_TYPE_F32) return __builtin_bit_cast(f32x4, load16(static_cast<const float*>(p) + i));
    u32x2 v;
    __builtin_memcpy(&v, static_cast<const uint16_t*>(p) + i, 8);
    f32x4 r;
    for (int k = 0; k < 4; k++) {
        const uint16_t h = (uint16_t)(v[k >> 1] >> ((k & 1) * 16));
        r[k] = type == GS_TYPE_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
    }
    return r;
}
__device__ __forceinline__ void store_elem4(void* p, int type, int64_t i, f32x4 v) {
    if (type == GS_TYPE_F32) {
        store16(static_cast<float*>(p) + i, __builtin_bit_cast(u32x4, v));
        return;
    }
    const u32x2 o = {pack2(v[0], v[1], type), pack2(v[2], v[3], type)};
    __builtin_memcpy(static_cast<uint16_t*>(p) + i, &o, 8);
}
__device__ __forceinline__ void load_elem8(const void* p, int type, int64_t i, float (&v)[8]) {
    if (type == GS_TYPE_F32) {
        const f32x4 a = load_elem4(p, type, i), b = load_elem4(p, type, i + 4);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            v[k] = a[k];
            v[4 + k] = b[k];
        }
    } else {
        const u32x4 w = load16(static_cast<const uint16_t*>(p) + i);
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const uint16_t h = (uint16_t)(w[k >> 1] >> ((k & 1) * 16));
            v[k] = type == GS_TYPE_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
        }
    }
}
__device__ __forceinline__ void store_elem8(void* p, int type, int64_t i, const float (&v)[8]) {
    if (type == GS_TYPE_F32) {
        store_elem4(p, type, i, f32x4{v[0], v[1], v[2], v[3]});
        store_elem4(p, type, i + 4, f32x4{v[4], v[5], v[6], v[7]});
    } else {
        store16(static_cast<uint16_t*>(p) + i,
                u32x4{pack2(v[0], v[1], type), pack2(v[2], v[3], type), pack2(v[4], v[5], type), pack2(v[6], v[7], type)});
    }
}

// 1 / (1 + e^-z): the reciprocal of infinity is 0, so large negative z give 0.
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

// relu keeps NaN; gelu is z Phi(z) with the error function.
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case GS_ACT_RELU: return z < 0.0f ? 0.0f : z;
        case GS_ACT_SILU: return z * sigmoid(z);
        case GS_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        default: return z;
    }
}
// value and derivative
__device__ __forceinline__ void act_both(float z, int act, float& v, float& d) {
    switch (act) {
        case GS_ACT_RELU:
            v = z < 0.0f ? 0.0f : z;
            d = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
            return;
        case GS_ACT_SILU: {
            const float p = sigmoid(z);
            v = z * p;
            d = p * fmaf(z, 1.0f - p, 1.0f);
            return;
        }
        case GS_ACT_GELU: {
            const float c = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
            v = z * c;
            d = fmaf(z, __expf(-0.5f * z * z) * 0.39894228040143268f, c);
            return;
        }
        default:
            v = z;
            d = 1.0f;
    }
}

// Eight values at once: the choice of the activation is made once.
template <int ACT>
__device__ __forceinline__ void act8_of(float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; k++) v[k] = act_value(v[k], ACT);
}
__device__ __forceinline__ void act8(float (&v)[8], int act) {
    if (act == GS_ACT_SILU)
        act8_of<GS_ACT_SILU>(v);
    else if (act == GS_ACT_GELU)
        act8_of<GS_ACT_GELU>(v);
    else if (act == GS_ACT_RELU)
        act8_of<GS_ACT_RELU>(v);
}
// v becomes the activation's value, d its derivative.
template <int ACT>
__device__ __forceinline__ void act8_both_of(float (&v)[8], float (&d)[8]) {
#pragma unroll
    for (int k = 0; k < 8; k++) {
        float a;
        act_both(v[k], ACT, a, d[k]);
        v[k] = a;
    }
}
__device__ __forceinline__ void act8_both(float (&v)[8], float (&d)[8], int act) {
    if (act == GS_ACT_SILU)
        act8_both_of<GS_ACT_SILU>(v, d);
    else if (act == GS_ACT_GELU)
        act8_both_of<GS_ACT_GELU>(v, d);
    else if (act == GS_ACT_RELU)
        act8_both_of<GS_ACT_RELU>(v, d);
    else
        act8_both_of<GS_ACT_NONE>(v, d);
}

}  // namespace gsmi
