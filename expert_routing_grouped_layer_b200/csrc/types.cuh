// types.cuh -- element types of the row operators: 16-byte and single-element access
// of bf16, f16 and fp32 rows, always widened to fp32 for arithmetic.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace moe {

// exp(x) and 1 / x by one special-function operation each, subnormal results as zero: within
// 2^-22 + |x| 2^-23 and 2^-23 of the value.
__device__ __forceinline__ float exp_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T>
__host__ __device__ constexpr bool is_half() { return false; }
template <>
__host__ __device__ constexpr bool is_half<__half>() { return true; }

// VEC consecutive elements, moved by one access where they fill 16 bytes.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T>
constexpr int kFullVec = 16 / (int)sizeof(T);

// Two fp32 values in a 64-bit register pair, and the packed operations on them (one
// instruction for both).
typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
    const float2 f = unpack2(v);
    return f.x + f.y;
}

// 16 bytes of T as pairs of fp32, and back (one rounding).
template <typename T>
constexpr int kPairs = 8 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ void widen(const uint4& u, f32x2 (&v)[kPairs<T>]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) {
        v[0] = pack2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        v[1] = pack2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (is_half<T>()) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[i] = pack2(f.x, f.y);
            } else {
                v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 narrow(const f32x2 (&v)[kPairs<T>]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
        const float2 a = unpack2(v[0]), b = unpack2(v[1]);
        w[0] = __float_as_uint(a.x); w[1] = __float_as_uint(a.y);
        w[2] = __float_as_uint(b.x); w[3] = __float_as_uint(b.y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(v[i]);
            if constexpr (is_half<T>()) {
                const __half2 h = __floats2half2_rn(f.x, f.y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four fp32 values rounded to a 16-bit type, packed.
template <typename T>
__device__ __forceinline__ uint2 narrow4(const float (&v)[4]) {
    uint2 r;
    if constexpr (is_half<T>()) {
        const __half2 a = __floats2half2_rn(v[0], v[1]), b = __floats2half2_rn(v[2], v[3]);
        r.x = *reinterpret_cast<const uint32_t*>(&a);
        r.y = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        r.x = *reinterpret_cast<const uint32_t*>(&a);
        r.y = *reinterpret_cast<const uint32_t*>(&b);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ uint4 narrow8(const float* v) {
    const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
    const uint2 x = narrow4<T>(a), y = narrow4<T>(b);
    return make_uint4(x.x, x.y, y.x, y.y);
}

// Rows of es-byte elements that 16-byte accesses reach; true for a matrix that is not there.
inline bool rows16(const void* p, long ld, int es) {
    return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * es) % 16 == 0);
}

}  // namespace moe
