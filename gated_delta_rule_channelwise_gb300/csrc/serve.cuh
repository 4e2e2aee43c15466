// What the serving operators (cgdr_serve.h) share: argument checks, 8-element vectors of the
// input types, packed-sequence lookups and fast elementary functions.
#pragma once

#include "cgdr_internal.cuh"
#include "cgdr_serve.h"

namespace cgdr {

inline bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Row strides of a vector-loaded tensor: not negative, a multiple of 16 bytes.
inline bool row_stride_ok(int64_t s, int esz) { return s >= 0 && s % (16 / esz) == 0; }
inline int esize(int dtype) { return dtype == CGDR_BF16 ? 2 : 4; }
inline bool dtype_ok(int dtype) { return dtype == CGDR_F32 || dtype == CGDR_BF16; }
constexpr int64_t kMaxTokens = 1 << 30;               // token indices stay well inside 32 bits
inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
inline cgdr_status launched() { return cudaGetLastError() == cudaSuccess ? CGDR_OK : CGDR_ERR_CUDA; }
// Elements from a tensor's first to its last, rows x ... with the given strides; 0 for no rows.
inline int64_t extent3(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t d) {
    return n0 <= 0 || n1 <= 0 ? 0 : (n0 - 1) * s0 + (n1 - 1) * s1 + d;
}

template <typename T> struct Vec;   // 16 bytes of T
template <> struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(const uint4 &r, float *f) {
        f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(const uint4 &r, float *f) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *f) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// First and one-past-last packed token of sequence b, clamped to [0, n] and not descending.
__device__ __forceinline__ int2 seq_span(const int32_t *cu, int b, int n) {
    const int lo = min(max(cu[b], 0), n);
    return make_int2(lo, min(max(cu[b + 1], lo), n));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;
// x / (1 + e^-x); where e^-x overflows the reciprocal is 0 and the result -0, as the quotient's is.
__device__ __forceinline__ float silu_f(float x) { return x * rcp(1.f + ex2(-kLog2e * x)); }

// Pairs of fp32 in a 64-bit register: one instruction for two multiply-adds (the arithmetic rate
// is that of two, the issue slot is saved).
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 both(float x) { return pair(x, x); }

__device__ __forceinline__ f32x2 silu_pair(f32x2 x) {
    const float2 m = split(mul2(x, both(-kLog2e)));
    const float2 w = split(add2(pair(ex2(m.x), ex2(m.y)), both(1.f)));
    return mul2(x, pair(rcp(w.x), rcp(w.y)));
}

}  // namespace cgdr
