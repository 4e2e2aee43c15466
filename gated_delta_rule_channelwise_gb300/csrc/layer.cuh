// What the operators of cgdr_layer.h share: eight-value vectors and the 8-bit format.
#pragma once

#include "cgdr_layer.h"
#include "serve.cuh"

namespace cgdr {

constexpr int kGroup = 128;                           // values of a scale
inline int groups_of(int n) { return (n + kGroup - 1) / kGroup; }
// Whether no two of the n x H rows of d elements overlap (a broadcast tensor is no output).
inline bool disjoint(int64_t n, int64_t st, int64_t H, int64_t sh, int64_t d) {
    if (n <= 0 || H <= 0) return true;
    const bool tokens_inside = H == 1 || (n > 1 && st < sh);
    const int64_t ni = tokens_inside ? n : H, si = tokens_inside ? st : sh, no = tokens_inside ? H : n, so = tokens_inside ? sh : st;
    return (ni == 1 || si >= d) && (no == 1 || so >= (ni - 1) * si + d);
}

// Eight values of T, as loaded: 16 bytes, or two times 16.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const void *p) { r = __ldg(static_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void fetch(const void *p) { r = *static_cast<const uint4 *>(p); }    // of what the call writes, too
    __device__ __forceinline__ void clear() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void unpack(float (&f)[8]) const { Vec<__nv_bfloat16>::unpack(r, f); }
    static __device__ __forceinline__ void store(void *p, const float (&f)[8]) {
        *static_cast<uint4 *>(p) = Vec<__nv_bfloat16>::pack(f);
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const void *p) {
        a = __ldg(static_cast<const float4 *>(p));
        b = __ldg(static_cast<const float4 *>(p) + 1);
    }
    __device__ __forceinline__ void fetch(const void *p) {
        a = static_cast<const float4 *>(p)[0];
        b = static_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(void *p, const float (&f)[8]) {
        static_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// The bits of a magnitude order as integers do, a NaN's above all.
__device__ __forceinline__ uint32_t top_of(const float (&f)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    return top;
}
// The largest over the 16 lanes that hold a group of 128 (all of the warp's lanes call).
__device__ __forceinline__ uint32_t top_of_group(uint32_t top) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
}
__device__ __forceinline__ float scale_of(uint32_t top) {
    const float s = __uint_as_float(top) * (1.f / 448.f);
    return s < 0x1p-126f ? 0x1p-126f : s;             // a NaN stays one
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Eight values in 8 bits, by the reciprocal of their scale.
__device__ __forceinline__ uint2 e4m3x8(const float (&f)[8], float inverse) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = e4m3x2(__fmul_rn(f[2 * j], inverse), __fmul_rn(f[2 * j + 1], inverse));
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

}  // namespace cgdr
