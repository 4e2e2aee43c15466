// What the operators of cgdr_layer.h share: eight-value vectors and the 8-bit format.
#pragma once

#include <utility>

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

// These kernels may be set up while the one before them in the stream ends: every thread waits for its results before it
// touches global memory.  What they read may be written while they are already there, so it is not read-only for as long as they live, as
// the read-only path (__ldg) asks: they read with ordinary loads, which stay behind the wait.  (No case was slower by that.)
__device__ __forceinline__ void wait_for_inputs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cgdr_status launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster, A &&...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster > 0 ? 2 : 1;
    if (cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...) == cudaSuccess) return CGDR_OK;
    cudaGetLastError();                               // (leaves no error behind in the library's runtime)
    return CGDR_ERR_CUDA;
}

// Eight values of T, as loaded (16 bytes, or two times 16) and as four pairs of fp32.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const void *p) { r = *static_cast<const uint4 *>(p); }
    __device__ __forceinline__ void clear() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void unpack(f32x2 (&f)[4]) const {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ void store(void *p, const f32x2 (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = split(f[i]);
            w[i] = pack_bf16x2(v.x, v.y);
        }
        *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<float> {
    ulonglong2 a, b;
    __device__ __forceinline__ void load(const void *p) {
        a = static_cast<const ulonglong2 *>(p)[0];
        b = static_cast<const ulonglong2 *>(p)[1];
    }
    __device__ __forceinline__ void clear() { a = b = make_ulonglong2(0, 0); }
    __device__ __forceinline__ void unpack(f32x2 (&f)[4]) const { f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; }
    static __device__ __forceinline__ void store(void *p, const f32x2 (&f)[4]) {
        static_cast<ulonglong2 *>(p)[0] = make_ulonglong2(f[0], f[1]);
        static_cast<ulonglong2 *>(p)[1] = make_ulonglong2(f[2], f[3]);
    }
};

// The largest of three, a NaN above all.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float top_of(const f32x2 (&f)[4], float top = 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = split(f[i]);
        top = max3_nan(top, fabsf(v.x), fabsf(v.y));
    }
    return top;
}
// The largest over the 16 lanes that hold a group of 128 (all of the warp's lanes call).
__device__ __forceinline__ float top_of_group(float top) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, top, o);
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(top) : "f"(top), "f"(x));
    }
    return top;
}
__device__ __forceinline__ float scale_of(float top) {
    float s;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(s) : "f"(top * (1.f / 448.f)), "f"(0x1p-126f));
    return s;
}
// Eight values in 8 bits, by the reciprocal of their scale.
__device__ __forceinline__ uint2 e4m3x8(const f32x2 (&f)[4], float inverse) {
    uint16_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = split(mul2(f[i], both(inverse)));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w[i]) : "f"(v.y), "f"(v.x));
    }
    uint2 r;
    asm("mov.b32 %0, {%1, %2};" : "=r"(r.x) : "h"(w[0]), "h"(w[1]));
    asm("mov.b32 %0, {%1, %2};" : "=r"(r.y) : "h"(w[2]), "h"(w[3]));
    return r;
}

}  // namespace cgdr
