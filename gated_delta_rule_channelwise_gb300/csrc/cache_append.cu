// Quantising append to the 8-bit cache (cgdr_cache_append).
//
// Bound by memory for prompts (k and v read once, a byte an element written) and by the launch for
// single tokens.  The unit of work is a run: consecutive packed tokens on consecutive slots of one
// page, for one head, of k or of v.  A block owns the run that begins at its token and with it the page's scale, so
// nothing is exchanged between blocks; a block whose token begins no run has nothing to do.  The
// run's largest magnitude has to be known before its first byte: the values are read for it, and
// again, from L1 or L2, to be rounded.
#include "serve.cuh"

namespace cgdr {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
    int n, Hkv, D, page, num_pages;
    const void *x[2];                                 // k, v
    int64_t st[2], sh[2], ex[2];                      // strides and footprints
    const int64_t *slots;
    int8_t *cache[2];
    float *scale[2];
    int *status;
};

// Largest magnitude; a NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float m, float x) { return x > m || x != x ? x : m; }

__device__ __forceinline__ int quantised(float x, float scale) {
    return min(max(__float2int_rn(__fdiv_rn(x, scale)), -127), 127);
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
    constexpr int V = Vec<T>::n;
    const int i = blockIdx.x, h = blockIdx.y, which = blockIdx.z, tid = threadIdx.x;
    const int64_t slot = p.slots[i];
    const int64_t slots = (int64_t)p.num_pages * p.page;
    if (slot < 0) return;
    if (slot >= slots) {
        if (tid == 0 && p.status != nullptr) atomicExch(p.status, (int)CGDR_ERR_BOUNDS);
        return;
    }
    const int off = (int)(slot % p.page);
    if (off > 0 && i > 0 && p.slots[i - 1] == slot - 1) return;       // inside a run

    __shared__ int s_len;
    __shared__ float s_max[kAppendThreads / 32];
    if (tid == 0) s_len = min(p.page - off, p.n - i);
    __syncthreads();
    // the run's length: up to the first token that is not on the next slot (a page has 128 at most)
    if (tid < min(p.page - off, p.n - i) && p.slots[i + tid] != slot + tid) atomicMin(&s_len, tid);
    __syncthreads();
    const int len = s_len;

    const int64_t unit = (slot / p.page) * p.Hkv + h;                 // the page's block of this head
    int8_t *dst = p.cache[which] + unit * p.page * p.D;
    const T *x = static_cast<const T *>(p.x[which]);
    const int per = p.D / V, vecs = len * per;
    auto vec = [&](int e, float (&f)[V]) {
        const int64_t at = (int64_t)(i + e / per) * p.st[which] + h * p.sh[which] + (e % per) * V;
        uint4 r = make_uint4(0, 0, 0, 0);
        if (range_in_bounds(at, V, p.ex[which], p.status, nullptr)) r = __ldg(reinterpret_cast<const uint4 *>(x + at));
        Vec<T>::unpack(r, f);
    };

    float top = 0.f;
    for (int e = tid; e < vecs; e += kAppendThreads) {
        float f[V];
        vec(e, f);
#pragma unroll
        for (int j = 0; j < V; ++j) top = max_nan(top, fabsf(f[j]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, d));
    if ((tid & 31) == 0) s_max[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) top = max_nan(top, s_max[w]);

    const float stored = p.scale[which][unit];
    const float had = off > 0 ? stored : 0.f;
    const float grown = max_nan(had, top * (1.f / 127.f));
    const float by = grown > 0.f ? grown : 1.f;       // nothing but zeros: any divisor gives them
    __syncthreads();                                  // every thread has read the scale that is replaced
    if (tid == 0) p.scale[which][unit] = grown;

    if (grown > had && off > 0) {                     // what the page holds, rounded to the larger scale
        for (int e = tid; e < off * p.D / 16; e += kAppendThreads) {
            uint4 r = reinterpret_cast<uint4 *>(dst)[e];
            uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t packed = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int q = (int8_t)(w[j] >> (8 * c));
                    packed |= (uint32_t)(quantised(__fmul_rn((float)q, had), by) & 0xFF) << (8 * c);
                }
                w[j] = packed;
            }
            reinterpret_cast<uint4 *>(dst)[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    for (int e = tid; e < vecs; e += kAppendThreads) {
        float f[V];
        vec(e, f);
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            w[j] = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) w[j] |= (uint32_t)(quantised(f[4 * j + c], by) & 0xFF) << (8 * c);
        }
        uint32_t *to = reinterpret_cast<uint32_t *>(dst + (int64_t)off * p.D + e * V);
        if (V == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[V / 4 - 1]);
        else *to = w[0];
    }
}

template <typename T>
cgdr_status launch_append(const AppendParams &p, cudaStream_t s) {
    cache_append_kernel<T><<<dim3(p.n, p.Hkv, 2), kAppendThreads, 0, s>>>(p);
    return launched();
}

cgdr_status check(const cgdr_append_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->n < 0 || a->Hkv <= 0 || a->num_pages < 0) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || !page_ok(a->page) || (a->D != 32 && a->D != 64 && a->D != 128)) return CGDR_ERR_UNSUPPORTED;
    if (a->n > kMaxTokens || a->Hkv > 65535) return CGDR_ERR_UNSUPPORTED;
    if (a->n == 0) return CGDR_OK;
    if (!a->k || !a->v || !a->slots || !a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale) return CGDR_ERR_INVALID_ARG;
    const int esz = esize(a->dtype);
    if (!aligned_to(a->k, 16) || !aligned_to(a->v, 16) || !aligned_to(a->k_cache, 16) || !aligned_to(a->v_cache, 16) ||
        !aligned_to(a->slots, 8) || !aligned_to(a->k_scale, 4) || !aligned_to(a->v_scale, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    if (!row_stride_ok(a->k_st, esz) || !row_stride_ok(a->k_sh, esz) || !row_stride_ok(a->v_st, esz) ||
        !row_stride_ok(a->v_sh, esz))
        return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

}  // namespace
}  // namespace cgdr

extern "C" cgdr_status cgdr_cache_append(const cgdr_append_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->n == 0) return st;
    AppendParams p{};
    p.n = a->n; p.Hkv = a->Hkv; p.D = a->D; p.page = a->page; p.num_pages = a->num_pages;
    p.x[0] = a->k; p.st[0] = a->k_st; p.sh[0] = a->k_sh; p.ex[0] = extent3(a->n, a->k_st, a->Hkv, a->k_sh, a->D);
    p.x[1] = a->v; p.st[1] = a->v_st; p.sh[1] = a->v_sh; p.ex[1] = extent3(a->n, a->v_st, a->Hkv, a->v_sh, a->D);
    p.slots = a->slots;
    p.cache[0] = a->k_cache; p.cache[1] = a->v_cache; p.scale[0] = a->k_scale; p.scale[1] = a->v_scale;
    p.status = a->status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == CGDR_BF16 ? launch_append<__nv_bfloat16>(p, s) : launch_append<float>(p, s);
}
