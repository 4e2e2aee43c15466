// Quantising append to the 8-bit cache (cgdr_cache_append).
//
// Single tokens are bound by the launch (64 tokens of 8 heads of 128: 3.0 us), prompts by the chain that every
// run goes through, once: slots, values, their largest magnitude, bytes.  2 x 128 values of 8 heads of 4,000
// tokens, 24.6 MB, take 10.0 us; their bytes alone are 3.7 us, the 28 instructions that a value took once were 14.
// The unit of work is a run: consecutive packed tokens on consecutive slots of one
// page, for one head, of k or of v.  Whoever has a run has its page's scale, so nothing is exchanged
// between blocks.  A block finds the runs that begin in its window of tokens: few of them (a prompt)
// it works on one after the other with all its threads, many (single tokens) a warp each.  The
// largest magnitude has to be known before the first byte: a thread keeps the first two vectors that it
// reads and reads the rest again, from L1 or L2 (one / four / eight kept: 5 / 9 / 7 % slower; 256 threads are as fast
// on pages of 64 and take 2.8 times as long on pages of 16).
// The quotient is only formed where its rounding is in doubt: x (1 / scale) is within 3e-5 of it.
#include "serve.cuh"

namespace cgdr {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
    int n, Hkv, D, page, num_pages, window;
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

// Four values as bytes of round(x / by), |x / by| <= 127.  Adding 1.5 2^23 rounds the product with the
// reciprocal to the nearest integer, ties to even, in the low bits; product and quotient are rounded
// from values 127 2^-23 apart at most, so where the product is 1e-4 off a tie the quotient rounds the same.
__device__ __forceinline__ uint32_t quantised4(f32x2 x, f32x2 y, float by, f32x2 inverse, bool sure) {
    constexpr float kMagic = 12582912.f;
    const f32x2 tx = mul2(x, inverse), ty = mul2(y, inverse), rx = add2(tx, both(kMagic)), ry = add2(ty, both(kMagic));
    const float2 bx = split(rx), ry2 = split(ry);
    const float2 ex = split(fma2(add2(rx, both(-kMagic)), both(-1.f), tx)), ey = split(fma2(add2(ry, both(-kMagic)), both(-1.f), ty));
    uint32_t b[4] = {__float_as_uint(bx.x), __float_as_uint(bx.y), __float_as_uint(ry2.x), __float_as_uint(ry2.y)};
    const float off = fmaxf(fmaxf(fabsf(ex.x), fabsf(ex.y)), fmaxf(fabsf(ey.x), fabsf(ey.y)));
    if (!sure || off > 0.5f - 1e-4f) {
        const float2 fx = split(x), fy = split(y);
        const float f[4] = {fx.x, fx.y, fy.x, fy.y};
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = (uint32_t)quantised(f[c], by);
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// The largest magnitude as bits, which order as integers do, a NaN above all: two bf16 to a word, or one fp32.
template <typename T> __device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w);
template <> __device__ __forceinline__ uint32_t larger<float>(uint32_t top, uint32_t w) { return max(top, w & 0x7FFFFFFFu); }
template <> __device__ __forceinline__ uint32_t larger<__nv_bfloat16>(uint32_t top, uint32_t w) { return __vmaxu2(top, w & 0x7FFF7FFFu); }

// One run by a warp, or (kBlock) by the block: tokens from i on into the page of `slot` from its offset on, up to the
// first token that is not on the next slot.  The values that a run of the greatest length would have are
// asked for before its length is known.
template <typename T, bool kBlock>
__device__ __forceinline__ void append_run(const AppendParams &p, int i, int64_t slot, int h, int which, uint32_t *s_max) {
    constexpr int V = Vec<T>::n, NT = kBlock ? kAppendThreads : 32, kKeep = 2;
    const int tid = kBlock ? threadIdx.x : threadIdx.x & 31;
    const int off = (int)(slot % p.page);
    const int64_t unit = (slot / p.page) * p.Hkv + h;                 // the page's block of this head
    int8_t *dst = p.cache[which] + unit * p.page * p.D;
    const T *x = static_cast<const T *>(p.x[which]);
    const int per = p.D / V, shift = 31 - __clz(per);                 // vectors of a token: a power of two
    const int most = min(p.page - off, p.n - i);                      // a page has 128 tokens at most
    const int64_t head = h * p.sh[which];
    auto vec = [&](int e) {
        const int64_t at = (int64_t)(i + (e >> shift)) * p.st[which] + head + (e & (per - 1)) * V;
        return range_in_bounds(at, V, p.ex[which], p.status, nullptr) ? __ldg(reinterpret_cast<const uint4 *>(x + at))
                                                                      : make_uint4(0, 0, 0, 0);
    };
    const float had = off > 0 ? p.scale[which][unit] : 0.f;

    uint4 kept[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) kept[k] = tid + k * NT < most * per ? vec(tid + k * NT) : make_uint4(0, 0, 0, 0);
    int len = most;
#pragma unroll
    for (int k = 3; k >= 0; --k) {
        const int t = (tid & 31) + 32 * k;
        if (t < most && p.slots[i + t] != slot + t) len = t;
    }
    len = __reduce_min_sync(0xffffffffu, len);
    const int vecs = len * per;
    uint32_t top = 0;
    auto over = [&](const uint4 &r) { top = larger<T>(larger<T>(larger<T>(larger<T>(top, r.x), r.y), r.z), r.w); };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
        if (tid + k * NT < vecs) over(kept[k]);
    for (int e = tid + kKeep * NT; e < vecs; e += NT) over(vec(e));
    if (V == 8) top = max(top << 16, top & 0xFFFF0000u);
    top = __reduce_max_sync(0xffffffffu, top);
    if (kBlock) {
        if ((tid & 31) == 0) s_max[tid >> 5] = top;
        __syncthreads();                              // also: every thread has read the scale that is replaced
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w) top = max(top, s_max[w]);
    }
    const float grown = max_nan(had, __uint_as_float(top) * (1.f / 127.f));
    const float by = grown > 0.f ? grown : 1.f;       // nothing but zeros: any divisor gives them
    const float inverse = __frcp_rn(by);
    const bool sure = grown > 0x1p-100f && grown < INFINITY;          // and not a NaN: 1 / by is as exact as numbers get
    if (!kBlock) __syncwarp();
    if (tid == 0) p.scale[which][unit] = grown;

    if (grown > had && off > 0) {                     // what the page holds, rounded to the larger scale
        for (int e = tid; e < off * p.D / 16; e += NT) {
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
    auto put = [&](int e, const uint4 &r) {
        float f[V];
        Vec<T>::unpack(r, f);
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            w[j] = quantised4(pair(f[4 * j], f[4 * j + 1]), pair(f[4 * j + 2], f[4 * j + 3]), by, both(inverse), sure);
        uint32_t *to = reinterpret_cast<uint32_t *>(dst + (int64_t)off * p.D + e * V);
        if (V == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(w[0], w[V / 4 - 1]);
        else *to = w[0];
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
        if (tid + k * NT < vecs) put(tid + k * NT, kept[k]);
    for (int e = tid + kKeep * NT; e < vecs; e += NT) put(e, vec(e));
    if (kBlock) __syncthreads();                      // s_max is free again
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, 6) cache_append_kernel(const AppendParams p) {
    constexpr int NW = kAppendThreads / 32;
    __shared__ int s_start[kAppendThreads], s_count;
    __shared__ int64_t s_slot[kAppendThreads];
    __shared__ uint32_t s_max[NW];
    const int tid = threadIdx.x, warp = tid >> 5, h = blockIdx.y, which = blockIdx.z;
    const int i0 = blockIdx.x * p.window;
    const int64_t slots = (int64_t)p.num_pages * p.page;
    if (tid == 0) s_count = 0;
    __syncthreads();
    if (tid < p.window && i0 + tid < p.n) {
        const int i = i0 + tid;
        const int64_t slot = p.slots[i];
        if (slot >= slots && h == 0 && which == 0 && p.status != nullptr) atomicExch(p.status, (int)CGDR_ERR_BOUNDS);
        // a run begins where a page does, or where the token before is on another slot
        if (slot >= 0 && slot < slots && (slot % p.page == 0 || i == 0 || p.slots[i - 1] != slot - 1))
        {
            const int at = atomicAdd(&s_count, 1);    // in any order: runs share nothing
            s_start[at] = i;
            s_slot[at] = slot;
        }
    }
    __syncthreads();
    const int runs = s_count;
    const bool alone = runs < NW;                     // the block on one run at a time
    for (int r = alone ? 0 : warp; r < runs; r += alone ? 1 : NW) {
        const int i = s_start[r];
        const int64_t slot = s_slot[r];
        if (alone) append_run<T, true>(p, i, slot, h, which, s_max);
        else append_run<T, false>(p, i, slot, h, which, s_max);
    }
}

// Tokens of a block's window: four where there are few tokens, a warp for each; up to 64 (a prompt's window then
// holds a run or two), as long as there are four blocks to an SM.  Up to 32 instead: the same on pages of 64, two
// thirds more time on pages of 16.
template <typename T>
cgdr_status launch_append(AppendParams &p, cudaStream_t s) {
    const int sms = device_sms();
    if (sms <= 0) return CGDR_ERR_CUDA;
    const int64_t units = 2 * (int64_t)p.Hkv;
    p.window = kAppendThreads / 32;
    while (p.window < 64 && p.n * units >= 8 * (int64_t)sms * p.window) p.window *= 2;
    cache_append_kernel<T><<<dim3((p.n + p.window - 1) / p.window, p.Hkv, 2), kAppendThreads, 0, s>>>(p);
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
