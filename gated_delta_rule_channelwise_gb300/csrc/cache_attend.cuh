// What the two attention kernels over the 8-bit cache share (cache_attend.cu: few query rows;
// cache_attend_prompt.cu: many).
#pragma once

#include "serve.cuh"

#include <cuda_fp16.h>

namespace cgdr {

struct AttendParams {
    int B, n, Hq, Hkv, G, tile, page, shift, width, num_pages, max_q, most;  // tile: rows of a tile, 8 or 16;
                                                       // most: cached tokens of a request at most
    float scale;
    const void *q;
    void *o;
    int64_t q_st, q_sh, o_st, o_sh, eq, eo, e_table;
    const int8_t *kc, *vc;
    const float *ks, *vs;
    const int32_t *table;
    int64_t table_sb;
    const int32_t *kv_lens, *cu;
    float *ml, *part;                                 // parts: [2 grid][tile][2] maximum and denominator, [2 grid][tile][D]
    int blocks, whole;                                // of the first kernel; nonzero: a block a unit, nothing split
    int splits, height;                               // parts of the cache, and rows of a part (cache_attend_prompt.cu)
    uint32_t polls;                                   // of a wait there
    int inject;                                       // test hook: its first wait of every block is on a barrier that nothing completes
    int *status;
};

constexpr int kBlockStep = 128;                       // cached tokens of a block's step in cache_attend.cu: its scheduling unit

// A request as the kernels see it.
struct Request {
    int first, q_len, kv, behind;                     // first query token, tokens, cached tokens, position of query token 0
    int units, steps;                                 // (row tile, head) pairs, block steps of each (cache_attend.cu)
};
__device__ __forceinline__ Request request(const AttendParams &p, int b) {
    const int2 span = seq_span(p.cu, b, p.n);
    const int len = span.y - span.x, kv = max(p.kv_lens[b], 0);
    Request r;
    r.first = span.x;
    r.q_len = min(len, p.max_q);
    r.kv = min(kv, p.most);
    r.behind = kv - len;
    r.units = (r.q_len * p.G + p.tile - 1) / p.tile * p.Hkv;
    r.steps = max((r.kv + kBlockStep - 1) / kBlockStep, 1);           // rows that see nothing are written, too
    return r;
}
__device__ __forceinline__ bool cut(const AttendParams &p, int b) {
    const int2 span = seq_span(p.cu, b, p.n);
    return span.y - span.x > p.max_q || p.kv_lens[b] > p.most;
}

__device__ __forceinline__ void report(int *status, int code) {
    if (status != nullptr) atomicExch(status, code);
}

constexpr float kUp = 8.f, kMost = 15.f;              // p' is carried times 2^kUp and stays below 2^kMost
constexpr float kLowest = -3e38f;                     // below every score: M before there is one
// Of a page whose v scale is below kZero the values are as good as zero, and p' only serves the denominator.  It is
// carried as if the scale were 2^kZeroLog: at 2^0 such a page would hold M up by -log2 vs over the others of its row and
// leave their p' no bits of fp16.  Not lower, so that 2^30 tokens of p' / 2^kZeroLog stay below 2^126.
constexpr float kZero = 0x1p-100f, kZeroLog = -80.f, kZeroInverse = -0x1p80f;     // below 0: p' is left out of p v
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two sign-flipped int8 in bytes 0 and 2 above exponent bytes -> their values as fp16.
__device__ __forceinline__ uint32_t less_bias(uint32_t x) {
    const uint32_t bias = 0x64806480u;                // 1152
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t low_pair(uint32_t w) { return less_bias(__byte_perm(w, 0x64646464u, 0x4140)); }
__device__ __forceinline__ uint32_t high_pair(uint32_t w) { return less_bias(__byte_perm(w, 0x64646464u, 0x4342)); }

// Four values of a row of o from a weighted sum and its denominator; a row that saw nothing is zero.
template <typename T>
__device__ __forceinline__ void put_row(const AttendParams &p, int tok, int head, int d, const float (&o)[4], float sum) {
    const int64_t off = (int64_t)tok * p.o_st + (int64_t)head * p.o_sh + d;
    const float by = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (in_bounds(off + e, p.eo, p.status, nullptr)) static_cast<T *>(p.o)[off + e] = Cvt<T>::from_f(sum == 0.f ? 0.f : o[e] * by);
}

// A second kernel that starts early waits here for the first.  Every thread does before it returns, so that
// what follows in the stream finds both kernels done.
__device__ __forceinline__ void joined() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Whether the tensor-core kernel takes the call, its workspace, and the call.
bool attend_prompt_supported(const cgdr_attend_args &a);
size_t attend_prompt_workspace(const cgdr_attend_args &a);
cgdr_status launch_attend_prompt(const cgdr_attend_args &a, AttendParams &p, float *ws, cudaStream_t s);

}  // namespace cgdr
