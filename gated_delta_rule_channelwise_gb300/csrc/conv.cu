// Short causal convolution (cgdr_conv): y[t] = act(bias + sum_j w[j] u[t - (W-1) + j]) per channel,
// u = the W-1 state rows followed by the sequence.
//
// Bound by memory: each x is read once and each y written once, 2 W + 4 operations per element.
// A thread owns 16 bytes of channels and walks along the tokens with the last W-1 rows in
// registers, so a row is loaded once per tile of tokens (plus W-1 rows where a tile begins).
// Tiles cut the packed token axis without regard to the sequences, which keeps ragged batches
// balanced; a tile that meets a sequence's first token takes over that sequence's state: it reads
// the old rows, writes the new ones (the sequence's last rows, read directly), and also computes the
// sequence's tokens up to number W-2, so that no other tile ever reads the state that it replaces.
#include "serve.cuh"

namespace cgdr {
namespace {

struct ConvParams {
    int B, T, C, n, tile;
    const void *x;
    void *o;
    int64_t x_sb, x_st, o_sb, o_st;
    const float *weight, *bias;
    void *state;
    const int32_t *cu;
    int *status;
    int64_t ex, eo, es;                               // footprints (index-checking build)
};

constexpr int kConvThreads = 128;
constexpr int kConvBatch = 4;                         // rows in flight per thread, next to the four computed on

template <typename T>
__device__ __forceinline__ uint4 load_vec(const T *p, int64_t off, int64_t n, int *st) {
    return range_in_bounds(off, Vec<T>::n, n, st, nullptr) ? __ldg(reinterpret_cast<const uint4 *>(p + off))
                                                           : make_uint4(0, 0, 0, 0);
}
// The state is written by the kernel that reads it: an ordinary load.
template <typename T>
__device__ __forceinline__ uint4 load_state(const T *p, int64_t off, int64_t n, int *st) {
    return range_in_bounds(off, Vec<T>::n, n, st, nullptr) ? *reinterpret_cast<const uint4 *>(p + off) : make_uint4(0, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ void store_vec(T *p, int64_t off, const uint4 &v, int64_t n, int *st) {
    if (range_in_bounds(off, Vec<T>::n, n, st, nullptr)) *reinterpret_cast<uint4 *>(p + off) = v;
}

template <int W, int V>
__device__ __forceinline__ void load_filter(const ConvParams &p, int c0, float (&w)[W][V], float (&bias)[V]) {
    float flat[W * V];
#pragma unroll
    for (int i = 0; i < W * V / 4; ++i)
        *reinterpret_cast<float4 *>(flat + 4 * i) = __ldg(reinterpret_cast<const float4 *>(p.weight + (int64_t)c0 * W) + i);
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) w[j][e] = flat[e * W + j];
#pragma unroll
    for (int e = 0; e < V; ++e) bias[e] = p.bias != nullptr ? __ldg(p.bias + c0 + e) : 0.f;
}

// One row: the window's W-1 rows and `now` give y; the window moves on.
template <typename T, int W, bool kSilu>
__device__ __forceinline__ uint4 conv_row(const float (&w)[W][Vec<T>::n], const float (&bias)[Vec<T>::n], uint4 (&win)[W - 1],
                                          const uint4 &now) {
    constexpr int V = Vec<T>::n;
    float acc[V], f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        Vec<T>::unpack(j < W - 1 ? win[j] : now, f);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(w[j][e], f[e], acc[e]);
    }
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
    win[W - 2] = now;
    if (kSilu) {
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = silu_f(acc[e]);
    }
    return Vec<T>::pack(acc);
}

struct Place {
    int b, pos, len;                                  // sequence (B: past the last token), place in it, its length
};
__device__ __forceinline__ Place place_of(const ConvParams &p, int i) {
    if (p.cu == nullptr) return i < p.n ? Place{i / p.T, i % p.T, p.T} : Place{p.B, 0, 0};
    int lo = 0, hi = p.B;                             // the first b with cu[b + 1] > i
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid + 1) > i) hi = mid;
        else lo = mid + 1;
    }
    if (lo >= p.B) return Place{p.B, 0, 0};
    const int2 s = seq_span(p.cu, lo, p.n);
    return Place{lo, max(i - s.x, 0), s.y - s.x};
}
// Where the tile that would begin at token i really begins: tokens 1 .. W-2 of a sequence belong to
// the tile that has its token 0.
template <int W>
__device__ __forceinline__ int tile_begin(const ConvParams &p, int i, Place &at) {
    at = place_of(p, i);
    if (at.b < p.B && at.pos > 0 && at.pos < W - 1) {
        i += min(W - 1, at.len) - at.pos;
        at = place_of(p, i);
    }
    return i;
}

template <typename T, int W, bool kSilu>
__global__ void __launch_bounds__(kConvThreads) conv_tokens_kernel(const ConvParams p) {
    constexpr int V = Vec<T>::n, U = kConvBatch;
    const int c0 = (blockIdx.x * kConvThreads + threadIdx.x) * V;
    if (c0 >= p.C) return;
    const T *x = static_cast<const T *>(p.x);
    T *o = static_cast<T *>(p.o), *state = static_cast<T *>(p.state);
    Place at, after;
    const int end0 = min((blockIdx.y + 1) * p.tile, p.n);
    const int end = end0 < p.n ? tile_begin<W>(p, end0, after) : p.n;
    int i = tile_begin<W>(p, blockIdx.y * p.tile, at);
    if (i >= end || at.b >= p.B) return;

    auto x_off = [&](int t) -> int64_t {
        return (p.cu == nullptr ? (t / p.T) * p.x_sb + (t % p.T) * p.x_st : t * p.x_st) + c0;
    };
    auto o_off = [&](int t) -> int64_t {
        return (p.cu == nullptr ? (t / p.T) * p.o_sb + (t % p.T) * p.o_st : t * p.o_st) + c0;
    };
    auto row = [&](int t) { return load_vec<T>(x, x_off(t), p.ex, p.status); };

    uint4 next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = i + u < end ? row(i + u) : make_uint4(0, 0, 0, 0);
    float w[W][V], bias[V];
    load_filter<W, V>(p, c0, w, bias);
    uint4 win[W - 1];
    if (at.pos > 0) {                                 // at least W-1 of the sequence's rows precede
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j] = row(i - (W - 1) + j);
    }
    while (i < end) {
        uint4 cur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            cur[u] = next[u];
            next[u] = i + U + u < end ? row(i + U + u) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i + u < end && at.b < p.B) {
                if (at.pos == 0) {                    // a sequence begins: its state in, its last rows out
                    const int64_t s0 = (int64_t)at.b * (W - 1) * p.C + c0;
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) win[j] = load_state<T>(state, s0 + (int64_t)j * p.C, p.es, p.status);
                    uint4 last[W - 1];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        const int k = at.len + j;     // row k of u: state rows first
                        last[j] = win[W - 2];
#pragma unroll
                        for (int m = 0; m < W - 1; ++m)
                            if (k == m) last[j] = win[m];
                        if (k >= W - 1) last[j] = row(i + u + k - (W - 1));
                    }
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) store_vec<T>(state, s0 + (int64_t)j * p.C, last[j], p.es, p.status);
                }
                store_vec<T>(o, o_off(i + u), conv_row<T, W, kSilu>(w, bias, win, cur[u]), p.eo, p.status);
                if (++at.pos >= at.len && i + u + 1 < end) at = place_of(p, i + u + 1);
            }
        }
        i += U;
    }
}

// One token a sequence: a thread owns 16 bytes of channels of one sequence.
template <typename T, int W, bool kSilu>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvParams p) {
    constexpr int V = Vec<T>::n;
    const int c0 = (blockIdx.x * kConvThreads + threadIdx.x) * V;
    const int b = blockIdx.y;
    if (c0 >= p.C) return;
    const T *x = static_cast<const T *>(p.x);
    T *o = static_cast<T *>(p.o), *state = static_cast<T *>(p.state);
    const int64_t s0 = (int64_t)b * (W - 1) * p.C + c0;
    const uint4 now = load_vec<T>(x, b * p.x_sb + c0, p.ex, p.status);
    uint4 win[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = load_state<T>(state, s0 + (int64_t)j * p.C, p.es, p.status);
    float w[W][V], bias[V];
    load_filter<W, V>(p, c0, w, bias);
    const uint4 y = conv_row<T, W, kSilu>(w, bias, win, now);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_vec<T>(state, s0 + (int64_t)j * p.C, win[j], p.es, p.status);
    store_vec<T>(o, b * p.o_sb + c0, y, p.eo, p.status);
}

template <typename T, int W, bool kSilu>
cgdr_status launch_tokens(const cgdr_conv_args &a, ConvParams &p, cudaStream_t s) {
    const int vecs = a.C / Vec<T>::n, gx = (vecs + kConvThreads - 1) / kConvThreads;
    if (a.cu == nullptr && a.T == 1) {
        for (int b0 = 0; b0 < a.B; b0 += 65535) {     // gridDim.y's limit
            const int nb = a.B - b0 < 65535 ? a.B - b0 : 65535;
            ConvParams q = p;
            q.x = static_cast<const T *>(p.x) + b0 * p.x_sb;
            q.o = static_cast<T *>(p.o) + b0 * p.o_sb;
            q.state = static_cast<T *>(p.state) + (int64_t)b0 * (W - 1) * a.C;
            q.ex -= b0 * p.x_sb; q.eo -= b0 * p.o_sb; q.es -= (int64_t)b0 * (W - 1) * a.C;
            conv_step_kernel<T, W, kSilu><<<dim3(gx, nb), kConvThreads, 0, s>>>(q);
        }
        return launched();
    }
    const int sms = device_sms();
    if (sms <= 0) return CGDR_ERR_CUDA;
    // The longest tile that still gives every SM eight blocks: a tile re-reads W-1 rows.
    int tile = 64;
    while (tile > 8 && (int64_t)gx * ((p.n + tile - 1) / tile) < 8 * sms) tile /= 2;
    while ((p.n + (int64_t)tile - 1) / tile > 65535) tile *= 2;
    p.tile = tile;
    conv_tokens_kernel<T, W, kSilu><<<dim3(gx, (p.n + tile - 1) / tile), kConvThreads, 0, s>>>(p);
    return launched();
}

template <typename T, int W>
cgdr_status launch_act(const cgdr_conv_args &a, ConvParams &p, cudaStream_t s) {
    return a.silu ? launch_tokens<T, W, true>(a, p, s) : launch_tokens<T, W, false>(a, p, s);
}

template <typename T>
cgdr_status launch_width(const cgdr_conv_args &a, ConvParams &p, cudaStream_t s) {
    return a.W == 2 ? launch_act<T, 2>(a, p, s) : a.W == 3 ? launch_act<T, 3>(a, p, s) : launch_act<T, 4>(a, p, s);
}

cgdr_status check(const cgdr_conv_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->B < 0 || a->C <= 0 || (a->cu ? a->n_tokens : a->T) < 0) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->W < 2 || a->W > 4) return CGDR_ERR_UNSUPPORTED;
    const int esz = esize(a->dtype);
    if (a->C % (16 / esz) != 0) return CGDR_ERR_UNSUPPORTED;
    if ((a->cu ? a->n_tokens : (int64_t)a->B * a->T) > kMaxTokens) return CGDR_ERR_UNSUPPORTED;
    if (a->B == 0 || (a->cu ? a->n_tokens : a->T) == 0) return CGDR_OK;
    if (!a->x || !a->o || !a->weight || !a->state) return CGDR_ERR_INVALID_ARG;
    if (!aligned_to(a->x, 16) || !aligned_to(a->o, 16) || !aligned_to(a->state, 16) || !aligned_to(a->weight, 16) ||
        !aligned_to(a->bias, 4) || !aligned_to(a->cu, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    if (!row_stride_ok(a->x_st, esz) || !row_stride_ok(a->o_st, esz)) return CGDR_ERR_ALIGNMENT;
    if (!a->cu && (!row_stride_ok(a->x_sb, esz) || !row_stride_ok(a->o_sb, esz))) return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

}  // namespace
}  // namespace cgdr

extern "C" cgdr_status cgdr_conv(const cgdr_conv_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->B == 0 || (a->cu ? a->n_tokens : a->T) == 0) return st;
    ConvParams p{};
    p.B = a->B; p.T = a->T; p.C = a->C; p.n = a->cu ? a->n_tokens : a->B * a->T;
    p.x = a->x; p.o = a->o; p.x_sb = a->x_sb; p.x_st = a->x_st; p.o_sb = a->o_sb; p.o_st = a->o_st;
    p.weight = a->weight; p.bias = a->bias; p.state = a->state; p.cu = a->cu; p.status = a->status;
    p.ex = a->cu ? extent3(1, 0, p.n, a->x_st, a->C) : extent3(a->B, a->x_sb, a->T, a->x_st, a->C);
    p.eo = a->cu ? extent3(1, 0, p.n, a->o_st, a->C) : extent3(a->B, a->o_sb, a->T, a->o_st, a->C);
    p.es = (int64_t)a->B * (a->W - 1) * a->C;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == CGDR_BF16 ? launch_width<__nv_bfloat16>(*a, p, s) : launch_width<float>(*a, p, s);
}
