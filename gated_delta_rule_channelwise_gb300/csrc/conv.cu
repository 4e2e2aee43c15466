// Short causal convolution (cgdr_conv): y[t] = act(bias + sum_j w[j] u[t - (W-1) + j]) per channel,
// u = the W-1 state rows followed by the sequence.
//
// Bound by memory: each x is read once and each y written once, 2 W + 4 operations per element.  4,001 tokens
// of 8,192 bf16 channels in five sequences, W = 4, silu: 131.7 MB in 25.8 us, 5.1 TB/s, 76 % of a plain copy's; the
// sigmoid's two special-function instructions a value are 7 us beside it.  Single tokens of 64 x 12,288 channels: 3.9 us.
// A thread owns four channels and walks along the tokens with the last W-1 rows in
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
// Rows that a thread loads at once, while it works on as many, and blocks of an SM: measured on 4001
// tokens of 8192 bf16 channels against 2 and 8 rows (16 and 38 % slower) and 6 blocks (17 %).
constexpr int kConvBatch = 4;
constexpr int kConvBlocks = 8;
constexpr int kConvTile = 64;                         // tokens of a tile at most

// Four channels of a row as they are stored: 8 bytes of bf16, 16 of fp32.
template <typename T> struct Raw;
template <> struct Raw<float> { using type = uint4; };
template <> struct Raw<__nv_bfloat16> { using type = uint2; };
template <typename T> using raw_t = typename Raw<T>::type;
constexpr int V = 4;                                  // channels of a thread

template <typename T>
__device__ __forceinline__ raw_t<T> load_row(const T *p, int64_t off, int64_t n, int *st) {
    return range_in_bounds(off, V, n, st, nullptr) ? __ldg(reinterpret_cast<const raw_t<T> *>(p + off)) : raw_t<T>{};
}
// The state is written by the kernel that reads it: an ordinary load.
template <typename T>
__device__ __forceinline__ raw_t<T> load_state(const T *p, int64_t off, int64_t n, int *st) {
    return range_in_bounds(off, V, n, st, nullptr) ? *reinterpret_cast<const raw_t<T> *>(p + off) : raw_t<T>{};
}
template <typename T>
__device__ __forceinline__ void store_row(T *p, int64_t off, const raw_t<T> &v, int64_t n, int *st) {
    if (range_in_bounds(off, V, n, st, nullptr)) *reinterpret_cast<raw_t<T> *>(p + off) = v;
}

// The same in two fp32 pairs.
struct Row {
    f32x2 v[2];
    __device__ __forceinline__ void set(const uint4 &r) {
        v[0] = pair(__uint_as_float(r.x), __uint_as_float(r.y));
        v[1] = pair(__uint_as_float(r.z), __uint_as_float(r.w));
    }
    __device__ __forceinline__ void set(const uint2 &r) {
        v[0] = pair(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u));
        v[1] = pair(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
    }
    __device__ __forceinline__ void get(uint4 &r) const {
        const float2 a = split(v[0]), b = split(v[1]);
        r = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    }
    __device__ __forceinline__ void get(uint2 &r) const {
        const float2 a = split(v[0]), b = split(v[1]);
        r = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y));
    }
};

// The filter, by taps, and the bias of a thread's channels.
template <int W>
struct Filter {
    f32x2 w[W][2], bias[2];
    __device__ __forceinline__ void load(const ConvParams &p, int c0) {
        float flat[V * W];
#pragma unroll
        for (int i = 0; i < W; ++i)
            *reinterpret_cast<float4 *>(flat + 4 * i) = __ldg(reinterpret_cast<const float4 *>(p.weight + (int64_t)c0 * W) + i);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][e] = pair(flat[2 * e * W + j], flat[(2 * e + 1) * W + j]);
            bias[e] = p.bias != nullptr ? pair(__ldg(p.bias + c0 + 2 * e), __ldg(p.bias + c0 + 2 * e + 1)) : pair(0.f, 0.f);
        }
    }
};

// One row: the window's W-1 rows and `raw` give y; the window moves on.
template <typename T, int W, bool kSilu>
__device__ __forceinline__ raw_t<T> conv_row(const Filter<W> &f, Row (&win)[W - 1], const raw_t<T> &raw) {
    Row now, y;
    now.set(raw);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        f32x2 acc = f.bias[e];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) acc = fma2(f.w[j][e], win[j].v[e], acc);
        acc = fma2(f.w[W - 1][e], now.v[e], acc);
        y.v[e] = kSilu ? silu_pair(acc) : acc;
    }
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) win[j] = win[j + 1];
    win[W - 2] = now;
    raw_t<T> out;
    y.get(out);
    return out;
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
__global__ void __launch_bounds__(kConvThreads, kConvBlocks) conv_tokens_kernel(const ConvParams p) {
    constexpr int U = kConvBatch;
    const int c0 = (blockIdx.y * kConvThreads + threadIdx.x) * V;
    if (c0 >= p.C) return;
    const T *x = static_cast<const T *>(p.x);
    T *o = static_cast<T *>(p.o), *state = static_cast<T *>(p.state);
    Place at, after;
    const int end0 = min((int)(blockIdx.x + 1) * p.tile, p.n);
    const int end = end0 < p.n ? tile_begin<W>(p, end0, after) : p.n;
    int i = tile_begin<W>(p, blockIdx.x * p.tile, at);
    if (i >= end || at.b >= p.B) return;

    auto x_off = [&](int t) -> int64_t {
        return (p.cu == nullptr ? (t / p.T) * p.x_sb + (t % p.T) * p.x_st : t * p.x_st) + c0;
    };
    auto o_off = [&](int t) -> int64_t {
        return (p.cu == nullptr ? (t / p.T) * p.o_sb + (t % p.T) * p.o_st : t * p.o_st) + c0;
    };
    auto row = [&](int t) { return load_row<T>(x, x_off(t), p.ex, p.status); };

    Filter<W> f;
    f.load(p, c0);
    Row win[W - 1];
    if (at.pos > 0) {                                 // at least W-1 of the sequence's rows precede
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j].set(row(i - (W - 1) + j));
    }
    while (i < end && at.b < p.B) {                   // the tile's part of one sequence after the other
        const int rows = max(min(at.len - at.pos, end - i), 1);
        int64_t xo = x_off(i), oo = o_off(i);
        if (at.pos == 0) {                            // a sequence begins: its state in, its last rows out
            const int64_t s0 = (int64_t)at.b * (W - 1) * p.C + c0;
            raw_t<T> old[W - 1], last[W - 1];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) old[j] = load_state<T>(state, s0 + (int64_t)j * p.C, p.es, p.status);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                win[j].set(old[j]);
                const int k = at.len + j;             // row k of u: state rows first
                last[j] = old[W - 2];
#pragma unroll
                for (int m = 0; m < W - 1; ++m)
                    if (k == m) last[j] = old[m];
                if (k >= W - 1) last[j] = row(i + k - (W - 1));
            }
#pragma unroll
            for (int j = 0; j < W - 1; ++j) store_row<T>(state, s0 + (int64_t)j * p.C, last[j], p.es, p.status);
        }
        raw_t<T> next[U];
        auto fetch = [&](int r) {                     // rows r .. r + U - 1 of the part
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r + u < rows) next[u] = load_row<T>(x, xo, p.ex, p.status);
                xo += p.x_st;
            }
        };
        auto put = [&](const raw_t<T> &v) {
            store_row<T>(o, oo, conv_row<T, W, kSilu>(f, win, v), p.eo, p.status);
            oo += p.o_st;
        };
        fetch(0);
        int r = 0;
        for (; r + U <= rows; r += U) {
            raw_t<T> cur[U];
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = next[u];
            fetch(r + U);
#pragma unroll
            for (int u = 0; u < U; ++u) put(cur[u]);
        }
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (r + u < rows) put(next[u]);
        i += rows;
        if (i < end) at = place_of(p, i);
    }
}

// One token a sequence: a thread owns four channels of one sequence.
template <typename T, int W, bool kSilu>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(const ConvParams p) {
    const int c0 = (blockIdx.x * kConvThreads + threadIdx.x) * V;
    const int b = blockIdx.y;
    if (c0 >= p.C) return;
    const T *x = static_cast<const T *>(p.x);
    T *o = static_cast<T *>(p.o), *state = static_cast<T *>(p.state);
    const int64_t s0 = (int64_t)b * (W - 1) * p.C + c0;
    const raw_t<T> now = load_row<T>(x, b * p.x_sb + c0, p.ex, p.status);
    raw_t<T> old[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) old[j] = load_state<T>(state, s0 + (int64_t)j * p.C, p.es, p.status);
    Filter<W> f;
    f.load(p, c0);
    Row win[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        win[j].set(old[j]);
        store_row<T>(state, s0 + (int64_t)j * p.C, j < W - 2 ? old[j + 1 < W - 1 ? j + 1 : 0] : now, p.es, p.status);
    }
    store_row<T>(o, b * p.o_sb + c0, conv_row<T, W, kSilu>(f, win, now), p.eo, p.status);
}

template <typename T, int W, bool kSilu>
cgdr_status launch_tokens(const cgdr_conv_args &a, ConvParams &p, cudaStream_t s) {
    const int gx = (a.C / V + kConvThreads - 1) / kConvThreads;
    // single tokens hand nothing from tile to tile: 3.9 us for 64 x 12,288 channels, 11.6 in the other kernel
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
    // Whole waves of resident blocks, with tiles of kConvTile tokens at most (a tile re-reads W-1 rows) and 8 at
    // least.
    const int64_t wave = kConvBlocks * sms, waves = ((int64_t)p.n * gx + wave * kConvTile - 1) / (wave * kConvTile);
    const int64_t tiles = waves * wave / gx > 0 ? waves * wave / gx : 1;
    int tile = (int)((p.n + tiles - 1) / tiles);
    if (tile < 8) tile = 8;
    p.tile = tile;
    conv_tokens_kernel<T, W, kSilu><<<dim3((p.n + tile - 1) / tile, gx), kConvThreads, 0, s>>>(p);
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
    if (a->C % (16 / esz) != 0 || a->C > 65535 * V * kConvThreads) return CGDR_ERR_UNSUPPORTED;
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
