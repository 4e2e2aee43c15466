// Rotary positions (cgdr_rotary): pairs of channels of every head turned by their token's angle, in place.
//
// A frequency is kept as a 64-bit fraction of a turn, so that position * frequency modulo a turn is one integer
// product, exact whatever the position; the nearest quarter turn is taken off before the remainder becomes fp32.
#include "layer.cuh"

namespace cgdr {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = kThreads;

struct RotaryParams {
    int n, Hq, H, half;                               // H = Hq + Hk
    int tokens;                                       // of a block
    int units, rows;                                  // vectors of pairs of a head, heads that a block takes at a time
    float scale;
    void *q, *k;
    int64_t q_st, q_sh, eq, k_st, k_sh, ek;           // strides, footprints
    const int32_t *positions;
    const double *freq;
    int *status;
};

// cos and sin of position * freq, times scale.
__device__ __forceinline__ float2 turn_of(int position, double freq, float scale) {
    double turns = freq * 0.15915494309189533577;     // 1 / (2 pi)
    turns -= floor(turns);
    const uint64_t phase = (uint64_t)position * __double2ull_rz(turns * 18446744073709551616.0);
    const uint64_t quarter = (phase + (1ull << 61)) >> 62;
    const float rest = (float)(int32_t)((int64_t)(phase - (quarter << 62)) >> 32) * 0x1p-31f;   // half turns, |rest| <= 1/4
    float s, c;
    sincospif(rest, &s, &c);
    const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
    float2 r = make_float2((quarter + 1) & 2 ? -cs : cs, quarter & 2 ? -sn : sn);
    if (!isfinite(freq)) r.x = r.y = __int_as_float(0x7FC00000);
    return make_float2(r.x * scale, r.y * scale);
}

template <typename T, int V> struct Lanes;            // V values of T in one load
template <> struct Lanes<__nv_bfloat16, 8> { using raw = uint4; };
template <> struct Lanes<__nv_bfloat16, 4> { using raw = uint2; };
template <> struct Lanes<__nv_bfloat16, 1> { using raw = uint16_t; };
template <> struct Lanes<float, 4> { using raw = uint4; };
template <> struct Lanes<float, 1> { using raw = uint32_t; };

template <typename T, int V> __device__ __forceinline__ void unpack(const typename Lanes<T, V>::raw &r, float (&f)[V]) {
    const T *t = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = Cvt<T>::to_f(t[e]);
}
template <typename T, int V> __device__ __forceinline__ typename Lanes<T, V>::raw pack(const float (&f)[V]) {
    typename Lanes<T, V>::raw r;
    T *t = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = Cvt<T>::from_f(f[e]);
    return r;
}

// A thread turns V pairs of a head at a time: V values i, i + 1, .. and their partners `half` further on, or 2 V
// neighbours.  The block's angles are in shared memory, formed once for all heads.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
    extern __shared__ float2 s_turn[];                // [tokens][half]
    using raw = typename Lanes<T, V>::raw;
    const int t0 = blockIdx.x * p.tokens, tokens = min(p.tokens, p.n - t0);
    for (int e = threadIdx.x; e < tokens * p.half; e += kThreads) {
        const int position = p.positions[t0 + e / p.half];
        if (position >= 0) s_turn[e] = turn_of(position, p.freq[e % p.half], p.scale);
    }
    __syncthreads();
    const int unit = threadIdx.x % p.units, lane = threadIdx.x / p.units;
    if (lane >= p.rows) return;
    for (int pair = lane; pair < tokens * p.H; pair += p.rows) {
        const int t = pair / p.H, head = pair - t * p.H;
        const bool key = head >= p.Hq;
        if (p.positions[t0 + t] < 0) continue;
        T *x = static_cast<T *>(key ? p.k : p.q);
        const int64_t at = (int64_t)(t0 + t) * (key ? p.k_st : p.q_st) + (int64_t)(key ? head - p.Hq : head) * (key ? p.k_sh : p.q_sh), ex = key ? p.ek : p.eq;
        const int64_t a = at + (kInterleaved ? 2 * V : V) * unit, b = kInterleaved ? a + V : a + p.half;
        if (!range_in_bounds(a, V, ex, p.status, nullptr) || !range_in_bounds(b, V, ex, p.status, nullptr)) continue;
        raw *pa = reinterpret_cast<raw *>(x + a), *pb = reinterpret_cast<raw *>(x + b);
        float u[V], v[V];
        unpack<T, V>(*pa, u);
        unpack<T, V>(*pb, v);
        const float2 *turn = s_turn + t * p.half + V * unit;
        if (kInterleaved) {                           // pairs lie next to each other, u's before v's
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float &x = 2 * e < V ? u[2 * e % V] : v[2 * e % V], &y = 2 * e + 1 < V ? u[(2 * e + 1) % V] : v[(2 * e + 1) % V];
                const float2 cs = turn[e];
                const float px = x, py = y;
                x = px * cs.x - py * cs.y;
                y = py * cs.x + px * cs.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 cs = turn[e];
                const float px = u[e], py = v[e];
                u[e] = px * cs.x - py * cs.y;
                v[e] = py * cs.x + px * cs.y;
            }
        }
        *pa = pack<T, V>(u);
        *pb = pack<T, V>(v);
    }
}

cgdr_status check(const cgdr_rotary_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->n < 0 || a->Hq <= 0 || a->Hk < 0 || a->D <= 0 || a->half <= 0 || a->half > a->D / 2) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->half > kMaxHalf || a->n > kMaxTokens || a->Hq > 65535 || a->Hk > 65535) return CGDR_ERR_UNSUPPORTED;
    if (a->n == 0) return CGDR_OK;
    if (!disjoint(a->n, a->q_st, a->Hq, a->q_sh, a->D) || !disjoint(a->n, a->k_st, a->Hk, a->k_sh, a->D)) return CGDR_ERR_INVALID_ARG;
    if (!a->q || (a->Hk > 0 && !a->k) || !a->positions || !a->freq) return CGDR_ERR_INVALID_ARG;
    const int esz = esize(a->dtype);
    if (!aligned_to(a->q, 16) || !aligned_to(a->positions, 4) || !aligned_to(a->freq, 8) || !aligned_to(a->status, 4)) return CGDR_ERR_ALIGNMENT;
    if (!row_stride_ok(a->q_st, esz) || !row_stride_ok(a->q_sh, esz)) return CGDR_ERR_ALIGNMENT;
    if (a->Hk > 0 && (!aligned_to(a->k, 16) || !row_stride_ok(a->k_st, esz) || !row_stride_ok(a->k_sh, esz))) return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

template <typename T, int V>
cgdr_status launch(RotaryParams &p, bool interleaved, cudaStream_t s) {
    const int sms = device_sms();
    if (sms <= 0) return CGDR_ERR_CUDA;
    p.units = p.half / V;
    p.rows = kThreads / p.units;
    p.tokens = 1;
    while (p.tokens < 4 && (int64_t)p.n >= (int64_t)p.tokens * 8 * sms) p.tokens *= 2;
    const unsigned grid = (unsigned)((p.n + p.tokens - 1) / p.tokens);
    const size_t bytes = (size_t)p.tokens * p.half * sizeof(float2);
    if (interleaved) rotary_kernel<T, V, true><<<grid, kThreads, bytes, s>>>(p);
    else rotary_kernel<T, V, false><<<grid, kThreads, bytes, s>>>(p);
    return launched();
}

}  // namespace
}  // namespace cgdr

extern "C" cgdr_status cgdr_rotary(const cgdr_rotary_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->n == 0) return st;
    RotaryParams p{};
    p.n = a->n; p.Hq = a->Hq; p.H = a->Hq + a->Hk; p.half = a->half;
    p.scale = a->scale;
    p.q = a->q; p.q_st = a->q_st; p.q_sh = a->q_sh; p.eq = extent3(a->n, a->q_st, a->Hq, a->q_sh, a->D);
    p.k = a->k; p.k_st = a->k_st; p.k_sh = a->k_sh; p.ek = extent3(a->n, a->k_st, a->Hk, a->k_sh, a->D);
    p.positions = a->positions; p.freq = a->freq; p.status = a->status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool il = a->interleaved != 0;
    if (a->dtype == CGDR_BF16)
        return a->half % 8 == 0 ? launch<__nv_bfloat16, 8>(p, il, s) : a->half % 4 == 0 ? launch<__nv_bfloat16, 4>(p, il, s)
                                                                                       : launch<__nv_bfloat16, 1>(p, il, s);
    return a->half % 4 == 0 ? launch<float, 4>(p, il, s) : launch<float, 1>(p, il, s);
}
