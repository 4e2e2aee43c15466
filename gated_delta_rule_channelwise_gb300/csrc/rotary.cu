// Rotary positions (cgdr_rotary): pairs of channels of every head turned by their token's angle, in place.
//
// A frequency is kept as a 64-bit fraction of a turn, so that position * frequency modulo a turn is one integer
// product, exact whatever the position; the nearest quarter turn is taken off and all that remains becomes fp32, so that the sine of a
// slow pair has fp32's bits, too.
// Bound by memory: 4,000 tokens of 32 + 8 heads of 128 bf16 (82 MB read and written) take 16.7 us, 12.1 at the copy rate; 4,011 tokens of 24 + 24
// heads of 96 fp32, half of each turned (74 MB, in pieces of 192 bytes) 18.8, 10.9; 64 tokens 2.2, a launch.
#include "layer.cuh"

namespace cgdr {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = kThreads;
constexpr int kMaxHeads = 65535;

struct RotaryParams {
    int n, Hq, H, half;                               // H = Hq + Hk
    int units, rows;                                  // vectors of pairs of a head, heads that a token's threads take at a time
    int shift;                                        // 2^shift threads to a token
    float scale;
    void *q, *k;
    int64_t q_st, q_sh, eq, k_st, k_sh, ek;           // strides, footprints
    const int32_t *positions;
    const double *freq;
    int *status;
};

// A frequency (radians a position) as a fraction of a turn times 2^64, modulo a turn: its 53 bits of mantissa times 2^66 / (2 pi),
// shifted by the exponent.
__device__ __forceinline__ uint64_t fraction_of(double freq) {
    const uint64_t bits = (uint64_t)__double_as_longlong(freq), low = bits & 0xFFFFFFFFFFFFFull;
    const int exponent = (int)(bits >> 52) & 0x7FF;
    const uint64_t m = exponent ? low | 1ull << 52 : low;
    constexpr uint64_t kInverse = 0xA2F9836E4E44152Aull;              // 2^66 / (2 pi)
    const uint64_t hi = __umul64hi(m, kInverse), lo = m * kInverse;
    const int down = 1077 - (exponent ? exponent : 1);
    const uint64_t r = down >= 128 ? 0 : down >= 64 ? hi >> (down - 64) : down > 0 ? hi << (64 - down) | lo >> down : down > -64 ? lo << -down : 0;
    return bits >> 63 ? 0 - r : r;
}
// cos and sin of position * freq, times scale.
__device__ __forceinline__ float2 turn_of(int position, double freq, float scale) {
    const uint64_t phase = (uint64_t)position * fraction_of(freq);
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const float rest = __ll2float_rn((int64_t)(phase - ((uint64_t)quarter << 62))) * 0x1p-63f;            // half turns, |rest| <= 1/4
    float s, c;
    sincospif(rest, &s, &c);
    const float cs = quarter & 1 ? s : c, sn = quarter & 1 ? c : s;
    float2 r = make_float2((quarter + 1) & 2 ? -cs : cs, quarter & 2 ? -sn : sn);
    if ((__double2hiint(freq) & 0x7FF00000) == 0x7FF00000) r.x = r.y = __int_as_float(0x7FC00000);
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

constexpr int kAhead = 3;                             // in the first case: two 17.3 us, three 16.7, four 20.5

// Some warps take a token.  A thread turns V pairs of a head at a time, V values i, i + 1, .. and their partners `half` further on, or 2 V
// neighbours, and goes on to the same pairs of other heads, so that it keeps its cos and sin in registers; kAhead heads
// are on their way together.  The angles are formed once for all heads, while the first values arrive.
template <typename T, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const RotaryParams p) {
    extern __shared__ float4 s_raw[];
    float *s_cos = reinterpret_cast<float *>(s_raw), *s_sin = s_cos + (kThreads >> p.shift) * p.half;   // [tokens][half] each
    using raw = typename Lanes<T, V>::raw;
    const int tokens = kThreads >> p.shift, t0 = blockIdx.x * tokens, mine = threadIdx.x >> p.shift, t = t0 + mine;
    const int l = threadIdx.x & ((1 << p.shift) - 1), lane = l / p.units, unit = l - lane * p.units;
    wait_for_inputs();
    const bool live = t < p.n && lane < p.rows && p.positions[t] >= 0;
    constexpr int64_t kStep = kInterleaved ? 2 * V : V;
    const int64_t far = kInterleaved ? V : p.half;
    T *q = static_cast<T *>(p.q) + t * p.q_st + kStep * unit, *k = static_cast<T *>(p.k) + t * p.k_st + kStep * unit;
    float c[V], s[V];
    for (int first = lane;; first += kAhead * p.rows) {
        raw a[kAhead], b[kAhead];
        T *at[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int head = first + j * p.rows;
            at[j] = nullptr;
            if (live && head < p.H) {
                const bool key = head >= p.Hq;
                T *x = key ? k + (head - p.Hq) * p.k_sh : q + head * p.q_sh;
                const int64_t off = x - static_cast<T *>(key ? p.k : p.q), ex = key ? p.ek : p.eq;
                if (range_in_bounds(off, V, ex, p.status, nullptr) && range_in_bounds(off + far, V, ex, p.status, nullptr)) {
                    at[j] = x;
                    a[j] = *reinterpret_cast<const raw *>(x);
                    b[j] = *reinterpret_cast<const raw *>(x + far);
                }
            }
        }
        if (first == lane) {                          // the first round, which every thread takes
            for (int e = threadIdx.x; e < tokens * p.half; e += kThreads) {
                const int i = e / p.half, position = t0 + i < p.n ? p.positions[t0 + i] : 0;
                const float2 turn = turn_of(position, p.freq[e - i * p.half], p.scale);
                s_cos[e] = turn.x;
                s_sin[e] = turn.y;
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) {
                c[e] = s_cos[mine * p.half + V * unit + e];
                s[e] = s_sin[mine * p.half + V * unit + e];
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (at[j] == nullptr) continue;
            float u[V], v[V];
            unpack<T, V>(a[j], u);
            unpack<T, V>(b[j], v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // interleaved pairs lie next to each other, a's before b's
                float &x = !kInterleaved ? u[e] : 2 * e < V ? u[2 * e % V] : v[2 * e % V];
                float &y = !kInterleaved ? v[e] : 2 * e + 1 < V ? u[(2 * e + 1) % V] : v[(2 * e + 1) % V];
                const float px = x, py = y;
                x = px * c[e] - py * s[e];
                y = py * c[e] + px * s[e];
            }
            *reinterpret_cast<raw *>(at[j]) = pack<T, V>(u);
            *reinterpret_cast<raw *>(at[j] + far) = pack<T, V>(v);
        }
        if (first + kAhead * p.rows >= p.H) break;
    }
}

cgdr_status check(const cgdr_rotary_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->n < 0 || a->Hq <= 0 || a->Hk < 0 || a->D <= 0 || a->half <= 0 || a->half > a->D / 2) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->half > kMaxHalf || a->n > kMaxTokens || a->Hq > kMaxHeads || a->Hk > kMaxHeads) return CGDR_ERR_UNSUPPORTED;
    if (a->n == 0) return CGDR_OK;
    if (!disjoint(a->n, a->q_st, a->Hq, a->q_sh, a->D) || !disjoint(a->n, a->k_st, a->Hk, a->k_sh, a->D)) return CGDR_ERR_INVALID_ARG;
    if (!a->q || (a->Hk > 0 && !a->k) || !a->positions || !a->freq) return CGDR_ERR_INVALID_ARG;
    if (a->Hk > 0 && a->k == a->q) return CGDR_ERR_INVALID_ARG;     // turned twice
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
    // Two warps to a token (one: 17.7 us in the first case above), or more: where a head has more vectors than that, or where there are too few tokens to fill the SMs.
    p.shift = 6;
    while ((1 << p.shift) < kThreads && ((1 << p.shift) < p.units || ((int64_t)p.n << p.shift) < (int64_t)kThreads * 2 * sms)) ++p.shift;
    p.rows = (1 << p.shift) / p.units;
    const int tokens = kThreads >> p.shift;
    const unsigned grid = (unsigned)((p.n + tokens - 1) / tokens);
    const size_t bytes = (size_t)2 * tokens * p.half * sizeof(float);
    return launch_early(interleaved ? rotary_kernel<T, V, true> : rotary_kernel<T, V, false>, grid, kThreads, bytes, s, 0, p);
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
