// Selective state space scan (cgdr_scan): per channel c and state n
//     h[n] = exp(A[c, n] d) h[n] + d x B[n],   y = sum_n C[n] h[n],   A = -exp(A_log).
//
// A thread holds four states of four neighbouring channels in registers, N/4 neighbouring lanes the
// channels' N states, a block 1024/N channels (16 for N = 128).  The tokens come in tiles of 8 (16): their
// rows are loaded into registers one tile ahead, turned into the fp32 values that the recurrence reads (d and d x
// once per channel, not once per state) and put into shared memory.  Arithmetic is in packed pairs of channels.
//
// The work is N exponentials and 4 N multiply-adds a token and channel, against 8 bytes: the scan is
// bound by instruction issue and the exponential unit (32 a clock of an SM), and, with few channels, by the length
// of the recurrence.  Then a sequence is cut into chunks.  The state that leaves a chunk is
// exp(A sum d) h_in + e, with e the chunk's own end state from zero, so one launch forms (sum d, e) of
// every chunk but the last, and a second runs all chunks, each joining its h_in from the pairs
// before it.  That does the exponentials twice, so chunks are as long as the SM count allows.
//
// Measured: one sequence of 4,000 tokens, 4,096 bf16 channels, N = 16, gated: 132 us for 262 M exponentials done
// twice, which are 57 us of their unit; the schedulers issue in 49 % of the cycles with the 12 warps that
// 160 registers a thread leave an SM (16 warps with fewer registers: 138 us).  Three sequences of 1 to 16,411 tokens,
// 24,618 in all, of 1,000 fp32 channels: 200 us.  A step of 64 x 4,096 channels: 8.8 us for 35.9 MB.
#include "serve.cuh"

namespace cgdr {
namespace {

struct ScanParams {
    int B, T, C, Cg, G, n, chunk, softplus, o_f32;
    const void *x, *dt, *z, *Bm, *Cm;
    int64_t x_sb, x_st, dt_sb, dt_st, z_sb, z_st, B_sb, B_st, C_sb, C_st, o_sb, o_st;
    void *o;
    const float *A_log, *D, *dt_bias;
    float *state;
    const int32_t *cu;
    float *ends, *sums;                               // workspace: [slots][C][N] end states, [slots][C] sums of d
    int slots;
    int *status;
    int64_t ex, edt, ez, eB, eC, eo;                  // footprints (index-checking build)
};

// A block's piece of a sequence.
struct Piece {
    int b, k, chunks, slot;                           // sequence, chunk, chunks of the sequence, workspace slot of chunk 0
    int t0, len;                                      // first token (packed: of all tokens; dense: of the sequence), tokens
};

// The item-th piece; `multi` counts only sequences of several chunks.  b = -1: there is none.
// Run by a whole warp.
__device__ __forceinline__ Piece find_piece(const ScanParams &p, int item, bool multi) {
    Piece r{-1, 0, 0, 0, 0, 0};
    if (p.cu == nullptr) {
        const int chunks = (p.T + p.chunk - 1) / p.chunk;
        r.b = item / chunks;
        if (r.b >= p.B) { r.b = -1; return r; }
        r.k = item % chunks;
        r.chunks = chunks;
        r.slot = r.b * chunks;
        r.t0 = r.k * p.chunk;
        r.len = min(p.chunk, p.T - r.t0);
        return r;
    }
    const int lane = threadIdx.x & 31;
    int items = 0, slots = 0;                         // of the sequences before
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int2 s = make_int2(0, 0);
        if (b < p.B) s = seq_span(p.cu, b, p.n);
        const int chunks = (s.y - s.x + p.chunk - 1) / p.chunk;
        const int own_slots = chunks > 1 ? chunks : 0, own = multi ? own_slots : chunks;
        int ci = own, si = own_slots;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, ci, d), v = __shfl_up_sync(0xffffffffu, si, d);
            if (lane >= d) { ci += u; si += v; }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, items + ci > item);
        if (hit != 0) {
            const int l = __ffs(hit) - 1;
            r.b = b0 + l;
            r.k = item - (items + __shfl_sync(0xffffffffu, ci - own, l));
            r.chunks = __shfl_sync(0xffffffffu, chunks, l);
            r.slot = slots + __shfl_sync(0xffffffffu, si - own_slots, l);
            const int lo = __shfl_sync(0xffffffffu, s.x, l), hi = __shfl_sync(0xffffffffu, s.y, l);
            r.t0 = lo + r.k * p.chunk;
            r.len = min(p.chunk, hi - r.t0);
            return r;
        }
        items += __shfl_sync(0xffffffffu, ci, 31);
        slots += __shfl_sync(0xffffffffu, si, 31);
    }
    return r;
}

// softplus(x) = max(x, 0) + log(1 + t), t = e^-|x|.  With s = t / (2 + t) <= 1/3 the logarithm is
// 2 atanh(s) = 2 s r(s^2), r(q) = 1 + q/3 + q^2/5 + ...; a polynomial of degree 4 through r's values
// at the Chebyshev points of [0, 1/9] is within 4e-9 of it.  Small results keep their relative
// accuracy, which a logarithm of 1 + t in fp32 would lose.
__device__ __forceinline__ f32x2 softplus_pair(f32x2 v) {
    const float2 x = split(v);
    const f32x2 t = pair(ex2(-kLog2e * fabsf(x.x)), ex2(-kLog2e * fabsf(x.y)));
    const float2 w = split(add2(t, both(2.f)));
    const f32x2 s = mul2(t, pair(rcp(w.x), rcp(w.y))), q = mul2(s, s);
    f32x2 r = fma2(q, both(0.14078889787197113f), both(0.13982579112052917f));
    r = fma2(r, q, both(0.20012298226356506f));
    r = fma2(r, q, both(0.3333316147327423f));
    r = fma2(r, q, both(1.f));
    return fma2(add2(s, s), r, pair(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}

// -exp(A_log) / log 2, finite: where the exponential overflows, an infinity times a step of zero (a tile's padding, or a
// softplus that underflows) would be a NaN, and exp(A 0) is 1.  A NaN compares false and stays.
__device__ __forceinline__ float rate(float A_log) {
    const float r = -kLog2e * expf(A_log);
    return r < -3e38f ? -3e38f : r;
}

// Eight consecutive elements as stored, and as fp32.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(f32x2 (&f)[4]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
};
template <> struct Eight<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const uint4 *>(p));
        b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(f32x2 (&f)[4]) const {
        f[0] = pair(__uint_as_float(a.x), __uint_as_float(a.y));
        f[1] = pair(__uint_as_float(a.z), __uint_as_float(a.w));
        f[2] = pair(__uint_as_float(b.x), __uint_as_float(b.y));
        f[3] = pair(__uint_as_float(b.z), __uint_as_float(b.w));
    }
};
template <typename T>
__device__ __forceinline__ void fetch(Eight<T> &v, const void *base, int64_t off, bool ok, int64_t n, int *st) {
    v.zero();
    if (ok && range_in_bounds(off, 8, n, st, nullptr)) v.load(static_cast<const T *>(base) + off);
}

// A block's shape.  A thread holds four states of each of four neighbouring channels: every value of
// d, d x, B and C that it reads from shared memory meets four states, which brings the reads (128 bytes
// a clock of the SM) to the level of the arithmetic; with four states of one channel they are twice
// the time of everything else.
template <int N>
struct ScanShape {
    static constexpr int LPC = N / 4;                                 // lanes that share four channels
    static constexpr int CH = N <= 64 ? 1024 / N : 16;                // channels of a block
    static constexpr int NT = CH / 4 * LPC;                           // 64 threads, 128 for N = 128
    static constexpr int TT = N == 16 ? 8 : 16;                       // tokens of a tile
    static constexpr int XV = TT * CH / 8;                            // eight-channel vectors of a tile (at most NT)
    static constexpr int BV = TT * N / 8, BPT = (BV + NT - 1) / NT;   // eight-state vectors, and of a thread
    static_assert(XV <= NT, "one vector of x a thread");
};
template <int N, bool kEnds>
struct ScanTile {
    using Sh = ScanShape<N>;
    float d[Sh::TT][Sh::CH], u[Sh::TT][Sh::CH];                       // d, d x
    float b[Sh::TT][N], c[kEnds ? 1 : Sh::TT][N];
    float y[kEnds ? 1 : Sh::TT][4][Sh::CH + 8];                       // four parts of every y, each in banks of its own
};

// kEnds: the first launch (end states and sums of d of every chunk but a sequence's last).
template <typename T, int N, bool kEnds>
__global__ void __launch_bounds__(ScanShape<N>::NT, N == 128 ? 3 : 6) scan_kernel(const ScanParams p) {
    using Sh = ScanShape<N>;
    constexpr int LPC = Sh::LPC, TT = Sh::TT;
    __shared__ __align__(16) ScanTile<N, kEnds> sm;
    const int tid = threadIdx.x, ch = tid / LPC * 4, q = tid % LPC;   // channels ch .. ch + 3, states 4 q .. 4 q + 3
    const Piece pc = find_piece(p, blockIdx.y, kEnds);
    if (pc.b < 0 || (kEnds && pc.k == pc.chunks - 1)) return;
    if (pc.chunks > 1 && pc.slot + pc.chunks > p.slots) return;       // offsets that do not ascend: more tokens than there are
    const int per = (p.Cg + Sh::CH - 1) / Sh::CH;                     // blocks of a group
    const int g = blockIdx.x / per, cg0 = (blockIdx.x % per) * Sh::CH, c0 = g * p.Cg + cg0;
    const bool live = cg0 + ch < p.Cg;                                // Cg is a multiple of 8: all four channels or none
    const int c = live ? c0 + ch : c0;

    // in pairs of channels: d and d x come from shared memory as pairs, and a pair of y needs no sum across
    f32x2 A[2][4], h[2][4] = {};
    auto load_four = [&](const float *src, f32x2 (&to)[2][4]) {       // [channel][state] rows of N
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 lo = *reinterpret_cast<const float4 *>(src + 2 * j * N), hi = *reinterpret_cast<const float4 *>(src + (2 * j + 1) * N);
            to[j][0] = pair(lo.x, hi.x); to[j][1] = pair(lo.y, hi.y); to[j][2] = pair(lo.z, hi.z); to[j][3] = pair(lo.w, hi.w);
        }
    };
    auto load_h = [&](const float *src) { load_four(src, h); };
    auto store_h = [&](float *dst) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float2 f[4] = {split(h[j][0]), split(h[j][1]), split(h[j][2]), split(h[j][3])};
            *reinterpret_cast<float4 *>(dst + 2 * j * N) = make_float4(f[0].x, f[1].x, f[2].x, f[3].x);
            *reinterpret_cast<float4 *>(dst + (2 * j + 1) * N) = make_float4(f[0].y, f[1].y, f[2].y, f[3].y);
        }
    };
    load_four(p.A_log + (int64_t)c * N + 4 * q, A);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 a = split(A[j][n]);
            A[j][n] = pair(rate(a.x), rate(a.y));
        }
    // h <- exp(A d) h + in, for state n of channels 2 j, 2 j + 1
    auto step = [&](int j, int n, f32x2 d, f32x2 in) {
        const float2 e = split(mul2(d, A[j][n]));
        h[j][n] = fma2(pair(ex2(e.x), ex2(e.y)), h[j][n], in);
    };
    float *hs = p.state + ((int64_t)pc.b * p.C + c) * N + 4 * q;
    auto end_of = [&](int k) { return p.ends + ((int64_t)(pc.slot + k) * p.C + c) * N + 4 * q; };
    if (pc.k == 0) {
        // the state of a sequence of several chunks is replaced by its last chunk's block, maybe
        // before this one starts: the first launch leaves a copy in the last chunk's slot
        if (kEnds || pc.chunks == 1) load_h(hs);
        else load_h(end_of(pc.chunks - 1));
        if (kEnds && live) store_h(end_of(pc.chunks - 1));
    } else if (!kEnds) {                              // join the chunks before this one
        load_h(end_of(0));
#pragma unroll 4
        for (int k = 1; k < pc.k; ++k) {
            const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(p.sums + (int64_t)(pc.slot + k) * p.C + c);
            f32x2 e[2][4];
            load_four(end_of(k), e);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                step(0, n, d.x, e[0][n]);
                step(1, n, d.y, e[1][n]);
            }
        }
    }

    // staging: eight channels of a token, and eight states of a token's B and C, to a thread
    const int xt = tid / (Sh::CH / 8), xc = tid % (Sh::CH / 8) * 8;
    const bool stages = tid < Sh::XV, xlive = stages && cg0 + xc < p.Cg;
    Eight<T> rx, rd, rz, rb[Sh::BPT], rc[Sh::BPT];
    f32x2 bias[4], skip[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        auto two = [&](const float *v) {
            return xlive && v != nullptr ? __ldg(reinterpret_cast<const float2 *>(v + c0 + xc) + e) : make_float2(0.f, 0.f);
        };
        const float2 b = two(p.dt_bias), d = kEnds ? make_float2(0.f, 0.f) : two(p.D);
        bias[e] = pair(b.x, b.y);
        skip[e] = pair(d.x, d.y);
    }
    // offsets of the thread's first rows; tiles are TT rows apart
    const int64_t at = p.cu != nullptr ? 0 : pc.b, row = pc.t0 + xt;
    int64_t ox = at * p.x_sb + row * p.x_st + c0 + xc, od = at * p.dt_sb + row * p.dt_st + c0 + xc,
            oz = at * p.z_sb + row * p.z_st + c0 + xc, oo = at * p.o_sb + row * p.o_st + c0 + xc, ob[Sh::BPT], oc[Sh::BPT];
#pragma unroll
    for (int i = 0; i < Sh::BPT; ++i) {
        const int v = tid + i * Sh::NT, bn = g * N + v % (N / 8) * 8;
        const int64_t brow = pc.t0 + v / (N / 8);
        ob[i] = at * p.B_sb + brow * p.B_st + bn;
        oc[i] = at * p.C_sb + brow * p.C_st + bn;
    }
    const bool gated = !kEnds && p.z != nullptr;
    auto load = [&](int left) {                       // of the tile's tokens on, `left` are left
        const bool ok = xlive && xt < left;
        fetch<T>(rx, p.x, ox, ok, p.ex, p.status);
        fetch<T>(rd, p.dt, od, ok, p.edt, p.status);
        if (!kEnds) fetch<T>(rz, p.z, oz, ok && gated, p.ez, p.status);
        ox += TT * p.x_st; od += TT * p.dt_st; oz += TT * p.z_st;
#pragma unroll
        for (int i = 0; i < Sh::BPT; ++i) {
            const int v = tid + i * Sh::NT;
            const bool okb = v < Sh::BV && v / (N / 8) < left;
            fetch<T>(rb[i], p.Bm, ob[i], okb, p.eB, p.status);
            if (!kEnds) fetch<T>(rc[i], p.Cm, oc[i], okb, p.eC, p.status);
            ob[i] += TT * p.B_st; oc[i] += TT * p.C_st;
        }
    };
    load(pc.len);
    f32x2 total[2] = {};
    for (int left = pc.len; left > 0; left -= TT) {
        const Eight<T> px = rx, pz = rz;              // what the tile's outputs need again
        if (stages) {
            const bool ok = xlive && xt < left;
            f32x2 x[4], d[4];
            rx.get(x);
            rd.get(d);
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = add2(d[e], bias[e]);
            if (p.softplus) {
#pragma unroll
                for (int e = 0; e < 4; ++e) d[e] = softplus_pair(d[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!ok) d[e] = both(0.f);            // past the end: exp(0) h + 0
                x[e] = mul2(x[e], d[e]);
            }
            ulonglong2 *to = reinterpret_cast<ulonglong2 *>(&sm.d[xt][xc]);
            to[0] = make_ulonglong2(d[0], d[1]);
            to[1] = make_ulonglong2(d[2], d[3]);
            to = reinterpret_cast<ulonglong2 *>(&sm.u[xt][xc]);
            to[0] = make_ulonglong2(x[0], x[1]);
            to[1] = make_ulonglong2(x[2], x[3]);
        }
#pragma unroll
        for (int i = 0; i < Sh::BPT; ++i) {
            const int v = tid + i * Sh::NT;
            if (v < Sh::BV) {
                f32x2 f[4];
                rb[i].get(f);
                ulonglong2 *to = reinterpret_cast<ulonglong2 *>(&sm.b[v / (N / 8)][v % (N / 8) * 8]);
                to[0] = make_ulonglong2(f[0], f[1]);
                to[1] = make_ulonglong2(f[2], f[3]);
                if (!kEnds) {
                    rc[i].get(f);
                    to = reinterpret_cast<ulonglong2 *>(&sm.c[v / (N / 8)][v % (N / 8) * 8]);
                    to[0] = make_ulonglong2(f[0], f[1]);
                    to[1] = make_ulonglong2(f[2], f[3]);
                }
            }
        }
        __syncthreads();
        load(left - TT);
        // the exponentials and inputs of the tokens are independent of the recurrence, which is one
        // multiply-add a token: unrolled, they run ahead of it
#pragma unroll 4
        for (int t = 0; t < TT; ++t) {
            const ulonglong2 dd = *reinterpret_cast<const ulonglong2 *>(&sm.d[t][ch]), uu = *reinterpret_cast<const ulonglong2 *>(&sm.u[t][ch]);
            const float4 bb = *reinterpret_cast<const float4 *>(&sm.b[t][4 * q]);
            const f32x2 d[2] = {dd.x, dd.y}, u[2] = {uu.x, uu.y}, b[4] = {both(bb.x), both(bb.y), both(bb.z), both(bb.w)};
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) step(j, n, d[j], mul2(u[j], b[n]));
            if (kEnds) {
                total[0] = add2(total[0], d[0]);
                total[1] = add2(total[1], d[1]);
            } else {
                const float4 cc = *reinterpret_cast<const float4 *>(&sm.c[kEnds ? 0 : t][4 * q]);
                f32x2 y2[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    y2[j] = fma2(both(cc.w), h[j][3], fma2(both(cc.z), h[j][2], fma2(both(cc.y), h[j][1], mul2(both(cc.x), h[j][0]))));
                // down to four lanes that hold parts of the same y: lanes give away half of their
                // channels, then half of what is left, then add whole values
                float *part = &sm.y[kEnds ? 0 : t][q & 3][ch];
                if (LPC == 4) {
                    *reinterpret_cast<ulonglong2 *>(part) = make_ulonglong2(y2[0], y2[1]);
                } else {
                    const float2 y01 = split(y2[0]), y23 = split(y2[1]);
                    const float y[4] = {y01.x, y01.y, y23.x, y23.y};
                    const bool hi4 = q & 4;
                    float r0 = hi4 ? y[2] : y[0], r1 = hi4 ? y[3] : y[1];
                    r0 += __shfl_xor_sync(0xffffffffu, hi4 ? y[0] : y[2], 4);
                    r1 += __shfl_xor_sync(0xffffffffu, hi4 ? y[1] : y[3], 4);
                    part += hi4 ? 2 : 0;
                    if (LPC == 8) {
                        *reinterpret_cast<float2 *>(part) = make_float2(r0, r1);
                    } else {
                        const bool hi8 = q & 8;
                        float r = hi8 ? r1 : r0;
                        r += __shfl_xor_sync(0xffffffffu, hi8 ? r0 : r1, 8);
                        if (LPC == 32) r += __shfl_xor_sync(0xffffffffu, r, 16);
                        if (q < 16) part[hi8 ? 1 : 0] = r;
                    }
                }
            }
        }
        __syncthreads();
        if (!kEnds && xlive && xt < left) {
            f32x2 y[4], x[4];
            px.get(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = mul2(skip[e], x[e]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 *part = reinterpret_cast<const ulonglong2 *>(&sm.y[kEnds ? 0 : xt][i][xc]);
                const ulonglong2 lo = part[0], hi = part[1];
                y[0] = add2(y[0], lo.x); y[1] = add2(y[1], lo.y);
                y[2] = add2(y[2], hi.x); y[3] = add2(y[3], hi.y);
            }
            if (gated) {
                f32x2 z[4];
                pz.get(z);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = mul2(y[e], silu_pair(z[e]));
                }
            }
            if (range_in_bounds(oo, 8, p.eo, p.status, nullptr)) {
                if (p.o_f32) {
                    ulonglong2 *o = reinterpret_cast<ulonglong2 *>(static_cast<float *>(p.o) + oo);
                    o[0] = make_ulonglong2(y[0], y[1]);
                    o[1] = make_ulonglong2(y[2], y[3]);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(split(y[e]).x, split(y[e]).y);
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + oo) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        oo += TT * p.o_st;
    }
    if (!live) return;
    if (kEnds) {
        store_h(end_of(pc.k));
        if (q == 0)
            *reinterpret_cast<ulonglong2 *>(p.sums + (int64_t)(pc.slot + pc.k) * p.C + c) = make_ulonglong2(total[0], total[1]);
    } else if (pc.k == pc.chunks - 1) {
        store_h(hs);
    }
}

// One token a sequence: a thread reads, updates and writes four states.  Bound by the state's bytes: 64 x 4,096 channels
// take 8.8 us (8.6 with rates that may be infinite), and 17.4 in the kernel above, which stages tiles of tokens.
constexpr int kStepThreads = 128;
template <typename T> __device__ __forceinline__ float4 four(const T *p);
template <> __device__ __forceinline__ float4 four<float>(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }
template <> __device__ __forceinline__ float4 four<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 r = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u), __uint_as_float(r.y << 16),
                       __uint_as_float(r.y & 0xFFFF0000u));
}

template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const ScanParams p) {
    constexpr int LPC = N / 4;
    const int q = threadIdx.x % LPC, b = blockIdx.y;
    int c = blockIdx.x * (kStepThreads / LPC) + threadIdx.x / LPC;
    const bool live = c < p.C;
    if (!live) c = 0;
    const int g = p.G == 1 ? 0 : c / p.Cg;
    float *hs = p.state + ((int64_t)b * p.C + c) * N + 4 * q;
    float4 h = *reinterpret_cast<const float4 *>(hs);
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p.A_log + (int64_t)c * N + 4 * q));
    auto one = [&](const void *base, int64_t off, int64_t n) {
        return in_bounds(off, n, p.status, nullptr) ? Cvt<T>::to_f(static_cast<const T *>(base)[off]) : 0.f;
    };
    auto quad = [&](const void *base, int64_t off, int64_t n) {
        return range_in_bounds(off, 4, n, p.status, nullptr) ? four<T>(static_cast<const T *>(base) + off)
                                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    const float x = one(p.x, b * p.x_sb + c, p.ex);
    float d = one(p.dt, b * p.dt_sb + c, p.edt) + (p.dt_bias != nullptr ? __ldg(p.dt_bias + c) : 0.f);
    const float4 bb = quad(p.Bm, b * p.B_sb + g * N + 4 * q, p.eB), cc = quad(p.Cm, b * p.C_sb + g * N + 4 * q, p.eC);
    if (p.softplus) d = split(softplus_pair(both(d))).x;
    const float u = d * x;
    h.x = fmaf(ex2(d * rate(a.x)), h.x, u * bb.x);
    h.y = fmaf(ex2(d * rate(a.y)), h.y, u * bb.y);
    h.z = fmaf(ex2(d * rate(a.z)), h.z, u * bb.z);
    h.w = fmaf(ex2(d * rate(a.w)), h.w, u * bb.w);
    if (live) *reinterpret_cast<float4 *>(hs) = h;
    float y = fmaf(cc.x, h.x, fmaf(cc.y, h.y, fmaf(cc.z, h.z, cc.w * h.w)));
#pragma unroll
    for (int k = LPC / 2; k > 0; k >>= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
    if (live && q == 0) {
        y += (p.D != nullptr ? __ldg(p.D + c) : 0.f) * x;
        if (p.z != nullptr) y *= silu_f(one(p.z, b * p.z_sb + c, p.ez));
        const int64_t off = b * p.o_sb + c;
        if (in_bounds(off, p.eo, p.status, nullptr)) {
            if (p.o_f32) static_cast<float *>(p.o)[off] = y;
            else static_cast<__nv_bfloat16 *>(p.o)[off] = __float2bfloat16_rn(y);
        }
    }
}

// Tokens of a chunk.  Two passes cost 1.7 times the instructions of one, but fill the SMs.  Measured on sequences of
// 1,000 tokens of 4,096 channels (0.84 warps to an SM each), whole / in chunks: two 136 / 70 us, four 142 / 152, six 188 / 213,
// eight 195 / 313.  So sequences of one length stay whole from three warps to an SM on; packed ones, whose lengths
// are not known here, from six (five of 1 to 1,000 tokens: 104 us in chunks, 150 whole).  The chunks are as many as
// make twelve warps, which is what fits at once (ten and sixteen: 14 and 13 % slower at one of 4,000 tokens).
int chunk_of(const cgdr_scan_args &a) {
    const int64_t sms = device_sms() > 0 ? device_sms() : 152;       // sizes workspaces without a device, too
    const int64_t warps = ((int64_t)a.C * a.N + 511) / 512;          // 16 states to a thread
    const int64_t n = a.cu ? a.n_tokens : (int64_t)a.B * a.T, longest = a.cu ? a.n_tokens : a.T;
    int64_t chunk = longest;
    if (warps * a.B < 3 * sms || a.cu) {
        chunk = n * warps / (12 * sms);
        // packed lengths are not known here: sequences up to twice the mean stay whole if there are enough
        if (warps * a.B >= 6 * sms && chunk < 2 * (n / a.B)) chunk = 2 * (n / a.B);
    }
    if (chunk < 64) chunk = 64;
    chunk = (chunk + 15) / 16 * 16;
    return (int)(chunk < longest ? chunk : longest);
}

// Workspace slots: chunks of the sequences that have several.
int64_t slots_of(const cgdr_scan_args &a, int chunk) {
    if (!a.cu) {
        const int64_t chunks = (a.T + chunk - 1) / chunk;
        return chunks > 1 ? a.B * chunks : 0;
    }
    return chunk < a.n_tokens ? 2 * ((int64_t)a.n_tokens / chunk) + 1 : 0;    // ceil(l / chunk) < 2 l / chunk for l > chunk
}

template <typename T, int N>
cgdr_status launch_scan(const cgdr_scan_args &a, ScanParams &p, cudaStream_t s) {
    if (!a.cu && a.T == 1) {
        constexpr int per = kStepThreads / (N / 4);
        scan_step_kernel<T, N><<<dim3((a.C + per - 1) / per, a.B), kStepThreads, 0, s>>>(p);
        return launched();
    }
    using Sh = ScanShape<N>;
    const int blocks = a.G * ((p.Cg + Sh::CH - 1) / Sh::CH);
    const int64_t pieces = a.cu ? (int64_t)a.n_tokens / p.chunk + a.B : (int64_t)a.B * ((a.T + p.chunk - 1) / p.chunk);
    if (pieces > 65535) return CGDR_ERR_UNSUPPORTED;
    if (p.slots > 0) {
        scan_kernel<T, N, true><<<dim3(blocks, p.slots), Sh::NT, 0, s>>>(p);
        if (cudaPeekAtLastError() != cudaSuccess) return launched();
    }
    scan_kernel<T, N, false><<<dim3(blocks, (unsigned)pieces), Sh::NT, 0, s>>>(p);
    return launched();
}

template <typename T>
cgdr_status launch_states(const cgdr_scan_args &a, ScanParams &p, cudaStream_t s) {
    switch (a.N) {
        case 16: return launch_scan<T, 16>(a, p, s);
        case 32: return launch_scan<T, 32>(a, p, s);
        case 64: return launch_scan<T, 64>(a, p, s);
        default: return launch_scan<T, 128>(a, p, s);
    }
}

bool empty(const cgdr_scan_args *a) { return a->B == 0 || (a->cu ? a->n_tokens : a->T) == 0; }

cgdr_status check(const cgdr_scan_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->B < 0 || a->C <= 0 || a->G <= 0 || (a->cu ? a->n_tokens : a->T) < 0 || a->C % a->G != 0) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || !dtype_ok(a->o_dtype)) return CGDR_ERR_UNSUPPORTED;
    if ((a->N != 16 && a->N != 32 && a->N != 64 && a->N != 128) || (a->C / a->G) % 8 != 0) return CGDR_ERR_UNSUPPORTED;
    if ((a->cu ? a->n_tokens : (int64_t)a->B * a->T) > kMaxTokens || a->B > 32768) return CGDR_ERR_UNSUPPORTED;
    if (empty(a)) return CGDR_OK;
    if (!a->x || !a->dt || !a->Bm || !a->Cm || !a->o || !a->A_log || !a->state) return CGDR_ERR_INVALID_ARG;
    if (!aligned_to(a->x, 16) || !aligned_to(a->dt, 16) || !aligned_to(a->z, 16) || !aligned_to(a->Bm, 16) ||
        !aligned_to(a->Cm, 16) || !aligned_to(a->o, 16) || !aligned_to(a->A_log, 16) || !aligned_to(a->state, 16) ||
        !aligned_to(a->D, 8) || !aligned_to(a->dt_bias, 8) || !aligned_to(a->cu, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    const int esz = esize(a->dtype), osz = esize(a->o_dtype);
    const bool tok = a->cu || a->T > 1, bat = !a->cu;
    const int64_t st[] = {a->x_st, a->dt_st, a->z ? a->z_st : 0, a->Bm_st, a->Cm_st};
    const int64_t sb[] = {a->x_sb, a->dt_sb, a->z ? a->z_sb : 0, a->Bm_sb, a->Cm_sb};
    for (int i = 0; i < 5; ++i)
        if ((tok && !row_stride_ok(st[i], esz)) || (bat && !row_stride_ok(sb[i], esz))) return CGDR_ERR_ALIGNMENT;
    if ((tok && !row_stride_ok(a->o_st, osz)) || (bat && !row_stride_ok(a->o_sb, osz))) return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

size_t workspace_of(const cgdr_scan_args &a) {
    if (!a.cu && a.T == 1) return 0;
    return (size_t)(slots_of(a, chunk_of(a)) * a.C * (a.N + 1)) * sizeof(float);
}

}  // namespace
}  // namespace cgdr

extern "C" {

size_t cgdr_scan_workspace_size(const cgdr_scan_args *a) {
    using namespace cgdr;
    return check(a) != CGDR_OK || empty(a) ? 0 : workspace_of(*a);
}

cgdr_status cgdr_scan(const cgdr_scan_args *a, void *ws, size_t ws_bytes, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || empty(a)) return st;
    const size_t need = workspace_of(*a);
    if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned_to(ws, 16))) return CGDR_ERR_WORKSPACE;
    ScanParams p{};
    p.B = a->B; p.T = a->T; p.C = a->C; p.G = a->G; p.Cg = a->C / a->G;
    p.n = a->cu ? a->n_tokens : a->B * a->T;
    p.softplus = a->softplus; p.o_f32 = a->o_dtype == CGDR_F32;
    p.x = a->x; p.x_sb = a->x_sb; p.x_st = a->x_st;
    p.dt = a->dt; p.dt_sb = a->dt_sb; p.dt_st = a->dt_st;
    p.z = a->z; p.z_sb = a->z_sb; p.z_st = a->z_st;
    p.Bm = a->Bm; p.B_sb = a->Bm_sb; p.B_st = a->Bm_st;
    p.Cm = a->Cm; p.C_sb = a->Cm_sb; p.C_st = a->Cm_st;
    p.o = a->o; p.o_sb = a->o_sb; p.o_st = a->o_st;
    p.A_log = a->A_log; p.D = a->D; p.dt_bias = a->dt_bias; p.state = a->state; p.cu = a->cu; p.status = a->status;
    const bool step = !a->cu && a->T == 1;
    p.chunk = step ? 1 : chunk_of(*a);
    p.slots = step ? 0 : (int)slots_of(*a, p.chunk);
    p.ends = static_cast<float *>(ws);
    p.sums = need > 0 ? p.ends + (int64_t)p.slots * a->C * a->N : nullptr;
    auto ext = [&](int64_t sb, int64_t st, int64_t d) { return a->cu ? extent3(1, 0, p.n, st, d) : extent3(a->B, sb, a->T, a->T > 1 ? st : 0, d); };
    p.ex = ext(a->x_sb, a->x_st, a->C); p.edt = ext(a->dt_sb, a->dt_st, a->C); p.ez = a->z ? ext(a->z_sb, a->z_st, a->C) : 0;
    p.eB = ext(a->Bm_sb, a->Bm_st, (int64_t)a->G * a->N); p.eC = ext(a->Cm_sb, a->Cm_st, (int64_t)a->G * a->N);
    p.eo = ext(a->o_sb, a->o_st, a->C);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == CGDR_BF16 ? launch_states<__nv_bfloat16>(*a, p, s) : launch_states<float>(*a, p, s);
}

}  // extern "C"
