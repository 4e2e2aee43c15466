// Selective state space scan (cgdr_scan): per channel c and state n
//     h[n] = exp(A[c, n] d) h[n] + d x B[n],   y = sum_n C[n] h[n],   A = -exp(A_log).
//
// A thread holds four states of one channel in registers, N/4 neighbouring lanes one channel, a
// block 16 channels.  The tokens come in tiles of 32: their rows are loaded into registers one tile
// ahead, turned into the fp32 values that the recurrence reads (d and d x once per channel, not once
// per state) and put into shared memory.
//
// The work is N exponentials and 4 N multiply-adds a token and channel, against 8 bytes: the scan is
// bound by instruction issue and the exponential unit, and, with few channels, by the length of the
// recurrence.  Then a sequence is cut into chunks.  The state that leaves a chunk is
// exp(A sum d) h_in + e, with e the chunk's own end state from zero, so one launch forms (sum d, e) of
// every chunk but the last, and a second runs all chunks, each joining its h_in from the pairs
// before it.  That does the exponentials twice, so chunks are as long as the SM count allows.
#include "serve.cuh"

namespace cgdr {
namespace {

constexpr int kCh = 16;                               // channels of a block
constexpr int kTok = 32;                              // tokens of a tile

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
// 2 atanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...); eight terms leave 2e-9 of it, and small results keep
// their relative accuracy, which a logarithm of 1 + t in fp32 would lose.
__device__ __forceinline__ float softplus_series(float x) {
    const float t = ex2(-kLog2e * fabsf(x));
    const float s = t * rcp(2.f + t), q = s * s;
    float r = 1.f / 15.f;
    r = fmaf(r, q, 1.f / 13.f);
    r = fmaf(r, q, 1.f / 11.f);
    r = fmaf(r, q, 1.f / 9.f);
    r = fmaf(r, q, 1.f / 7.f);
    r = fmaf(r, q, 1.f / 5.f);
    r = fmaf(r, q, 1.f / 3.f);
    r = fmaf(r, q, 1.f);
    return fmaxf(x, 0.f) + 2.f * s * r;
}

// Eight consecutive elements as stored, and as fp32.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const { Vec<__nv_bfloat16>::unpack(a, f); }
};
template <> struct Eight<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = __ldg(reinterpret_cast<const uint4 *>(p));
        b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        Vec<float>::unpack(a, f);
        Vec<float>::unpack(b, f + 4);
    }
};
template <typename T>
__device__ __forceinline__ void fetch(Eight<T> &v, const void *base, int64_t off, bool ok, int64_t n, int *st) {
    v.zero();
    if (ok && range_in_bounds(off, 8, n, st, nullptr)) v.load(static_cast<const T *>(base) + off);
}

// kEnds: the first launch (end states and sums of d of every chunk but a sequence's last).
template <typename T, int N, bool kEnds>
__global__ void __launch_bounds__(4 * N) scan_kernel(const ScanParams p) {
    constexpr int LPC = N / 4;                        // lanes of a channel
    __shared__ __align__(16) float2 s_du[kTok][kCh];  // d, d x
    __shared__ __align__(16) float s_B[kTok][N];
    __shared__ __align__(16) float s_C[kEnds ? 1 : kTok][N];
    __shared__ __align__(16) float s_y[kEnds ? 1 : kTok][kCh];
    const int tid = threadIdx.x, ch = tid / LPC, q = tid % LPC;
    const Piece pc = find_piece(p, blockIdx.y, kEnds);
    if (pc.b < 0 || (kEnds && pc.k == pc.chunks - 1)) return;
    if (pc.chunks > 1 && pc.slot + pc.chunks > p.slots) return;       // offsets that do not ascend: more tokens than there are
    const int per = (p.Cg + kCh - 1) / kCh;           // blocks of a group
    const int g = blockIdx.x / per, cg0 = (blockIdx.x % per) * kCh, c0 = g * p.Cg + cg0;
    const bool live = cg0 + ch < p.Cg;
    const int c = live ? c0 + ch : c0;

    float A[4], h[4];
    {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p.A_log + (int64_t)c * N + 4 * q));
        A[0] = -kLog2e * expf(a.x); A[1] = -kLog2e * expf(a.y); A[2] = -kLog2e * expf(a.z); A[3] = -kLog2e * expf(a.w);
    }
    auto load4 = [&](const float *src) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
    };
    float *hs = p.state + ((int64_t)pc.b * p.C + c) * N + 4 * q;
    auto end_of = [&](int k) { return p.ends + ((int64_t)(pc.slot + k) * p.C + c) * N + 4 * q; };
    if (pc.k == 0) {
        // the state of a sequence of several chunks is replaced by its last chunk's block, maybe
        // before this one starts: the first launch leaves a copy in the last chunk's slot
        if (kEnds || pc.chunks == 1) load4(hs);
        else load4(end_of(pc.chunks - 1));
        if (kEnds && live) *reinterpret_cast<float4 *>(end_of(pc.chunks - 1)) = make_float4(h[0], h[1], h[2], h[3]);
    } else if (kEnds) {
        h[0] = h[1] = h[2] = h[3] = 0.f;
    } else {                                          // join the chunks before this one
        load4(end_of(0));
        for (int k = 1; k < pc.k; ++k) {
            const float d = p.sums[(int64_t)(pc.slot + k) * p.C + c];
            const float4 e = *reinterpret_cast<const float4 *>(end_of(k));
            h[0] = fmaf(ex2(d * A[0]), h[0], e.x); h[1] = fmaf(ex2(d * A[1]), h[1], e.y);
            h[2] = fmaf(ex2(d * A[2]), h[2], e.z); h[3] = fmaf(ex2(d * A[3]), h[3], e.w);
        }
    }

    // staging: threads 0 .. 63 take eight channels of a token each, every thread eight states of B and C
    const int xt = tid >> 1, xc = (tid & 1) * 8;
    const bool xlive = tid < 2 * kTok && cg0 + xc < p.Cg;
    const int bt = tid / (N / 8), bn = (tid % (N / 8)) * 8;
    Eight<T> rx, rd, rz, rb, rc;
    float bias[8], skip[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        bias[e] = xlive && p.dt_bias != nullptr ? __ldg(p.dt_bias + c0 + xc + e) : 0.f;
        skip[e] = xlive && p.D != nullptr ? __ldg(p.D + c0 + xc + e) : 0.f;
    }
    const bool packed = p.cu != nullptr;
    auto row = [&](int64_t sb, int64_t st, int t) { return (packed ? 0 : pc.b * sb) + (int64_t)t * st; };
    auto load = [&](int first) {
        const int t = pc.t0 + first + xt, tb = pc.t0 + first + bt;
        const bool ok = xlive && first + xt < pc.len, okb = first + bt < pc.len;
        fetch<T>(rx, p.x, row(p.x_sb, p.x_st, t) + c0 + xc, ok, p.ex, p.status);
        fetch<T>(rd, p.dt, row(p.dt_sb, p.dt_st, t) + c0 + xc, ok, p.edt, p.status);
        fetch<T>(rb, p.Bm, row(p.B_sb, p.B_st, tb) + g * N + bn, okb, p.eB, p.status);
        if (!kEnds) {
            fetch<T>(rc, p.Cm, row(p.C_sb, p.C_st, tb) + g * N + bn, okb, p.eC, p.status);
            fetch<T>(rz, p.z, row(p.z_sb, p.z_st, t) + c0 + xc, ok && p.z != nullptr, p.ez, p.status);
        }
    };
    load(0);
    float total = 0.f;
    for (int first = 0; first < pc.len; first += kTok) {
        float dx[8], gate[8];                         // what the tile's outputs need again: D x, and the gate
        if (tid < 2 * kTok) {
            float x[8], d[8];
            rx.get(x);
            rd.get(d);
            const bool ok = xlive && first + xt < pc.len;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = d[e] + bias[e];
                if (p.softplus) v = softplus_series(v);
                if (!ok) v = 0.f;                     // past the end: exp(0) h + 0
                s_du[xt][xc + e] = make_float2(v, v * x[e]);
                dx[e] = skip[e] * x[e];
            }
            if (!kEnds) rz.get(gate);
        }
        {
            float f[8];
            rb.get(f);
            *reinterpret_cast<float4 *>(&s_B[bt][bn]) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4 *>(&s_B[bt][bn + 4]) = make_float4(f[4], f[5], f[6], f[7]);
            if (!kEnds) {
                rc.get(f);
                *reinterpret_cast<float4 *>(&s_C[bt][bn]) = make_float4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<float4 *>(&s_C[bt][bn + 4]) = make_float4(f[4], f[5], f[6], f[7]);
            }
        }
        __syncthreads();
        load(first + kTok);
#pragma unroll 4
        for (int t = 0; t < kTok; ++t) {
            const float2 du = s_du[t][ch];
            const float4 b = *reinterpret_cast<const float4 *>(&s_B[t][4 * q]);
            h[0] = fmaf(ex2(du.x * A[0]), h[0], du.y * b.x);
            h[1] = fmaf(ex2(du.x * A[1]), h[1], du.y * b.y);
            h[2] = fmaf(ex2(du.x * A[2]), h[2], du.y * b.z);
            h[3] = fmaf(ex2(du.x * A[3]), h[3], du.y * b.w);
            if (kEnds) total += du.x;
            else {
                const float4 cc = *reinterpret_cast<const float4 *>(&s_C[t][4 * q]);
                float y = cc.x * h[0];
                y = fmaf(cc.y, h[1], y);
                y = fmaf(cc.z, h[2], y);
                y = fmaf(cc.w, h[3], y);
#pragma unroll
                for (int d = LPC / 2; d > 0; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
                if (q == 0) s_y[t][ch] = y;
            }
        }
        __syncthreads();
        if (!kEnds && xlive && first + xt < pc.len) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y[e] = s_y[xt][xc + e] + dx[e];
                if (p.z != nullptr) y[e] *= silu_f(gate[e]);
            }
            const int64_t off = row(p.o_sb, p.o_st, pc.t0 + first + xt) + c0 + xc;
            if (range_in_bounds(off, 8, p.eo, p.status, nullptr)) {
                if (p.o_f32) {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.o) + off);
                    o[0] = make_float4(y[0], y[1], y[2], y[3]);
                    o[1] = make_float4(y[4], y[5], y[6], y[7]);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + off) = Vec<__nv_bfloat16>::pack(y);
                }
            }
        }
    }
    if (!live) return;
    if (kEnds) {
        *reinterpret_cast<float4 *>(end_of(pc.k)) = make_float4(h[0], h[1], h[2], h[3]);
        if (q == 0) p.sums[(int64_t)(pc.slot + pc.k) * p.C + c] = total;
    } else if (pc.k == pc.chunks - 1) {
        *reinterpret_cast<float4 *>(hs) = make_float4(h[0], h[1], h[2], h[3]);
    }
}

// One token a sequence: a thread reads, updates and writes four states.  Bound by the state's bytes.
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
    const int64_t unit = (int64_t)blockIdx.x * (kStepThreads / LPC) + threadIdx.x / LPC;
    const int q = threadIdx.x % LPC;
    const bool live = unit < (int64_t)p.B * p.C;
    const int b = live ? (int)(unit / p.C) : 0, c = live ? (int)(unit % p.C) : 0, g = c / p.Cg;
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
    if (p.softplus) d = softplus_series(d);
    const float u = d * x, s = -kLog2e * d;
    h.x = fmaf(ex2(s * expf(a.x)), h.x, u * bb.x);
    h.y = fmaf(ex2(s * expf(a.y)), h.y, u * bb.y);
    h.z = fmaf(ex2(s * expf(a.z)), h.z, u * bb.z);
    h.w = fmaf(ex2(s * expf(a.w)), h.w, u * bb.w);
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

// Tokens of a chunk: a sequence's whole length where the channels and sequences alone give every
// SM sub-partition a warp in flight for half the time that two passes would take; else as many
// chunks as give each two warps.
int chunk_of(const cgdr_scan_args &a) {
    const int64_t sms = device_sms() > 0 ? device_sms() : 152;       // sizes workspaces without a device, too
    const int64_t blocks = (int64_t)a.G * ((a.C / a.G + kCh - 1) / kCh), warps = blocks * (a.N / 8);
    const int64_t n = a.cu ? a.n_tokens : (int64_t)a.B * a.T, seqs = a.B;
    const int64_t longest = a.cu ? a.n_tokens : a.T;
    int64_t chunk = longest;
    if (warps * seqs < 2 * sms || a.cu) {
        chunk = n * warps / (8 * sms);
        // packed lengths are not known here: sequences up to twice the mean stay whole if there are enough
        if (warps * seqs >= 2 * sms && chunk < 2 * (n / seqs)) chunk = 2 * (n / seqs);
    }
    if (chunk < 2 * kTok) chunk = 2 * kTok;
    chunk = (chunk + kTok - 1) / kTok * kTok;
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
        const int64_t units = (int64_t)a.B * a.C, per = kStepThreads / (N / 4);
        scan_step_kernel<T, N><<<(unsigned)((units + per - 1) / per), kStepThreads, 0, s>>>(p);
        return launched();
    }
    const int blocks = a.G * ((p.Cg + kCh - 1) / kCh);
    const int64_t pieces = a.cu ? (int64_t)a.n_tokens / p.chunk + a.B : (int64_t)a.B * ((a.T + p.chunk - 1) / p.chunk);
    if (pieces > 65535) return CGDR_ERR_UNSUPPORTED;
    if (p.slots > 0) {
        scan_kernel<T, N, true><<<dim3(blocks, p.slots), 4 * N, 0, s>>>(p);
        if (cudaPeekAtLastError() != cudaSuccess) return launched();
    }
    scan_kernel<T, N, false><<<dim3(blocks, (unsigned)pieces), 4 * N, 0, s>>>(p);
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
        !aligned_to(a->D, 4) || !aligned_to(a->dt_bias, 4) || !aligned_to(a->cu, 4) || !aligned_to(a->status, 4))
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
