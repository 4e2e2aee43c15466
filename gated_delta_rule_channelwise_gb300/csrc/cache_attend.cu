// Attention over the 8-bit paged cache (cgdr_cache_attend).
//
// For single tokens the cache's bytes are the time: 2 D bytes a token and head are read once.  64 requests of 100
// to 8000 cached tokens, 8 heads of 128: 532 MB in 102 us, 5.2 TB/s; one of 131,071: 269 MB in 58 us.  Of both
// about 15 us are the launches, the first pages' latency and the join; the rest runs at 6.1 TB/s.  A warp
// takes 16 cached tokens at a time, all of D: a 16-token piece never crosses a page, is contiguous in
// the cache, and streams through the warp's own ring of shared-memory stages by cp.async, so the
// four warps of a block never wait for one another until they join their softmax states at the end.
// The tokens are the 16 rows of the mma.sync m16n8k16 products and the columns are queries: (query
// token, query head of the group) pairs that share one key-value head, eight or sixteen to a tile.
// Both products are taken transposed, s^T = k q^T and o^T = v^T p^T, so eight queries cost half of
// what sixteen do, in products and in registers; a p^T tile changes from result to operand by two
// 8 x 8 transpositions (movmatrix).  tcgen05 has no use here: its smallest tile has 64 rows.
//
// int8 -> fp16 is exact and takes no conversion instruction: the byte with its sign bit flipped,
// placed under the exponent byte 0x64, is the fp16 number 1024 + 128 + value, and one packed
// subtraction leaves the value.  The order of d within a product is free as long as both operands
// share it, so a lane reads contiguous bytes: of keys g = l / 4 and g + 8 its D/4 bytes from (l % 4) D/4
// on; of values 2j, 2j+1, 2j+8, 2j+9 (j = l % 4) its D/8 bytes from g D/8 on.
//
// The scales stay out of the products: k's multiplies the score; v's becomes part of the exponent,
// p' = 2^(s + log2 vs - M), with its own running maximum M of s + log2 vs, so that p' lies in (0, 1]
// whatever the scales are and fits fp16; the denominator adds p' / vs (of pages of zeros, which have
// no logarithm, see kZero).  M follows the maximum loosely:
// it is only looked for, over the lanes, when some score passes it by more than 2^7, which in a tile whose
// rows are all in use is rare after the first step, and a vote otherwise.  (Unused rows of a tile keep M at kLowest and
// pass it in every step, so a tile that is not full looks each time; their results go nowhere.)  p' is carried times 2^8: it stays below 2^15 even so,
// and keeps fp16's relative accuracy down to 2^-22 of the largest (2^-33 of it is where it ends).
//
// A unit is (request, row tile, key-value head), its cost the 128-token steps of its cache.  Where units are
// many or short each has a block; else, as lengths differ, every block takes an equal share of the steps of all
// units in a row.  A unit that one block has from end to end it writes out; of the others each block
// leaves a part (maximum, denominator, weighted sum), at most two of them, one for a unit that
// began before its share and one for a unit that goes on after it, and a second kernel joins a unit's parts.
//
// bf16 queries are scaled by a power of two per row to magnitudes below 2 and are then exact in fp16
// down to 2^-14 of the row's largest (beyond that their error is below 2^-25 of it).  fp32 queries
// and their probabilities are carried as two fp16 parts.
#include "cache_attend.cuh"

namespace cgdr {
namespace {

constexpr int kWarps = 4;
constexpr int kHalf = 16, kStep = 2 * kHalf;          // cached tokens of a product's tile, and of a warp's step
constexpr int kStages = 2;
static_assert(kBlockStep == kWarps * kStep, "a block's step");
constexpr int kMinShare = 2;                          // steps of a block's share at least: joining costs about as much
constexpr int kInfos = 320;                           // pages whose numbers and scales a block holds at a time

// The steps of all requests, and a block's share of them; worked out by a whole block of NT threads.
struct Share {
    int64_t total, size;                              // steps, steps of a block
};
template <int NT>
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t *s_sum) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    int64_t t = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) t += s_sum[w];
    return t;
}
template <int NT>
__device__ __forceinline__ Share share_of(const AttendParams &p, int64_t *s_sum) {
    int64_t mine = 0;
    for (int b = threadIdx.x; b < p.B; b += NT) {
        const Request r = request(p, b);
        mine += (int64_t)r.units * r.steps;
    }
    Share s;
    s.total = block_sum<NT>(mine, s_sum);
    s.size = max((s.total + p.blocks - 1) / p.blocks, (int64_t)kMinShare);
    return s;
}

__device__ __forceinline__ void mma_f16_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
constexpr int kMaxKv = 1 << 30;                       // positions stay well inside 32 bits

// What a block holds of a page, in 16 bytes.
struct PageInfo {
    int page;                                         // -1: outside the cache
    float k;                                          // k's scale
    float lv, iv;                                     // log2 and reciprocal of v's scale; kZeroLog and kZeroInverse where
                                                      // that is (as good as) zero, and so are the values
};

template <int D, int NQ, typename T>
struct AttendShape {                                                  // NQ: tiles of eight queries, 1 or 2
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;              // fp16 parts of q and p
    static constexpr int STAGE = 2 * kStep * D;                       // k and v bytes of a step
    static constexpr int RING = kWarps * kStages * STAGE;
    static constexpr int JOIN = kWarps * 8 * NQ * (D + 4) * 4;        // the warps' softmax states, in the ring's place
    static constexpr int BYTES = RING > JOIN ? RING : JOIN;
    static constexpr int BLOCKS = D == 128 ? (NQ == 1 && sizeof(T) == 2 ? 3 : 2) : 6 - NQ - (sizeof(T) == 4 ? 1 : 0); // of an SM, by registers
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {          // an 8 x 8 tile of fp16 over the warp
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Where a 16-byte piece of a 128-byte line of a stage is kept: its number xor this.  A quarter of a warp
// reads the keys of two tokens (every other piece of two lines) or the values of four pairs (two pieces
// of every other line): without it those meet the same banks two and four times.
template <int D>
__device__ __forceinline__ int k_swizzle(int line) { return D == 128 ? line & 1 : 0; }
template <int D>
__device__ __forceinline__ int v_swizzle(int line) { return D == 128 ? line & 6 : D == 64 ? (line & 3) << 1 : 0; }

// One unit's steps [step0, step1), by a whole block.
template <int D, int NQ, typename T>
__device__ __forceinline__ void attend_unit(const AttendParams &p, const Request &rq, int b, int unit, int step0, int step1,
                                            unsigned char *smem) {
    using Sh = AttendShape<D, NQ, T>;
    constexpr int PARTS = Sh::PARTS, KS = D / 16, MT = D / 16, R = 8 * NQ;            // k steps of k q^T, row tiles of v^T p^T
    PageInfo *info = reinterpret_cast<PageInfo *>(smem + Sh::BYTES);  // [kInfos + 1]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
    const int hk = unit % p.Hkv, row0 = unit / p.Hkv * R, rows = rq.q_len * p.G;
    const int kv = rq.kv, behind = rq.behind;
    const int last_row = min(row0 + R, rows) - 1;
    const int begin = step0 * kBlockStep;
    const int end = min(min(step1 * kBlockStep, kv), behind + last_row / p.G + 1);    // what some row of the tile sees
    const int all_see = min(kv, behind + row0 / p.G + 1);             // what every row sees

    // the queries' bytes first: they arrive while the pages are looked up
    uint4 raw[NQ][D / 4 / Vec<T>::n];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int row = row0 + 8 * n + g;
        const int64_t off = (int64_t)(rq.first + row / p.G) * p.q_st + (int64_t)(hk * p.G + row % p.G) * p.q_sh + j * (D / 4);
#pragma unroll
        for (int v = 0; v < D / 4 / Vec<T>::n; ++v) {
            raw[n][v] = make_uint4(0, 0, 0, 0);
            if (row < rows && range_in_bounds(off + v * Vec<T>::n, Vec<T>::n, p.eq, p.status, nullptr))
                raw[n][v] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + off) + v);
        }
    }
    unsigned char *ring = smem + warp * kStages * Sh::STAGE;
    const uint32_t ring_s = smem_u32(ring);
    const int span = kInfos * p.page;                  // cached tokens whose pages are held at a time
    // the pages of `span` tokens from `from` on, and the copies of the warp's first steps among them
    int steps = 0, page0 = 0, from = begin;
    auto issue = [&](int step, int stage) {           // copies of a step's 16 keys and 16 values
        if (step < steps) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = from + step * kStep + u * kHalf, page = info[(at >> p.shift) - page0].page;
                if (page >= 0) {
                    const int64_t src = ((((int64_t)page * p.Hkv + hk) << p.shift) + (at & (p.page - 1))) * D + lane * 16;
                    const uint32_t dst = ring_s + stage * Sh::STAGE + 2 * u * kHalf * D;
#pragma unroll
                    for (int c = 0; c < kHalf * D / 16 / 32; ++c) {
                        const int line = 4 * c + (lane >> 3), piece = lane & 7;
                        cp_async16(dst + line * 128 + (piece ^ k_swizzle<D>(line)) * 16, p.kc + src + c * 512, true);
                        cp_async16(dst + kHalf * D + line * 128 + (piece ^ v_swizzle<D>(line)) * 16, p.vc + src + c * 512, true);
                    }
                }
            }
        }
        cp_async_commit();
    };
    // Page numbers first, so that the copies can start; the scales are on their way meanwhile, and what is
    // made of them follows with ready().
    constexpr int kOf = (kInfos + 32 * kWarps) / (32 * kWarps);       // pages of a thread
    int last = 0;
    float ks[kOf], vs[kOf];
    auto open = [&]() {
        steps = (max(min(end - from, span), 0) + kStep - 1) / kStep;
        page0 = from >> p.shift;
        last = ((from + steps * kStep - 1) >> p.shift) - page0;
#pragma unroll
        for (int r = 0; r < kOf; ++r) {
            const int i = tid + r * 32 * kWarps;
            ks[r] = 0.f;
            vs[r] = 0.f;
            if (i <= last) {
                const int64_t at = b * p.table_sb + page0 + i;
                const bool held = (page0 + i) << p.shift < end;      // the last step may reach past the request's pages
                int page = held && in_bounds(at, p.e_table, p.status, nullptr) ? p.table[at] : -1;
                if (page < 0 || page >= p.num_pages) {
                    if (held) report(p.status, (int)CGDR_ERR_BOUNDS);
                    page = -1;
                } else {
                    ks[r] = __ldg(p.ks + (int64_t)page * p.Hkv + hk);
                    vs[r] = __ldg(p.vs + (int64_t)page * p.Hkv + hk);
                }
                info[i].page = page;
            }
        }
        __syncthreads();
        issue(warp, 0);
        issue(warp + kWarps, 1);
    };
    auto ready = [&]() {
#pragma unroll
        for (int r = 0; r < kOf; ++r) {
            const int i = tid + r * 32 * kWarps;
            if (i <= last) {
                // A NaN is not below kZero: by lv it reaches every row that sees the page.  iv leaves it out (fmaxf does),
                // as 0 times that would reach the denominators of the rows that do not.
                const bool zero = vs[r] < kZero;
                info[i].k = ks[r];
                info[i].lv = zero ? kZeroLog : log2f(vs[r]);
                info[i].iv = zero ? kZeroInverse : fmaxf(1.f / vs[r], 0.f);
            }
        }
        __syncthreads();
    };
    open();

    // query g of each tile as B operands, and what belongs to the queries 2 j, 2 j + 1 of this lane's results
    int seen[NQ][2];
    float row_scale[NQ][2];
    uint32_t qb[PARTS][NQ][KS][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        float f[D / 4];
#pragma unroll
        for (int v = 0; v < D / 4 / Vec<T>::n; ++v) Vec<T>::unpack(raw[n][v], f + v * Vec<T>::n);
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(f[e]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^ex <= top < 2^(ex + 1), or four times that at the type's end; rows of (almost) nothing stay as they are
        const int ex = top > 0x1p-100f && top < INFINITY ? min((int)(__float_as_uint(top) >> 23) - 127, 126) : 0;
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        const float scale = __uint_as_float((uint32_t)(127 + ex) << 23) * p.scale * kLog2e;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int mine = row0 + 8 * n + 2 * j + e;
            row_scale[n][e] = __shfl_sync(0xffffffffu, scale, 4 * (2 * j + e));
            seen[n][e] = mine < rows ? min(behind + mine / p.G + 1, kv) : 0;          // positions below this one
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float x = f[4 * s + 2 * c] * down, y = f[4 * s + 2 * c + 1] * down;
                const uint32_t hi = half2_bits(x, y);
                qb[0][n][s][c] = hi;
                if (PARTS == 2) {
                    const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                    qb[PARTS - 1][n][s][c] = half2_bits(x - back.x, y - back.y);
                }
            }
    }
    float M[NQ][2], l[NQ][2];
    float acc[MT][NQ][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        M[n][0] = M[n][1] = kLowest;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
    }

    ready();
    while (true) {
    int stage = 0;
    for (int step = warp; step < steps; step += kWarps) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();                                 // every lane's copies have landed
        const unsigned char *bytes = ring + stage * Sh::STAGE;
        PageInfo f[2];
        int at[2];                                    // of what lies outside the cache: a position that no row sees
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            at[u] = from + step * kStep + u * kHalf;
            f[u] = info[(at[u] >> p.shift) - page0];
            if (f[u].page < 0) at[u] = INT32_MAX - kHalf;
        }

        // scores: tokens g (0, 1) and g + 8 (2, 3) of each half for queries 2 j, 2 j + 1
        float s[2][NQ][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t w[2][D / 16];                    // bytes j D/4 .. (j+1) D/4 of keys g, g + 8
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const unsigned char *src = bytes + (2 * u * kHalf + g + 8 * t) * D;
                if (D >= 64) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 r = *reinterpret_cast<const uint4 *>(src + (((D / 64) * j + c) ^ k_swizzle<D>(g)) * 16);
                        w[t][4 * c] = r.x; w[t][4 * c + 1] = r.y; w[t][4 * c + 2] = r.z; w[t][4 * c + 3] = r.w;
                    }
                } else {
                    const uint2 r = *reinterpret_cast<const uint2 *>(src + 8 * j);
                    w[t][0] = r.x; w[t][1] = r.y;
                }
            }
#pragma unroll
            for (int n = 0; n < NQ; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.f;
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                const uint32_t x = w[0][c] ^ 0x80808080u, y = w[1][c] ^ 0x80808080u;
                const uint32_t a[4] = {low_pair(x), low_pair(y), high_pair(x), high_pair(y)};
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) mma_f16_16x8x16(s[u][n], a, qb[part][n][c][0], qb[part][n][c][1]);
            }
        }
        // p' = 2^d, d = s + log2 vs - (M - kUp); a NaN compares false and goes through
        float d[2][NQ][4];
        auto exponents = [&]() {
            bool more = false;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float c = f[u].k * row_scale[n][q], base = f[u].lv - (M[n][q] - kUp);
#pragma unroll
                        for (int e = q; e < 4; e += 2) d[u][n][e] = fmaf(s[u][n][e], c, base);
                    }
                if (at[u] + kHalf > all_see) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (at[u] + g + (e >> 1) * 8 >= seen[n][e & 1]) d[u][n][e] = -INFINITY;
                }
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) more |= d[u][n][e] > kMost;
            }
            return more;
        };
        if (__any_sync(0xffffffffu, exponents())) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float m = M[n][q];
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = q; e < 4; e += 2)
                            if (at[u] + g + (e >> 1) * 8 < seen[n][q]) m = fmaxf(m, fmaf(s[u][n][e], f[u].k * row_scale[n][q], f[u].lv));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                    const float shrink = ex2(M[n][q] - m);
                    M[n][q] = m;
                    l[n][q] *= shrink;
#pragma unroll
                    for (int i = 0; i < MT; ++i) { acc[i][n][q] *= shrink; acc[i][n][q + 2] *= shrink; }
                }
            exponents();
        }
        uint32_t pb[2][PARTS][NQ][2];                 // p' 2^kUp as B operands
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) d[u][n][e] = ex2(d[u][n][e]);
#pragma unroll
                for (int q = 0; q < 2; ++q) l[n][q] = fmaf(d[u][n][q] + d[u][n][q + 2], fabsf(f[u].iv), l[n][q]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float x = d[u][n][2 * h], y = d[u][n][2 * h + 1];
                    const uint32_t hi = half2_bits(x, y);
                    pb[u][0][n][h] = transposed(hi);
                    if (PARTS == 2) {
                        const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        pb[u][PARTS - 1][n][h] = transposed(half2_bits(x - back.x, y - back.y));
                    }
                }
            }
            if (f[u].iv < 0.f) {                      // whatever the bytes are, the values are zero
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int part = 0; part < PARTS; ++part) pb[u][part][n][0] = pb[u][part][n][1] = 0u;
            }
        }
        // v^T p^T: row g (g + 8) of tile i is d = g D/8 + 2 i (+ 1)
        constexpr int VB = D / 8;                     // bytes of a lane per value: 16, 8 or 4
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t v[4][VB / 4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int row = 2 * j + (t & 1) + 8 * (t >> 1), at16 = row * D + g * VB;
                const unsigned char *src = bytes + (2 * u + 1) * kHalf * D + (at16 ^ (v_swizzle<D>(at16 >> 7) * 16));
                if (VB == 16) {
                    const uint4 r = *reinterpret_cast<const uint4 *>(src);
                    v[t][0] = r.x; v[t][VB / 4 > 1 ? 1 : 0] = r.y; v[t][VB / 4 > 2 ? 2 : 0] = r.z; v[t][VB / 4 > 3 ? 3 : 0] = r.w;
                } else if (VB == 8) {
                    const uint2 r = *reinterpret_cast<const uint2 *>(src);
                    v[t][0] = r.x; v[t][VB / 4 > 1 ? 1 : 0] = r.y;
                } else {
                    v[t][0] = *reinterpret_cast<const uint32_t *>(src);
                }
            }
#pragma unroll
            for (int c = 0; c < VB / 4; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {         // bytes 0, 1 (2, 3) of both values of a pair, interleaved
                    const uint32_t sel = h ? 0x7362 : 0x5140;
                    const uint32_t x = __byte_perm(v[0][c], v[1][c], sel) ^ 0x80808080u, y = __byte_perm(v[2][c], v[3][c], sel) ^ 0x80808080u;
                    const uint32_t a[4] = {low_pair(x), high_pair(x), low_pair(y), high_pair(y)};
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) mma_f16_16x8x16(acc[2 * c + h][n], a, pb[u][part][n][0], pb[u][part][n][1]);
                }
        }
        __syncwarp();                                 // the stage is read before it is filled again
        issue(step + 2 * kWarps, stage);
        stage ^= 1;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                                  // infos and stages are free again
    from += span;
    if (from >= end) break;
    open();
    ready();
    }

    // join the four warps: [warp][row][M, l, -, -, o...] in the ring's place
    float *join = reinterpret_cast<float *>(smem);
    constexpr int W = D + 4;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float sum = l[n][q];
            sum += __shfl_xor_sync(0xffffffffu, sum, 4);
            sum += __shfl_xor_sync(0xffffffffu, sum, 8);
            sum += __shfl_xor_sync(0xffffffffu, sum, 16);
            float *to = join + (warp * R + 8 * n + 2 * j + q) * W;
            if (g == 0) *reinterpret_cast<float2 *>(to) = make_float2(M[n][q], sum);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2 *>(to + 4 + g * (D / 8) + 2 * i) = make_float2(acc[i][n][q], acc[i][n][q + 2]);
        }
    __syncthreads();
    for (int e = tid; e < R * D / 4; e += 32 * kWarps) {
        const int r = e / (D / 4), d = e % (D / 4) * 4, row = row0 + r;
        if (row >= rows) continue;
        const float *from = join + r * W;
        float m = kLowest;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, from[w * R * W]);
        float sum = 0.f;
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2(from[w * R * W] - m);
            const float4 x = *reinterpret_cast<const float4 *>(from + w * R * W + 4 + d);
            sum = fmaf(f, from[w * R * W + 1], sum);
            o[0] = fmaf(f, x.x, o[0]); o[1] = fmaf(f, x.y, o[1]); o[2] = fmaf(f, x.z, o[2]); o[3] = fmaf(f, x.w, o[3]);
        }
        if (step0 > 0 || step1 < rq.steps) {          // a part: of a unit begun before (0) or going on after (1)
            const int64_t slot = 2 * (int64_t)blockIdx.x + (step0 > 0 ? 0 : 1);
            *reinterpret_cast<float4 *>(p.part + (slot * R + r) * D + d) = make_float4(o[0], o[1], o[2], o[3]);
            if (d == 0) *reinterpret_cast<float2 *>(p.ml + (slot * R + r) * 2) = make_float2(m, sum);
        } else {
            put_row<T>(p, rq.first + row / p.G, hk * p.G + row % p.G, d, o, sum);
        }
    }
    __syncthreads();                                  // the ring is free again
}

template <int D, int NQ, typename T>
__global__ void __launch_bounds__(32 * kWarps, AttendShape<D, NQ, T>::BLOCKS) cache_attend_kernel(const AttendParams p) {
    constexpr int NT = 32 * kWarps;
    extern __shared__ __align__(128) unsigned char smem[];              // copies of 512 bytes: misaligned to a line, each takes two
    __shared__ int64_t s_sum[NT / 32], s_at;
    __shared__ int s_b;
    int b;
    int64_t left, at;                                 // steps to do, from this one of request b on
    if (p.whole) {
        b = blockIdx.y;
        const Request r = request(p, b);
        // the last rows, which see the most, first: what runs at the end is short (fp32, up to 400 tokens of four
        // requests over 2000 cached: 159 -> 151 us)
        at = (int64_t)(r.units - 1 - (int)blockIdx.x) * r.steps;
        left = (int)blockIdx.x < r.units ? r.steps : 0;
    } else {
        const Share share = share_of<NT>(p, s_sum);
        at = share.size * blockIdx.x;
        left = min(share.size, share.total - at);
        // the request of the first step, and the step in it: by prefix sums over groups of NT requests
        if (threadIdx.x == 0) s_b = p.B;
        for (int b0 = 0; left > 0 && b0 < p.B; b0 += NT) {
            int64_t mine = 0;
            if (b0 + threadIdx.x < p.B) {
                const Request r = request(p, b0 + threadIdx.x);
                mine = (int64_t)r.units * r.steps;
            }
            int64_t upto = mine;
            const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += x;
            }
            __syncthreads();
            if (lane == 31) s_sum[warp] = upto;
            __syncthreads();
            int64_t group = 0;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) {
                if (w < warp) upto += s_sum[w];
                group += s_sum[w];
            }
            if (at < group) {
                if (at < upto && at >= upto - mine) {
                    s_b = b0 + threadIdx.x;
                    s_at = at - (upto - mine);
                }
                break;
            }
            at -= group;
        }
        __syncthreads();
        b = s_b;
        at = b < p.B ? s_at : 0;
    }
    for (; b < p.B && left > 0; ++b) {
        const Request r = request(p, b);
        const int64_t all = (int64_t)r.units * r.steps;
        while (at < all && left > 0) {
            const int unit = (int)(at / r.steps), step0 = (int)(at % r.steps);
            const int step1 = (int)min((int64_t)r.steps, step0 + left);
            attend_unit<D, NQ, T>(p, r, b, unit, step0, step1, smem);
            at += step1 - step0;
            left -= step1 - step0;
        }
        at = at > all ? at - all : 0;
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < p.B; i += NT)
            if (cut(p, i)) report(p.status, (int)CGDR_ERR_CAPACITY);
}

// Joins the parts of a unit: four rows to a block, four groups of threads that take every fourth part.
constexpr int kJoinRows = 4, kJoinGroups = 4;
template <int D, typename T>
__global__ void __launch_bounds__(kJoinRows * kJoinGroups * D / 4) cache_join_kernel(const AttendParams p) {
    constexpr int LANES = kJoinRows * D / 4, NT = LANES * kJoinGroups;
    __shared__ int64_t s_sum[NT / 32];
    __shared__ float4 s_o[kJoinGroups][LANES];
    __shared__ float2 s_ml[kJoinGroups][LANES];
    const int b = blockIdx.z, unit = blockIdx.x, lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
    const Request rq = request(p, b);
    const int r = blockIdx.y * kJoinRows + lane / (D / 4), d = lane % (D / 4) * 4;
    const int row = unit / p.Hkv * p.tile + r, rows = rq.q_len * p.G;
    if (unit >= rq.units || unit / p.Hkv * p.tile + (int)blockIdx.y * kJoinRows >= rows) return joined();
    const Share share = share_of<NT>(p, s_sum);
    int64_t before = 0;
    for (int i = threadIdx.x; i < b; i += NT) {
        const Request x = request(p, i);
        before += (int64_t)x.units * x.steps;
    }
    const int64_t at = block_sum<NT>(before, s_sum) + (int64_t)unit * rq.steps;
    const int64_t first = at / share.size, last = (at + rq.steps - 1) / share.size;
    joined();
    if (first == last) return;                        // written out by its one block
    float m = kLowest, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int64_t c = first + group; c <= last; c += kJoinGroups) {
        const int64_t slot = 2 * c + (c == first ? 1 : 0);
        const float2 ml = *reinterpret_cast<const float2 *>(p.ml + (slot * p.tile + r) * 2);
        const float4 x = *reinterpret_cast<const float4 *>(p.part + (slot * p.tile + r) * D + d);
        const float top = fmaxf(m, ml.x), keep = ex2(m - top), add = ex2(ml.x - top);
        sum = fmaf(add, ml.y, sum * keep);
        o.x = fmaf(add, x.x, o.x * keep); o.y = fmaf(add, x.y, o.y * keep);
        o.z = fmaf(add, x.z, o.z * keep); o.w = fmaf(add, x.w, o.w * keep);
        m = top;
    }
    s_o[group][lane] = o;
    s_ml[group][lane] = make_float2(m, sum);
    __syncthreads();
    if (group != 0 || row >= rows) return;
    m = kLowest;
#pragma unroll
    for (int i = 0; i < kJoinGroups; ++i) m = fmaxf(m, s_ml[i][lane].x);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinGroups; ++i) {
        const float f = ex2(s_ml[i][lane].x - m);
        const float4 x = s_o[i][lane];
        sum = fmaf(f, s_ml[i][lane].y, sum);
        v[0] = fmaf(f, x.x, v[0]); v[1] = fmaf(f, x.y, v[1]); v[2] = fmaf(f, x.z, v[2]); v[3] = fmaf(f, x.w, v[3]);
    }
    put_row<T>(p, rq.first + row / p.G, unit % p.Hkv * p.G + row % p.G, d, v, sum);
}

// Rows of a tile: eight where that holds all of a request's (64 requests of one token and four heads: 102 us, 150 in
// tiles of 16).
int tile_of(const cgdr_attend_args &a) {
    const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv);
    return rows <= 8 ? 8 : 16;
}
int64_t most_of(const cgdr_attend_args &a) {
    return a.max_kv < (int64_t)a.width * a.page ? a.max_kv : (int64_t)a.width * a.page;
}
int64_t steps_of(const cgdr_attend_args &a) {         // of a unit at most
    const int64_t kv = most_of(a);
    return kv > 0 ? (kv + kBlockStep - 1) / kBlockStep : 1;
}
// Blocks of the first kernel that run at a time.
template <int D, int NQ, typename T>
int64_t resident() {
    return (int64_t)(device_sms() > 0 ? device_sms() : 152) * AttendShape<D, NQ, T>::BLOCKS;  // sizes workspaces without a device, too
}
template <int NQ>
int64_t tiles_of(const cgdr_attend_args &a) { return ((int64_t)a.max_q * (a.Hq / a.Hkv) + 8 * NQ - 1) / (8 * NQ); }
// Whether every unit goes to a block of its own, which needs no schedule, no workspace and no second kernel,
// but leaves the SMs to the longest unit where units are few or long.  With u = units / resident blocks, the
// limit is 8 steps of 128 tokens where u is small and 40 from u = 1 on.  Measured (bf16, D 128, whole / shared;
// lengths spread from 100 to the stated one; units of one token and four heads unless said):
//   u 0.14: 1024 tokens 9.9 / 11.5 us, 2048 16.8 / 12.6       u 0.6 (8 tokens): 4096 45 / 58, 8192 83 / 75
//   u 1.1:  1024 21 / 32, 4096 59 / 67, 8192 110 / 105        u 2.2: 4096 106 / 116, 8192 207 / 193
// Tiles of 16 rows have no limit from u = 1.5 on: a block that takes several of their units one after the other
// waits for instructions a third of its time (fp32, u 1.7: 8192 tokens 174 / 276; bf16, D 64, u 3.4: 204 / 274).
// Requests of unequal tokens launch blocks that find no unit; beyond a few for each that does, the shares win.
constexpr int kWholeSteps = 8, kWholeMore = 32, kWholeEmpty = 4;
template <int D, int NQ, typename T>
bool whole(const cgdr_attend_args &a) {
    const int64_t at_once = resident<D, NQ, T>(), grid = a.B * tiles_of<NQ>(a) * a.Hkv;
    const int64_t rows = ((int64_t)a.n * (a.Hq / a.Hkv) + 8 * NQ - 1) / (8 * NQ) * a.Hkv;      // units of full tiles
    const int64_t units = grid < rows + (int64_t)a.B * a.Hkv ? grid : rows + (int64_t)a.B * a.Hkv;
    if (grid > kWholeEmpty * (units > at_once ? units : at_once)) return false;
    if (NQ == 2 && 2 * units >= 3 * at_once) return true;
    return steps_of(a) <= kWholeSteps + kWholeMore * (units < at_once ? units : at_once) / at_once;
}
// Blocks of the first kernel where they share: all that fit, but no more than shares of kMinShare steps need.
template <int D, int NQ, typename T>
int blocks_of(const cgdr_attend_args &a) {
    const int64_t most = resident<D, NQ, T>();
    const int64_t need = ((int64_t)a.B * a.Hkv * tiles_of<NQ>(a) * steps_of(a) + kMinShare - 1) / kMinShare;
    return (int)(need < most ? need : most);
}
template <int D, int NQ, typename T>
size_t workspace_for(const cgdr_attend_args &a) {
    const int blocks = blocks_of<D, NQ, T>(a);
    return blocks > 1 && !whole<D, NQ, T>(a) ? (size_t)2 * blocks * 8 * NQ * (D + 2) * sizeof(float) : 0;
}

template <int D, int NQ, typename T>
cgdr_status launch_attend(const cgdr_attend_args &a, AttendParams &p, float *ws, cudaStream_t s) {
    using Sh = AttendShape<D, NQ, T>;
    static SmemOnce smem_once;
    constexpr int kBytes = Sh::BYTES + (kInfos + 1) * (int)sizeof(PageInfo);
    if (!smem_limit_once(smem_once, reinterpret_cast<const void *>(cache_attend_kernel<D, NQ, T>), kBytes)) return CGDR_ERR_CUDA;
    const int64_t tiles = tiles_of<NQ>(a);
    if (whole<D, NQ, T>(a)) {
        p.whole = 1;
        cache_attend_kernel<D, NQ, T><<<dim3((unsigned)(tiles * a.Hkv), a.B), 32 * kWarps, kBytes, s>>>(p);
        return launched();
    }
    p.blocks = blocks_of<D, NQ, T>(a);
    p.part = ws;
    p.ml = ws != nullptr ? ws + (size_t)2 * p.blocks * p.tile * D : nullptr;
    cache_attend_kernel<D, NQ, T><<<p.blocks, 32 * kWarps, kBytes, s>>>(p);
    if (p.blocks > 1) {
        if (cudaPeekAtLastError() != cudaSuccess) return launched();
        const int64_t rows = tiles > 1 ? p.tile : (int64_t)a.max_q * p.G;
        // begins while the first kernel ends, finds its unit, and waits for that kernel's parts
        cudaLaunchConfig_t c{};
        c.gridDim = dim3((unsigned)(tiles * a.Hkv), (unsigned)((rows + kJoinRows - 1) / kJoinRows), a.B);
        c.blockDim = dim3(kJoinRows * kJoinGroups * D / 4);
        c.stream = s;
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        c.attrs = &early;
        c.numAttrs = 1;
        if (cudaLaunchKernelEx(&c, cache_join_kernel<D, T>, p) != cudaSuccess) return launched();
    }
    return launched();
}

#define CGDR_ATTEND_CASES(CALL) \
    if (a.dtype == CGDR_BF16) { \
        if (tile_of(a) == 8) return a.D == 128 ? CALL(128, 1, __nv_bfloat16) : a.D == 64 ? CALL(64, 1, __nv_bfloat16) : CALL(32, 1, __nv_bfloat16); \
        return a.D == 128 ? CALL(128, 2, __nv_bfloat16) : a.D == 64 ? CALL(64, 2, __nv_bfloat16) : CALL(32, 2, __nv_bfloat16); \
    } \
    if (tile_of(a) == 8) return a.D == 128 ? CALL(128, 1, float) : a.D == 64 ? CALL(64, 1, float) : CALL(32, 1, float); \
    return a.D == 128 ? CALL(128, 2, float) : a.D == 64 ? CALL(64, 2, float) : CALL(32, 2, float);
size_t workspace_of(const cgdr_attend_args &a) {
#define CGDR_CALL(D, NQ, T) workspace_for<D, NQ, T>(a)
    CGDR_ATTEND_CASES(CGDR_CALL)
#undef CGDR_CALL
}
cgdr_status launch_of(const cgdr_attend_args &a, AttendParams &p, float *ws, cudaStream_t s) {
#define CGDR_CALL(D, NQ, T) launch_attend<D, NQ, T>(a, p, ws, s)
    CGDR_ATTEND_CASES(CGDR_CALL)
#undef CGDR_CALL
}
#undef CGDR_ATTEND_CASES

cgdr_status check(const cgdr_attend_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->B < 0 || a->n < 0 || a->Hq <= 0 || a->Hkv <= 0 || a->Hq % a->Hkv != 0 || a->width < 0 || a->num_pages < 0 ||
        a->max_q < 0 || a->max_kv < 0 || a->path < CGDR_ATTEND_AUTO || a->path > CGDR_ATTEND_TILES)
        return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || !page_ok(a->page) || (a->D != 32 && a->D != 64 && a->D != 128)) return CGDR_ERR_UNSUPPORTED;
    if (a->B > 65535 || a->n > kMaxTokens || a->max_kv >= kMaxKv) return CGDR_ERR_UNSUPPORTED;
    if (((int64_t)a->max_q * (a->Hq / a->Hkv) + 16) * a->Hkv > INT32_MAX) return CGDR_ERR_UNSUPPORTED;
    if (a->B == 0 || a->n == 0 || a->max_q == 0) return CGDR_OK;
    if (!a->q || !a->o || !a->kv_lens || !a->cu) return CGDR_ERR_INVALID_ARG;
    if (a->max_kv > 0 && a->width > 0 && (!a->k_cache || !a->v_cache || !a->k_scale || !a->v_scale || !a->block_table))
        return CGDR_ERR_INVALID_ARG;
    if (a->table_sb < (a->B > 1 ? a->width : 0)) return CGDR_ERR_INVALID_ARG;
    if (!aligned_to(a->q, 16) || !aligned_to(a->o, esize(a->dtype)) || !aligned_to(a->k_cache, 16) || !aligned_to(a->v_cache, 16) ||
        !aligned_to(a->k_scale, 4) || !aligned_to(a->v_scale, 4) || !aligned_to(a->block_table, 4) ||
        !aligned_to(a->kv_lens, 4) || !aligned_to(a->cu, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    const int esz = esize(a->dtype);
    if (!row_stride_ok(a->q_st, esz) || !row_stride_ok(a->q_sh, esz) || a->o_st < 0 || a->o_sh < 0) return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

}  // namespace
}  // namespace cgdr

extern "C" {

size_t cgdr_cache_attend_workspace_size(const cgdr_attend_args *a) {
    using namespace cgdr;
    if (check(a) != CGDR_OK || a->B == 0 || a->n == 0 || a->max_q == 0) return 0;
    return attend_prompt_supported(*a) ? attend_prompt_workspace(*a) : workspace_of(*a);
}

cgdr_status cgdr_cache_attend(const cgdr_attend_args *a, void *ws, size_t ws_bytes, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->B == 0 || a->n == 0 || a->max_q == 0) return st;
    const bool prompt = attend_prompt_supported(*a);
    const size_t need = prompt ? attend_prompt_workspace(*a) : workspace_of(*a);
    if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned_to(ws, 16))) return CGDR_ERR_WORKSPACE;
    AttendParams p{};
    p.B = a->B; p.n = a->n; p.Hq = a->Hq; p.Hkv = a->Hkv; p.G = a->Hq / a->Hkv; p.page = a->page; p.shift = __builtin_ctz(a->page); p.width = a->width;
    p.num_pages = a->num_pages; p.max_q = a->max_q;
    p.most = (int)most_of(*a); p.tile = tile_of(*a);
    p.scale = a->scale > 0.f ? a->scale : 1.f / sqrtf((float)a->D);
    p.q = a->q; p.q_st = a->q_st; p.q_sh = a->q_sh; p.o = a->o; p.o_st = a->o_st; p.o_sh = a->o_sh;
    p.eq = extent3(a->n, a->q_st, a->Hq, a->q_sh, a->D); p.eo = extent3(a->n, a->o_st, a->Hq, a->o_sh, a->D);
    p.kc = a->k_cache; p.vc = a->v_cache; p.ks = a->k_scale; p.vs = a->v_scale;
    p.table = a->block_table; p.table_sb = a->table_sb; p.e_table = (a->B - 1) * a->table_sb + a->width;
    p.kv_lens = a->kv_lens; p.cu = a->cu; p.status = a->status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return prompt ? launch_attend_prompt(*a, p, static_cast<float *>(ws), s) : launch_of(*a, p, static_cast<float *>(ws), s);
}

}  // extern "C"
