// Attention over the 8-bit paged cache for many query rows (prompts): bf16 queries, D = 128.
//
// The same mathematics and number formats as cache_attend.cu, on tcgen05: a block takes 256 rows
// ((query token, head of the group) pairs of one request and key-value head) as two tiles of 128, and
// walks over the cache 64 tokens at a time.
//   - Four warps bring in k and v bytes by cp.async, two steps ahead, and turn them into fp16 tiles once for
//     both row tiles: k as it lies, v transposed on the way by stmatrix (rows d, columns tokens).
//   - Four threads issue the products: s = q k^T into tensor memory, and o += p v with p from tensor memory,
//     for each tile.  s of the next step is under way while p of this one is formed.
//   - Four warps for each row tile, a thread a row, read s, form p' = 2^(s + log2 vs - M + kUp), and put it
//     back as fp16.  o stays in tensor memory; it is rescaled when a row's maximum has grown by
//     more than 2^7, which after the first steps is rare.
// The tile is as wide as tensor memory allows (two o, two s and two p take 448 of 512 columns), because every row
// shares the conversions.  A step of 64 tokens by 256 rows is 16,384 exponentials (512 cycles of that unit),
// about 900 issue cycles of the four schedulers for softmax and conversions, and products of 768 cycles (q k^T, 64
// columns wide, is bound by reading q and k from shared memory: 384 cycles a tile, not 256) and 512.  It takes
// 1,980.  With the softmax cut down to a load and a store and no loader work it is 1,600 still: most of it is the
// products and the hand-overs between the warps, and two threads a row instead of one, with half of the softmax
// each, gained nothing (153 us against 139 for 8 x 128 tokens over 8,192).
// Three prompts of 500 to 2011 tokens over up to 4,000 cached ones, 32 heads on 8: 171 GFLOP in 209 us,
// 816 TFLOP/s, 42 % of what a large bf16 matrix product reaches; the rows kernel took 1,020 us there.
#include "cache_attend.cuh"
#include "tc05.cuh"

namespace cgdr {
namespace {

using namespace tc05;

constexpr int D = 128;
constexpr int kTile = 128;                            // rows of a tile
constexpr int kTok = 64;                              // cached tokens of a step
constexpr int kGroups = kTok / 16;                    // a group of 16 tokens lies in one page
constexpr int kSoft = 128;                            // softmax threads of a tile
constexpr int kLoad = 128;                            // loading threads
constexpr int kThreads = 2 * kSoft + kLoad + 4 * 32;  // and four warps that issue the products
constexpr int kRaw = 2 * kTok * D;                    // k and v bytes of a step
constexpr int kRawStages = 3;
constexpr uint32_t kPolls = 1u << 18;                 // of a wait, before it gives up (args.wait_polls, 0)

constexpr int kQBytes = kTile * D * 2, kKBytes = kTok * D * 2, kVBytes = D * kTok * 2;
constexpr int kOffQ = 0, kOffK = 2 * kQBytes, kOffV = kOffK + 2 * kKBytes, kOffRaw = kOffV + 2 * kVBytes;
constexpr int kOffScale = kOffRaw + kRawStages * kRaw;                // float2 [4][kGroups]: ring of four steps
constexpr int kOffRawScale = kOffScale + 4 * kGroups * 8;            // float2 [kRawStages][kGroups]: scales as copied
constexpr int kOffBar = kOffRawScale + kRawStages * kGroups * 8;
enum Bar { kQFull, kKFull, kKFree = kKFull + 2, kVFull = kKFree + 2, kVFree = kVFull + 2, kSFull = kVFree + 2, kSFree = kSFull + 2,
           kPFull = kSFree + 2, kPvDone = kPFull + 2, kDrain = kPvDone + 2, kNever = kDrain + 4, kBars };
constexpr int kBytes = kOffBar + kBars * 8 + 1024;    // and the room to align to 1024 bytes

constexpr int kTmemO = 0, kTmemS = 2 * D, kTmemP = kTmemS + 2 * kTok, kTmemCols = 512;

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Where a 16-byte piece of a token's 128 bytes is kept among them: its number xor this.
__device__ __forceinline__ int raw_swizzle(int token) { return ((token & 1) << 2) | ((token >> 1) & 3); }

__device__ __forceinline__ void stmatrix_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(addr));
    return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 64 consecutive fp32 columns of this thread's TMEM lane (warp-wide), in one instruction.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __noinline__ bool keep_waiting(uint32_t bar, uint32_t parity, volatile int *stop, int *status, uint32_t polls) {
    for (uint32_t it = 0; it < polls; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*stop) return false;
    }
    *stop = 1;
    report(status, (int)CGDR_ERR_TIMEOUT);
    return false;
}

__global__ void __launch_bounds__(kThreads, 1) cache_attend_prompt_kernel(const AttendParams p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_stop, s_never;          // a wait gave up: everybody leaves; (never set)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // the last rows, which see the most, first: what runs at the end is short
    const int b = blockIdx.y, hk = blockIdx.x, part = blockIdx.z % p.splits, pairs = gridDim.z / p.splits,
              pair_at = pairs - 1 - blockIdx.z / p.splits, row0 = pair_at * 2 * kTile;
    const Request rq = request(p, b);
    const int rows = rq.q_len * p.G, kv = rq.kv, behind = rq.behind;
    if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0 && cut(p, b)) report(p.status, (int)CGDR_ERR_CAPACITY);
    if (row0 >= rows) return;
    const int tiles = rows - row0 > kTile ? 2 : 1, last_row = min(row0 + 2 * kTile, rows) - 1;
    const int end = min(kv, behind + last_row / p.G + 1);             // what the last row sees
    const int all_steps = end > 0 ? (end + kTok - 1) / kTok : 0, share = (all_steps + p.splits - 1) / p.splits;
    const int steps = max(min(all_steps - part * share, share), 0), from = part * share * kTok;  // the part's, and its first position

    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    auto bar = [&](int i) { return base + kOffBar + 8 * i; };
    if (tid == 0) {
        s_stop = 0;
        mbar_init(bar(kQFull), tiles * kSoft / 32);
        s_never = 0;
        for (int i = 0; i < 4; ++i) mbar_init(bar(kDrain + i), 1);
        mbar_init(bar(kNever), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kKFull + i), kLoad / 32);
            mbar_init(bar(kVFull + i), kLoad / 32);
            mbar_init(bar(kKFree + i), tiles);
            mbar_init(bar(kVFree + i), tiles);
            mbar_init(bar(kSFull + i), 2);            // the products, and the thread that issued them (for what it has seen)
            mbar_init(bar(kSFree + i), kSoft / 32);
            mbar_init(bar(kPFull + i), kSoft / 32);
            mbar_init(bar(kPvDone + i), 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kThreads / 32 - 1) tmem_alloc(smem_u32(&s_tmem), kTmemCols);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = s_tmem;

    // false: this wait, or another thread's, gave up.  The first look is straight-line code: a wait that is
    // over already costs 50 cycles so, and 190 as a loop.
    auto wait = [&](int which, uint32_t parity) -> bool {
        if (mbar_try_wait(bar(which), parity)) return true;
        return keep_waiting(bar(which), parity, &s_stop, p.status, p.polls);
    };
    auto done = [&](int which) {                      // a warp's arrival
        __syncwarp();
        if (lane == 0) arrive(bar(which));
    };

    if (warp < 2 * kSoft / 32) {
        // ---------------------------------------------------------------- softmax: a thread a row
        const int tile = warp / (kSoft / 32), r = tid % kSoft, row = row0 + tile * kTile + r;
        if (tile < tiles) {
            const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
            const int tok = rq.first + row / p.G, head = hk * p.G + row % p.G;
            const bool ok = row < rows;
            const int seen = (ok ? min(behind + row / p.G + 1, kv) : 0) - from;
            const int all_see = (row0 + (tile + 1) * kTile <= rows ? min(kv, behind + (row0 + tile * kTile) / p.G + 1) : 0) - from;
            float scale;
            {
                // the row in fp16, scaled by a power of two to magnitudes below 2 (4 at the type's end)
                const int64_t off = (int64_t)tok * p.q_st + (int64_t)head * p.q_sh;
                uint4 raw[D / 8];                     // all of it at once: the row costs one latency
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    raw[c] = make_uint4(0, 0, 0, 0);
                    if (ok && range_in_bounds(off + 8 * c, 8, p.eq, p.status, nullptr))
                        raw[c] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + off) + c);
                }
                float top = 0.f;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    Vec<__nv_bfloat16>::unpack(raw[c], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
                }
                const int ex = top > 0x1p-100f && top < INFINITY ? min((int)(__float_as_uint(top) >> 23) - 127, 126) : 0;
                const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
                scale = __uint_as_float((uint32_t)(127 + ex) << 23) * p.scale * kLog2e;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    Vec<__nv_bfloat16>::unpack(raw[c], f);
                    sts128(base + kOffQ + tile * kQBytes + sw_off16(kTile, r, 8 * c), half2_bits(f[0] * down, f[1] * down),
                           half2_bits(f[2] * down, f[3] * down), half2_bits(f[4] * down, f[5] * down), half2_bits(f[6] * down, f[7] * down));
                }
                fence_smem_to_async();
                done(kQFull);
            }
            float M = kLowest, l = 0.f;
            bool go = true;
            const uint32_t t_s = tmem + lanes + kTmemS + tile * kTok, t_p = tmem + lanes + kTmemP + tile * (kTok / 2),
                           t_o = tmem + lanes + kTmemO + tile * D;
            for (int i = 0; i < steps && go; ++i) {
                go = __all_sync(0xffffffffu, p.inject ? wait(kNever, 0) : wait(kSFull + tile, i & 1));
                if (!go) break;
                fence_after_sync();
                float x[kTok];
                tmem_ld64(t_s, x);
                fence_before_sync();
                done(kSFree + tile);
                // x <- exponents s + log2 vs; their largest
                float iv[kGroups];
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    float ks, vs;
                    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks), "=f"(vs) : "r"(base + kOffScale + ((i & 3) * kGroups + g) * 8));
                    // a scale that is (as good as) zero: the values are zero, whatever the bytes; below zero: no page
                    const bool zero = vs < kZero;
                    // of a NaN 0, which leaves the rows that do not see it as they are: lv takes it to the others
                    iv[g] = zero ? kZeroInverse : fmaxf(rcp(vs), 0.f);
                    const f32x2 c = both(ks * scale), lv = both(vs < 0.f ? -INFINITY : zero ? kZeroLog : lg2(vs));
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 y = split(fma2(pair(x[16 * g + e], x[16 * g + e + 1]), c, lv));
                        x[16 * g + e] = y.x;
                        x[16 * g + e + 1] = y.y;
                    }
                }
                if ((i + 1) * kTok > all_see) {
#pragma unroll
                    for (int e = 0; e < kTok; ++e)
                        if (i * kTok + e >= seen) x[e] = -INFINITY;
                }
                float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int e = 4; e < kTok; ++e) m4[e & 3] = fmaxf(m4[e & 3], x[e]);
                const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                if (__any_sync(0xffffffffu, top > M + (kMost - kUp))) {
                    const float m = fmaxf(M, top), shrink = ex2(M - m);
                    M = m;
                    l *= shrink;
                    if (i > 0) {                      // o is at rest once the last step's product is done
                        go = __all_sync(0xffffffffu, wait(kPvDone + tile, (i - 1) & 1));
                        if (!go) break;
                        fence_after_sync();
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            float o[16];
                            tmem_ld16(t_o + c, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= shrink;
                            tmem_st16(t_o + c, o);
                        }
                    }
                }
                if (i > 0) {                          // the last step's p has been read
                    go = __all_sync(0xffffffffu, wait(kPvDone + tile, (i - 1) & 1));
                    if (!go) break;
                    fence_after_sync();
                }
                const f32x2 less = both(kUp - M);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float w[kTok / 4];                // fp16 pairs
#pragma unroll
                    for (int g = 2 * half; g < 2 * half + 2; ++g) {
                        f32x2 sum = both(0.f);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 d = split(add2(pair(x[16 * g + e], x[16 * g + e + 1]), less));
                            const float a = ex2(d.x), c = ex2(d.y);
                            sum = add2(sum, pair(a, c));
                            w[8 * (g & 1) + e / 2] = __uint_as_float(iv[g] < 0.f ? 0u : half2_bits(a, c));
                        }
                        l = fmaf(split(sum).x + split(sum).y, fabsf(iv[g]), l);
                    }
                    tmem_st16(t_p + 16 * half, w);
                }
                fence_before_sync();
                done(kPFull + tile);
            }
            if (steps > 0 && go) go = __all_sync(0xffffffffu, wait(kPvDone + tile, (steps - 1) & 1));
            if (go) {
                fence_after_sync();
                const float by = l == 0.f ? 0.f : 1.f / l;
                const int64_t off = (int64_t)tok * p.o_st + (int64_t)head * p.o_sh;
                const int64_t slot = (((int64_t)(b * p.Hkv + hk) * pairs + pair_at) * p.splits + part) * p.height + tile * kTile + r;
                if (p.splits > 1 && ok) *reinterpret_cast<float2 *>(p.ml + 2 * slot) = make_float2(M, l);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float o[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e) o[e] = 0.f;
                    if (steps > 0) {
                        tmem_ld32(t_o + 64 * h, *reinterpret_cast<float (*)[32]>(o));
                        tmem_ld32(t_o + 64 * h + 32, *reinterpret_cast<float (*)[32]>(o + 32));
                    }
                    if (ok) {
                        // column 8 m + 2 j + e, m = 8 h + 2 w + t, holds d = 64 h + 16 j + 4 w + 2 t + e
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int w = 0; w < 4; w += 2) {
                                float y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = o[16 * (w + e / 4) + 8 * (e / 2 % 2) + 2 * j + e % 2];
                                if (p.splits > 1) {
                                    float4 *to = reinterpret_cast<float4 *>(p.part + slot * D + 64 * h + 16 * j + 4 * w);
                                    to[0] = make_float4(y[0], y[1], y[2], y[3]);
                                    to[1] = make_float4(y[4], y[5], y[6], y[7]);
                                    continue;
                                }
                                const int64_t at = off + 64 * h + 16 * j + 4 * w;
                                if (!range_in_bounds(at, 8, p.eo, p.status, nullptr)) continue;
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = l == 0.f ? 0.f : y[e] * by;
                                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + at) = Vec<__nv_bfloat16>::pack(y);
                            }
                    }
                }
            }
        }
    } else if (warp < (2 * kSoft + kLoad) / 32) {
        // ---------------------------------------------------------------- loading and converting
        const int t = tid - 2 * kSoft, w = t >> 5;
        // Nothing here waits for a load in the step that issues it: page numbers are looked at a step after they
        // are asked for, and scales come with the copies.
        int page = -1;                                // lanes 0 .. 3: table entry of that group of the step to be copied next
        auto look = [&](int i) {
            const int pos = from + i * kTok + 16 * lane;
            const int64_t at = b * p.table_sb + (pos >> p.shift);
            page = -1;
            if (lane < kGroups && pos < end && in_bounds(at, p.e_table, p.status, nullptr)) page = __ldg(p.table + at);
        };
        // this thread's 16 bytes of a group: of token t / 8, piece t % 8 (the swizzle depends on the token modulo 8)
        const int64_t unit_bytes = (int64_t)D << p.shift, page_bytes = unit_bytes * p.Hkv;
        const int8_t *kc = p.kc + hk * unit_bytes + t * 16, *vc = p.vc + hk * unit_bytes + t * 16;
        const uint32_t mine = base + kOffRaw + (t >> 3) * D + ((t & 7) ^ raw_swizzle(t >> 3)) * 16;
        auto copy = [&](int i, int stage) {           // step i's bytes and scales; its pages are in `page`
            if (i < steps) {
                if (page >= p.num_pages) page = -1;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const int pg = __shfl_sync(0xffffffffu, page, g);
                    if (pg >= 0) {
                        const int64_t src = pg * page_bytes + ((from + i * kTok + 16 * g) & (p.page - 1)) * D;
                        const uint32_t to = mine + stage * kRaw + 16 * g * D;
                        cp_async16(to, kc + src, true);
                        cp_async16(to + kTok * D, vc + src, true);
                    }
                }
                if (t < kGroups) {                    // k's scale, then v's; below zero: no page
                    const uint32_t to = base + kOffRawScale + (stage * kGroups + t) * 8;
                    if (page >= 0) {
                        cp_async4(to, p.ks + (int64_t)page * p.Hkv + hk, true);
                        cp_async4(to + 4, p.vs + (int64_t)page * p.Hkv + hk, true);
                    } else {
                        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(0.f), "f"(-1.f) : "memory");
                        if (from + i * kTok + 16 * t < end) report(p.status, (int)CGDR_ERR_BOUNDS);
                    }
                }
            }
            cp_async_commit();
        };
        int stage = 0;                                // of raw bytes: i modulo 3
        look(0);
        copy(0, 0);
        look(1);
        copy(1, 1);
        look(2);
        bool go = true;
        for (int i = 0; i < steps; ++i) {             // every warp takes part in every step's barrier, even when a wait gave up
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            named_bar_sync<1, kLoad>();               // everybody's copies of step i, and their reads of step i - 1
            copy(i + 2, stage == 0 ? 2 : stage - 1);
            look(i + 3);
            const uint32_t raw = base + kOffRaw + stage * kRaw, raw_scale = base + kOffRawScale + (stage * kGroups + t) * 8;
            stage = stage == kRawStages - 1 ? 0 : stage + 1;
            const int st = i & 1;
            uint4 kv4[4];                             // 16 bytes of four keys
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int token = 16 * w + 8 * (n >> 1) + (lane & 7), piece = (lane >> 3) + 4 * (n & 1);
                kv4[n] = lds128(raw + token * D + (piece ^ raw_swizzle(token)) * 16);
            }
            if (go && i >= 2) go = __all_sync(0xffffffffu, wait(kKFree + st, ((i >> 1) - 1) & 1));
            if (!go) continue;
            // (the softmax threads have left step i - 4 behind: the products of step i - 2 are done, which were issued
            // after they had read s of step i - 3)
            if (t < kGroups) {
                uint32_t ks, vs;
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(ks), "=r"(vs) : "r"(raw_scale));
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(base + kOffScale + ((i & 3) * kGroups + t) * 8), "r"(ks), "r"(vs) : "memory");
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {             // two 16-byte pieces of a key's fp16 row each
                const int token = 16 * w + 8 * (n >> 1) + (lane & 7), piece = (lane >> 3) + 4 * (n & 1);
                const uint32_t a[4] = {kv4[n].x ^ 0x80808080u, kv4[n].y ^ 0x80808080u, kv4[n].z ^ 0x80808080u, kv4[n].w ^ 0x80808080u};
                const uint32_t to = base + kOffK + st * kKBytes;
                sts128(to + sw_off16(kTok, token, 16 * piece), low_pair(a[0]), high_pair(a[0]), low_pair(a[1]), high_pair(a[1]));
                sts128(to + sw_off16(kTok, token, 16 * piece + 8), low_pair(a[2]), high_pair(a[2]), low_pair(a[3]), high_pair(a[3]));
            }
            fence_smem_to_async();
            done(kKFull + st);
#pragma unroll
            for (int n = 0; n < 4; ++n) {             // and of four values: eight tokens (n / 2) by half of d (n % 2) at a time
                const int token = 8 * (2 * w + (n >> 1)) + (lane >> 2), piece = (lane & 3) + 4 * (n & 1);
                kv4[n] = lds128(raw + kTok * D + token * D + (piece ^ raw_swizzle(token)) * 16);
            }
            if (i >= 2) go = __all_sync(0xffffffffu, wait(kVFree + st, ((i >> 1) - 1) & 1));
            if (!go) continue;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const uint32_t a[4] = {kv4[n].x ^ 0x80808080u, kv4[n].y ^ 0x80808080u, kv4[n].z ^ 0x80808080u, kv4[n].w ^ 0x80808080u};
#pragma unroll
                for (int c = 0; c < 2; ++c) {         // four 8 x 8 tiles, of rows 8 m .. 8 m + 7 each
                    const int row = 8 * (8 * (n & 1) + 4 * c + (lane >> 3)) + (lane & 7);
                    stmatrix_t(base + kOffV + st * kVBytes + sw_off16(D, row, 8 * (2 * w + (n >> 1))), low_pair(a[2 * c]), high_pair(a[2 * c]),
                               low_pair(a[2 * c + 1]), high_pair(a[2 * c + 1]));
                }
            }
            fence_smem_to_async();
            done(kVFull + st);
        }
        cp_async_wait_all();
    } else {
        // ---------------------------------------------------------------- the products
        // A warp for each tile's scores and one for each tile's sums: issuing a product takes as long as it runs,
        // and waits cost hundreds of cycles, so one thread for all four left the tensor core idle two thirds of the time.
        const int which = warp - (2 * kSoft + kLoad) / 32, tile = which & 1;
        if (lane == 0 && tile < tiles && steps > 0) {
            bool go = true;
            if (which < 2) {
                go = wait(kQFull, 0);
                for (int i = 0; i < steps && go; ++i) {
                    go = wait(kKFull + (i & 1), (i >> 1) & 1);
                    if (go && i > 0) go = wait(kSFree + tile, (i - 1) & 1);
                    if (!go) break;
                    fence_after_sync();
                    gemm16<kTok, D>(tmem + kTmemS + tile * kTok, base + kOffQ + tile * kQBytes, base + kOffK + (i & 1) * kKBytes, false);
                    arrive(bar(kSFull + tile));
                    commit(bar(kSFull + tile));
                    commit(bar(kKFree + (i & 1)));
                }
            } else {
                for (int i = 0; i < steps && go; ++i) {
                    go = wait(kVFull + (i & 1), (i >> 1) & 1);
                    if (go) go = wait(kPFull + tile, i & 1);
                    if (!go) break;
                    fence_after_sync();
                    gemm16_ts<D, kTok>(tmem + kTmemO + tile * D, tmem + kTmemP + tile * (kTok / 2), base + kOffV + (i & 1) * kVBytes, i > 0);
                    commit(bar(kPvDone + tile));
                    commit(bar(kVFree + (i & 1)));
                }
            }
            if (!go) {                                // what was issued has to end before its memory is given up
                commit(bar(kDrain + which));
                keep_waiting(bar(kDrain + which), 0, &s_never, nullptr, kPolls);
            }
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    if (warp == kThreads / 32 - 1) {
        fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the parts of a row: a warp a row, four values a lane.
constexpr int kJoinRows = 8;
__global__ void __launch_bounds__(32 * kJoinRows) cache_join_prompt_kernel(const AttendParams p) {
    const int per = p.height / kJoinRows, hk = blockIdx.x / per, r = blockIdx.x % per * kJoinRows + (threadIdx.x >> 5), d = 4 * (threadIdx.x & 31);
    const int row = blockIdx.z * 2 * kTile + r;
    const Request rq = request(p, blockIdx.y);
    joined();
    if (row >= rq.q_len * p.G) return;
    const int64_t slot = ((int64_t)(blockIdx.y * p.Hkv + hk) * gridDim.z + blockIdx.z) * p.splits * p.height + r;
    float m = kLowest, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int i = 0; i < p.splits; ++i) {
        const float2 ml = *reinterpret_cast<const float2 *>(p.ml + 2 * (slot + (int64_t)i * p.height));
        const float4 x = *reinterpret_cast<const float4 *>(p.part + (slot + (int64_t)i * p.height) * D + d);
        const float top = fmaxf(m, ml.x), keep = ex2(m - top), add = ex2(ml.x - top);
        sum = fmaf(add, ml.y, sum * keep);
        o[0] = fmaf(add, x.x, o[0] * keep); o[1] = fmaf(add, x.y, o[1] * keep);
        o[2] = fmaf(add, x.z, o[2] * keep); o[3] = fmaf(add, x.w, o[3] * keep);
        m = top;
    }
    put_row<__nv_bfloat16>(p, rq.first + row / p.G, hk * p.G + row % p.G, d, o, sum);
}

struct Plan {
    int64_t pairs, blocks;
    int height, splits;                               // rows of a block, parts of the cache
    double us;
};
// The parts that a row pair's cache is cut into: as many as pay, in rounds of one block to an SM.  Measured (us): a round
// takes 1.02 for a step of 64 cached tokens and 10 to begin and end, 0.88 and 6 with one row tile; a second kernel, which
// joins the parts, adds 3 and 0.2 a part, and they pass at 8 TB/s, mostly through L2.  512 tokens of 8 heads, groups of 4, over 8192
// cached tokens: 83 in two parts, 140 in one; 128 tokens: 33 in eight, 140 in one.
Plan plan_of(const cgdr_attend_args &a) {
    const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv), sms = device_sms() > 0 ? device_sms() : 152;
    const int64_t kv = a.max_kv < (int64_t)a.width * a.page ? a.max_kv : (int64_t)a.width * a.page, steps = (kv + kTok - 1) / kTok;
    Plan best{(rows + 2 * kTile - 1) / (2 * kTile), 0, rows > kTile ? 2 * kTile : kTile, 1, 0.0};
    best.blocks = best.pairs * a.Hkv * a.B;
    for (int n = 1; n <= 32 && (n == 1 || 4 * n <= steps); ++n) {
        if (n > 1 && best.blocks * n > 2 * sms) break;
        const double rounds = (double)((best.blocks * n + sms - 1) / sms), step = best.height > kTile ? 1.02 : 0.88, ends = best.height > kTile ? 10.0 : 6.0;
        const double join = n > 1 ? 3.0 + 0.2 * n + (double)best.blocks * n * best.height * (D + 2) * 8.0 / 8e6 : 0.0;
        const double us = rounds * (ends + (double)((steps + n - 1) / n) * step) + join;
        if (n == 1 || us < best.us) { best.splits = n; best.us = us; }
    }
    return best;
}

}  // namespace

// Where this kernel covers the call and is expected to need less time than the other one, which was measured to take
// 16 rows past 24,000 cached tokens in a microsecond, and 10 more.  Both are taken to do max_q rows of every request.  For one
// of 2,000 tokens among 63 of one, 8,000 cached each, this kernel (706 us) is better than the other (3,164), and two calls,
// 170 and 229, than either.  8 heads, groups of 4; there / here:
//   1 request of 32 tokens:  512 cached 9.7 / 13.1, 2048 16 / 15, 8192 33 / 21
//   1 request of 128 tokens: 512 cached 12 / 19, 2048 28 / 21, 8192 91 / 33
//   8 requests of 16 tokens: 512 cached 12 / 13, 2048 28 / 24, 8192 93 / 67
bool attend_prompt_supported(const cgdr_attend_args &a) {
    const int64_t rows = (int64_t)a.max_q * (a.Hq / a.Hkv), pairs = (rows + 2 * kTile - 1) / (2 * kTile);
    if (a.path == CGDR_ATTEND_ROWS || a.dtype != CGDR_BF16 || a.D != D || pairs > 65535 || !aligned_to(a.o, 16) || (a.o_st | a.o_sh) % 8 != 0)
        return false;
    if (a.path == CGDR_ATTEND_TILES) return true;
    const double other = 10.0 + (double)a.B * a.Hkv * (double)((rows + 15) / 16) * (double)a.max_kv / 24000.0;
    return rows > 32 && plan_of(a).us < other;
}

size_t attend_prompt_workspace(const cgdr_attend_args &a) {
    const Plan plan = plan_of(a);
    return plan.splits > 1 ? (size_t)plan.blocks * plan.splits * plan.height * (D + 2) * sizeof(float) : 0;
}

cgdr_status launch_attend_prompt(const cgdr_attend_args &a, AttendParams &p, float *ws, cudaStream_t s) {
    static SmemOnce smem_once;
    if (!smem_limit_once(smem_once, reinterpret_cast<const void *>(cache_attend_prompt_kernel), kBytes)) return CGDR_ERR_CUDA;
    const Plan plan = plan_of(a);
    p.polls = a.wait_polls > 0 ? (uint32_t)a.wait_polls : a.wait_polls < 0 ? (uint32_t)(-(int64_t)a.wait_polls) : kPolls;
    p.inject = a.wait_polls < 0;
    p.splits = plan.splits;
    p.height = plan.height;
    p.part = ws;
    p.ml = ws != nullptr ? ws + (size_t)plan.blocks * plan.splits * plan.height * D : nullptr;
    cache_attend_prompt_kernel<<<dim3(a.Hkv, a.B, (unsigned)(plan.pairs * plan.splits)), kThreads, kBytes, s>>>(p);
    if (plan.splits > 1) {
        if (cudaPeekAtLastError() != cudaSuccess) return launched();
        cudaLaunchConfig_t c{};
        c.gridDim = dim3((unsigned)(a.Hkv * (plan.height / kJoinRows)), a.B, (unsigned)plan.pairs);
        c.blockDim = dim3(32 * kJoinRows);
        c.stream = s;
        cudaLaunchAttribute early{};
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        c.attrs = &early;
        c.numAttrs = 1;
        if (cudaLaunchKernelEx(&c, cache_join_prompt_kernel, p) != cudaSuccess) return launched();
    }
    return launched();
}

}  // namespace cgdr
