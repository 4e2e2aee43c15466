// Matrix product of 8-bit operands with scales for blocks of 128 (cgdr_matmul), for few rows of x.
//
// What counts here is how fast w is read: o^T = w x^T, so that the 128 rows of the tensor core's tile are rows of w, and
// 16 to 64 rows of x are its columns.  A cluster of CTAs takes 128 rows of w, each CTA a part of K; the parts of a row of x
// are sent to one CTA of the cluster, which adds them in their order: no workspace, and no order of arrival in a result.
// Block by block of K as in the tiles kernel: a product in tensor memory, taken from there, scaled and added up in registers, a
// thread a row of w.
// One row by 12288 x 4096 (50.4 MB) takes 11.7 us, 64 rows by 4096 x 12288 14.2: the bytes at the copy rate are 7.4 and 7.6, the launch is
// 2, and the parts meet in 0.4 and 1.6 (they pass between shared memories at 17 bytes a clock).  A cluster barrier after the parts have been read
// cost 0.9, sends of 4 bytes instead of 16 another 0.4.
#include "fp8.cuh"

namespace cgdr {
namespace {

using namespace fp8;

constexpr int kRows = 128;                            // of w
constexpr int kSum = 128;                             // threads that add up
constexpr int kThreads = kSum + 64;                   // and a warp that copies, one that multiplies
constexpr int kAhead = 16;                            // blocks of K whose scales are brought in together
constexpr int kMaxSplit = 8;

template <int BT> struct Shape {
    static constexpr int residents = 2;               // CTAs of an SM
    static constexpr int stages = BT == 16 ? 5 : BT == 64 ? 3 : 4, sums = 4;
    static constexpr int a = kRows * kBlockK, b = BT * kBlockK, stage = a + b, columns = sums * BT;
    static constexpr int scales = stages * stage, meet = scales + kAhead * BT * 4, bars = meet + (BT + kMaxSplit - 1) * kRows * 4;
    enum { full, empty = full + stages, ready = empty + stages, taken = ready + sums, drain = taken + sums, met, never, count };
    static constexpr int bytes = bars + count * 8 + 1024;
    static_assert(residents * (bytes + 1024) <= 228 * 1024 && residents * columns <= 512, "shared and tensor memory of an SM");
};

__device__ __forceinline__ uint32_t at_rank(uint32_t addr, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// A phase 0 that is over, once more, so that what other CTAs of the cluster have sent is seen.
__device__ __forceinline__ bool seen_by_cluster(uint32_t bar) {
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(done) : "r"(bar) : "memory");
    return done != 0;
}

template <int BT>
__global__ void __launch_bounds__(kThreads, Shape<BT>::residents) matmul_few_kernel(const __grid_constant__ MatmulParams p, const int split) {
    using S = Shape<BT>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_stop;
    __shared__ uint32_t s_issued;                     // copies of this CTA (index-checking build)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    auto bar = [&](int i) { return base + S::bars + 8 * i; };
    const int tiles_t = (p.n + BT - 1) / BT, rank = blockIdx.x % split, unit = blockIdx.x / split, t0 = unit % tiles_t * BT, n0 = unit / tiles_t * kRows;
    const int have = min(BT, p.n - t0), slice = (have + split - 1) / split;     // rows of x; those whose sums meet in a CTA
    const int b0 = (int)((int64_t)p.blocks * rank / split), b1 = (int)((int64_t)p.blocks * (rank + 1) / split);

    if (tid == 0) {
        s_stop = 0;
        for (int i = 0; i < S::stages; ++i) {
            mbar_init(bar(S::full + i), 1);
            mbar_init(bar(S::empty + i), 1);
        }
        for (int i = 0; i < S::sums; ++i) {
            mbar_init(bar(S::ready + i), 1);
            mbar_init(bar(S::taken + i), kSum / 32);
        }
        mbar_init(bar(S::drain), 1);
        mbar_init(bar(S::met), 1);
        mbar_init(bar(S::never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        expect(bar(S::met), (split - 1) * max(min(slice, have - rank * slice), 0) * kRows * 4);
    }
    if (warp == kThreads / 32 - 1) tmem_alloc(smem_u32(&s_tmem), S::columns);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");       // this CTA's barriers exist (and are fenced)
    wait_for_inputs();
    const uint32_t tmem = s_tmem;
    auto wait = [&](int which, uint32_t parity) -> bool {
        if (mbar_try_wait(bar(which), parity)) return true;
        return keep_waiting(bar(which), parity, &s_stop, p.status, p.polls);
    };

    if (warp < kSum / 32) {
        const uint32_t t_lane = tmem + ((uint32_t)(32 * warp) << 16);
        const float *ws = p.ws + (int64_t)(n0 / kBlockK) * p.blocks;
        f32x2 acc[BT / 2];
#pragma unroll
        for (int c = 0; c < BT / 2; ++c) acc[c] = both(0.f);
        bool go = true;
        for (int b = b0; b < b1; ++b) {               // every warp takes part in the barriers, even when a wait gave up
            const int i = b - b0, sum = i % S::sums;
            if (i % kAhead == 0) {
                named_bar_sync<1, kSum>();
                for (int e = tid; e < kAhead * BT; e += kSum) {
                    const int t = e / kAhead, k = e % kAhead;
                    float s = 0.f;
                    if (b + k < b1 && t0 + t < p.n) s = p.xs[(int64_t)(t0 + t) * p.blocks + b + k] * ws[b + k];
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + S::scales + (k * BT + t) * 4), "f"(s) : "memory");
                }
                named_bar_sync<1, kSum>();
            }
            if (go) go = __all_sync(0xffffffffu, p.inject ? wait(S::never, 0) : wait(S::ready + sum, (i / S::sums) & 1));
            if (!go) continue;
            fence_after_sync();
            uint32_t d[2][16];
            const uint32_t from = t_lane + sum * BT, scale = base + S::scales + (i % kAhead) * BT * 4;
            ask16(from, d[0]);
#pragma unroll
            for (int c = 0; c < BT; c += 16) {
                uint32_t (&now)[16] = d[c / 16 & 1];
                there();
                pin(now);
                if (c + 16 < BT) ask16(from + c + 16, d[c / 16 + 1 & 1]);
                else {
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) arrive(bar(S::taken + sum));
                }
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    f32x2 s0, s1;
                    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(s0), "=l"(s1) : "r"(scale + (c + e) * 4));
                    acc[(c + e) / 2] = fma2(pair(__uint_as_float(now[e]), __uint_as_float(now[e + 1])), s0, acc[(c + e) / 2]);
                    acc[(c + e) / 2 + 1] = fma2(pair(__uint_as_float(now[e + 2]), __uint_as_float(now[e + 3])), s1, acc[(c + e) / 2 + 1]);
                }
            }
        }
        // Every product of this CTA is done, and with them every copy: its sums take the operands' place, [BT][128].  Row t of x
        // meets in CTA t / slice, which has room for every other CTA's part, [split][slice][128].
#pragma unroll
        for (int t = 0; t < BT; ++t) {
            const float2 f = cgdr::split(acc[t / 2]);
            if (go && t < have) asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + (t * kRows + tid) * 4), "f"(t % 2 ? f.y : f.x) : "memory");
        }
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        named_bar_sync<1, kSum>();
        for (int t = warp; t < have; t += kSum / 32) {   // (after a wait that gave up, too, whatever is there: so every part arrives)
            const int to = t / slice;
            if (to == rank) continue;
            const float4 x = *reinterpret_cast<const float4 *>(smem_raw + (base - smem_u32(smem_raw)) + (t * kRows + 4 * lane) * 4);
            asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];"
                         ::"r"(at_rank(base + S::meet + ((rank * slice + t - to * slice) * kRows + 4 * lane) * 4, to)), "r"(__float_as_uint(x.x)), "r"(__float_as_uint(x.y)),
                         "r"(__float_as_uint(x.z)), "r"(__float_as_uint(x.w)), "r"(at_rank(bar(S::met), to)) : "memory");
        }
        go = __all_sync(0xffffffffu, wait(S::met, 0) && seen_by_cluster(bar(S::met))) && go;
        const int col = n0 + 4 * lane, left = min(4, p.N - col);
        const int mine = go && left > 0 ? min(slice, have - rank * slice) : 0;
        constexpr int kAtOnce = 4;
        for (int i0 = warp; i0 < mine; i0 += kAtOnce * (kSum / 32)) {
            float o[kAtOnce][4];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
            for (int q = 0; q < split; ++q) {
                float4 x[kAtOnce];
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j)
                    x[j] = *reinterpret_cast<const float4 *>(smem_raw + (base - smem_u32(smem_raw)) + (q == rank ? 0 : S::meet) + ((q * slice + min(i0 + j * (kSum / 32), mine - 1)) * kRows + 4 * lane) * 4);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    o[j][0] += x[j].x; o[j][1] += x[j].y; o[j][2] += x[j].z; o[j][3] += x[j].w;
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int i = i0 + j * (kSum / 32);
                const int64_t at = (int64_t)(t0 + rank * slice + i) * p.o_st + col;
                if (i >= mine || !range_in_bounds(at, left, p.eo, p.status, nullptr)) continue;
                if (p.o_f32) {
                    float *dst = static_cast<float *>(p.o) + at;
                    if (left == 4) *reinterpret_cast<float4 *>(dst) = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
                    else
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < left) dst[e] = o[j][e];
                } else {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.o) + at;
                    if (left == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o[j][0], o[j][1]), pack_bf16x2(o[j][2], o[j][3]));
                    else
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            if (e < left) dst[e] = __float2bfloat16_rn(o[j][e]);
                }
            }
        }
    } else if (warp == kSum / 32) {
        bool go = true;
        int at = 0;
        for (; at < b1 - b0; ++at) {
            const int st = at % S::stages;
            if (at >= S::stages) go = __all_sync(0xffffffffu, wait(S::empty + st, (at / S::stages - 1) & 1));
            if (!go) break;
            copy_boxes(base + st * S::stage, S::a, S::stage, &p.mw, n0, &p.mx, t0, (b0 + at) * kBlockK, bar(S::full + st));
        }
        copies_land<S::stages>(bar(S::full), at);
        if (lane == 0) s_issued = at;
    } else {
        bool go = true;
        for (int at = 0; at < b1 - b0; ++at) {
            const int st = at % S::stages, sum = at % S::sums;
            if (at >= S::sums) go = wait(S::taken + sum, (at / S::sums - 1) & 1);
            if (go) go = wait(S::full + st, (at / S::stages) & 1);
            go = __all_sync(0xffffffffu, go);
            if (!go) break;
            fence_after_sync();
            mma_block<BT>(tmem + sum * BT, base + st * S::stage, base + st * S::stage + S::a);
            commit_warp(bar(S::empty + st));
            commit_warp(bar(S::ready + sum));
        }
        products_end(bar(S::drain));
    }
    __syncwarp();
    if (warp >= kSum / 32) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    fence_before_sync();
    __syncthreads();
    if (tid == 0) check_over<S::stages>(bar(S::full), s_issued, bar(S::drain), p.status);
    if (warp == kThreads / 32 - 1) {
        fence_after_sync();
        tmem_dealloc(tmem, S::columns);
    }
    // Every part has arrived, so nobody touches this CTA's shared memory any more, unless a wait gave up: then it stays until
    // the others have left or given up, too, and their parts, which they have sent by then, are here.
    if (s_stop) {
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        mbar_wait(bar(S::met), 0, kMatmulPolls);
    }
}

// Parts of K: as many as let all CTAs be resident at once, two on an SM.  Clusters of more than four leave more of them empty
// and take longer to meet, so they need a third of the SMs to spare or parts of eight blocks; every part has two blocks at least.  Measured, us:
//   N x K, n            parts 1     2     3     4     5     6     8
//   4096 x 4096, 1       10.1   7.3   6.8   6.5   6.9   7.0   6.7
//   4096 x 4096, 64      15.6  10.7   9.8   8.8   9.1   9.6  10.2
//   4096 x 4096, 128     15.7  10.8  11.0  10.2  14.9  15.5  16.3
//   12288 x 4096, 64     18.2  15.0  15.0  19.0  19.4  23.6  24.8
//   1000 x 4096, 64      15.1   9.7   8.4   7.3   7.0   6.7   6.4
//   1000 x 4096, 128     15.2   9.7   8.4   7.4   7.1   6.8   7.6
//   1000 x 4096, 384     15.7  10.3  10.5   9.5   9.2  13.6  14.6
//   4096 x 12288, 64     37.2  21.7  18.1  16.0  16.6  15.1  15.1
//   2048 x 1024, 64       7.8   6.1   6.0   5.5   5.4   5.5   6.4
int split_of(int64_t tiles, int blocks) {
    const int64_t sms = device_sms() > 0 ? device_sms() : 152;
    int64_t split = 19 * sms / (10 * tiles);
    if (split > 4 && split * tiles > 17 * sms / 10) split = 17 * sms / (10 * tiles) > 4 ? 17 * sms / (10 * tiles) : 4;
    if (split > kMaxSplit) split = kMaxSplit;
    if (split > 4 && split * tiles > 2 * sms / 3 && split * 8 > blocks) split = 2 * sms / (3 * tiles) > 4 ? 2 * sms / (3 * tiles) : 4;
    if (split > blocks / 2) split = blocks / 2;
    return split < 1 ? 1 : (int)split;
}

template <int BT> cgdr_status launch(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s) {
    static SmemOnce smem_once;
    if (!smem_limit_once(smem_once, reinterpret_cast<const void *>(matmul_few_kernel<BT>), Shape<BT>::bytes)) return CGDR_ERR_CUDA;
    if (!encode_rows(p.mx, a.x, a.K, a.n, a.x_st, BT) || !encode_rows(p.mw, a.w, a.K, a.N, a.w_st, kRows)) return CGDR_ERR_ALIGNMENT;
    const int64_t tiles = (int64_t)((a.n + BT - 1) / BT) * groups_of(a.N);
    const int split = split_of(tiles, p.blocks);
    if (tiles * split > INT32_MAX) return CGDR_ERR_UNSUPPORTED;
    return launch_early(matmul_few_kernel<BT>, (unsigned)(tiles * split), kThreads, Shape<BT>::bytes, s, split, p, split);
}

}  // namespace

// This kernel, where its tiles are few enough to be split, unless K is so short that there is little to split; where K is
// long, also where they just run all at once.  Here / the better of the two tile widths there, us:
//   4096 x 4096:   n = 64 8.5 / 11.1,    128 10.0 / 11.2,  256 12.8 / 11.3,  320 19.3 / 11.5
//   12288 x 4096:  n = 32 12.6 / 13.5,   64 14.1 / 13.6,   128 20.3 / 13.9
//   4096 x 12288:  n = 64 14.3 / 26.8,   128 17.8 / 28.6,  192 21.3 / 28.0,  256 27.0 / 28.2,  320 46.6 / 28.1
//   1000 x 4096:   n = 512 10.0 / 11.4,  640 10.9 / 11.5,  1000 12.6 / 11.5
//   512 x 512:     n = 16 3.4 / 3.6,     64 4.9 / 3.5
bool matmul_few(const cgdr_matmul_args &a) {
    if (a.path != CGDR_MATMUL_AUTO) return a.path == CGDR_MATMUL_FEW;
    const int64_t sms = device_sms() > 0 ? device_sms() : 152, tiles = (int64_t)((a.n + 63) / 64) * groups_of(a.N);
    if (a.n <= 16) return tiles <= 19 * sms / 10;
    return groups_of(a.K) > 8 && tiles <= (a.n <= 32 || groups_of(a.K) > 64 ? 19 : 12) * sms / 20;
}

// 16, 32 or 64 rows of x a tile.  (128 of them take an SM for one CTA: 13.1 us against 10.1 for 128 rows of 4096 x 4096.)
cgdr_status launch_matmul_few(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s) {
    return a.n <= 16 ? launch<16>(a, p, s) : a.n <= 32 ? launch<32>(a, p, s) : launch<64>(a, p, s);
}

}  // namespace cgdr
