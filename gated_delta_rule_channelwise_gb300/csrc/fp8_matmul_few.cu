// Matrix product of 8-bit operands with scales for blocks of 128 (cgdr_matmul), for few rows of x.
//
// What counts here is how fast w is read: o^T = w x^T, so that the 128 rows of the tensor core's tile are rows of w, and
// the 16 to 128 rows of x are its columns.  A cluster of CTAs takes 128 rows of w, each CTA a part of K; their sums meet
// in shared memory, added in the order of the parts.  Block by block of K as in the tiles kernel: a product in tensor
// memory, taken from there, scaled and added up in registers, a thread a row of w.
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
    static constexpr int stages = BT == 16 ? 6 : BT == 32 ? 5 : BT == 64 ? 4 : 3, sums = BT == 128 ? 2 : 4;
    static constexpr int a = kRows * kBlockK, b = BT * kBlockK, stage = a + b, columns = sums * BT < 32 ? 32 : sums * BT;
    static constexpr int scales = stages * stage, bars = scales + kAhead * BT * 4;
    enum { full, empty = full + stages, ready = empty + stages, taken = ready + sums, drain = taken + sums, never, count };
    static constexpr int bytes = bars + count * 8 + 1024;
    static_assert(BT * kRows * 4 <= stages * stage, "the sums that meet take the place of the operands");
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int BT>
__global__ void __launch_bounds__(kThreads, 2) matmul_few_kernel(const __grid_constant__ MatmulParams p, const int split) {
    using S = Shape<BT>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_stop, s_never;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    auto bar = [&](int i) { return base + S::bars + 8 * i; };
    const int tiles_t = (p.n + BT - 1) / BT, rank = blockIdx.x % split, unit = blockIdx.x / split, t0 = unit % tiles_t * BT, n0 = unit / tiles_t * kRows;
    const int b0 = (int)((int64_t)p.blocks * rank / split), b1 = (int)((int64_t)p.blocks * (rank + 1) / split);

    if (tid == 0) {
        s_stop = 0;
        s_never = 0;
        for (int i = 0; i < S::stages; ++i) {
            mbar_init(bar(S::full + i), 1);
            mbar_init(bar(S::empty + i), 1);
        }
        for (int i = 0; i < S::sums; ++i) {
            mbar_init(bar(S::ready + i), 1);
            mbar_init(bar(S::taken + i), kSum / 32);
        }
        mbar_init(bar(S::drain), 1);
        mbar_init(bar(S::never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kThreads / 32 - 1) tmem_alloc(smem_u32(&s_tmem), S::columns);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
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
                    if (b + k < b1 && t0 + t < p.n) s = __ldg(p.xs + (int64_t)(t0 + t) * p.blocks + b + k) * __ldg(ws + b + k);
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
        // every product of this CTA is done, and with them every copy: its sums take the operands' place, [BT][128]
        if (go) {
#pragma unroll
            for (int c = 0; c < BT / 2; ++c) {
                const float2 f = cgdr::split(acc[c]);
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + (2 * c * kRows + tid) * 4), "f"(f.x) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((2 * c + 1) * kRows + tid) * 4), "f"(f.y) : "memory");
            }
        }
    } else if (warp == kSum / 32) {
        if (lane == 0) {
            bool go = true;
            int at = 0;
            for (; at < b1 - b0; ++at) {
                const int st = at % S::stages;
                if (at >= S::stages) go = wait(S::empty + st, (at / S::stages - 1) & 1);
                if (!go) break;
                expect(bar(S::full + st), S::stage);
                copy_box(base + st * S::stage, &p.mw, (b0 + at) * kBlockK, n0, bar(S::full + st));
                copy_box(base + st * S::stage + S::a, &p.mx, (b0 + at) * kBlockK, t0, bar(S::full + st));
            }
            if (!go)                                  // what is on its way has to land before the block ends
                for (int u = at > S::stages ? at - S::stages : 0; u < at; ++u)
                    keep_waiting(bar(S::full + u % S::stages), (u / S::stages) & 1, &s_never, nullptr, kMatmulPolls);
        }
    } else if (lane == 0) {
        bool go = true;
        for (int at = 0; at < b1 - b0; ++at) {
            const int st = at % S::stages, sum = at % S::sums;
            if (at >= S::sums) go = wait(S::taken + sum, (at / S::sums - 1) & 1);
            if (go) go = wait(S::full + st, (at / S::stages) & 1);
            if (!go) break;
            fence_after_sync();
            mma_block<BT>(tmem + sum * BT, base + st * S::stage, base + st * S::stage + S::a);
            commit(bar(S::empty + st));
            commit(bar(S::ready + sum));
        }
        if (!go) {                                    // and what was issued has to end
            commit(bar(S::drain));
            keep_waiting(bar(S::drain), 0, &s_never, nullptr, kMatmulPolls);
        }
    }
    __syncwarp();
    fence_before_sync();
    cluster_sync();                                   // everybody's sums are there
    if (warp < kSum / 32) {
        const int col = n0 + 4 * lane;
        for (int t = rank + split * warp; t < BT && t0 + t < p.n; t += split * (kSum / 32)) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < split; ++q) {
                uint32_t from;
                float x[4];
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(base + (t * kRows + 4 * lane) * 4), "r"(q));
                asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(from));
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += x[e];
            }
            const int64_t at = (int64_t)(t0 + t) * p.o_st + col;
            const int have = min(4, p.N - col);
            if (have <= 0 || !range_in_bounds(at, have, p.eo, p.status, nullptr)) continue;
            if (p.o_f32) {
                float *dst = static_cast<float *>(p.o) + at;
                if (have == 4) *reinterpret_cast<float4 *>(dst) = make_float4(o[0], o[1], o[2], o[3]);
                else
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (e < have) dst[e] = o[e];
            } else {
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.o) + at;
                if (have == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
                else
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (e < have) dst[e] = __float2bfloat16_rn(o[e]);
            }
        }
    }
    __syncwarp();
    cluster_sync();                                   // nobody leaves while its sums are read
    if (warp == kThreads / 32 - 1) {
        fence_after_sync();
        tmem_dealloc(tmem, S::columns);
    }
}

// Parts of K.
int split_of(const cgdr_matmul_args &a, int tiles) {
    const int64_t sms = device_sms() > 0 ? device_sms() : 152;
    const int blocks = groups_of(a.K);
    int best = 1;
    int64_t least = INT64_MAX;
    for (int s = 1; s <= kMaxSplit && s <= blocks; ++s) {
        const int64_t waves = ((int64_t)tiles * s + 2 * sms - 1) / (2 * sms), cost = waves * ((blocks + s - 1) / s + 3);
        if (cost < least) { least = cost; best = s; }
    }
    return best;
}

template <int BT> cgdr_status launch(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s) {
    static SmemOnce smem_once;
    if (!smem_limit_once(smem_once, reinterpret_cast<const void *>(matmul_few_kernel<BT>), Shape<BT>::bytes)) return CGDR_ERR_CUDA;
    if (!encode_rows(p.mx, a.x, a.K, a.n, a.x_st, BT) || !encode_rows(p.mw, a.w, a.K, a.N, a.w_st, kRows)) return CGDR_ERR_ALIGNMENT;
    const int64_t tiles = (int64_t)((a.n + BT - 1) / BT) * groups_of(a.N);
    const int split = split_of(a, (int)(tiles < INT32_MAX / 16 ? tiles : INT32_MAX / 16));
    if (tiles * split > INT32_MAX) return CGDR_ERR_UNSUPPORTED;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)(tiles * split));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = Shape<BT>::bytes;
    c.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = split;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, matmul_few_kernel<BT>, p, split) != cudaSuccess) { cudaGetLastError(); return CGDR_ERR_CUDA; }
    return launched();
}

}  // namespace

bool matmul_few(const cgdr_matmul_args &a) {
    return a.path == CGDR_MATMUL_FEW || (a.path == CGDR_MATMUL_AUTO && a.n <= 128);
}

cgdr_status launch_matmul_few(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s) {
    return a.n <= 16 ? launch<16>(a, p, s) : a.n <= 32 ? launch<32>(a, p, s) : a.n <= 64 ? launch<64>(a, p, s) : launch<128>(a, p, s);
}

}  // namespace cgdr
