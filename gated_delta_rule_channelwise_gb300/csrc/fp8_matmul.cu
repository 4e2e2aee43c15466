// Matrix product of 8-bit operands with scales for blocks of 128 (cgdr_matmul): entry point, and the kernel for
// tiles of 128 rows of x.
//
// The scales change with every block of K, so a block's product (four instructions of K = 32) is a sum of its own in
// tensor memory, which 256 threads take from there, scale and add up in registers: a thread has a row of x and half of the
// tile's columns, so that both scales are one number to it.  Two such sums fit tensor memory: one is formed while the other
// is taken.  One warp copies operands ahead, one issues the products.
// 4,001 x 12,288 x 4,096: 154 to 158 us (the GPU is near its power limit), 2,580 TFLOP/s, 0.68 of twice what a large bf16 product reaches.  A block of
// 128 x 256 x 128 takes 710 cycles there (the slope along K; without copies 680), the products alone 512, the sums alone 560, and a sum that is
// handed over and back waits 390; a tile begins and ends in 4,000 more, of which most is 64 KB of results on their way while every SM stores.
// A block of 128 columns takes 460 to 490, of which issuing takes 400 and its operands' way from L2 425.
#include "fp8.cuh"

namespace cgdr {
namespace {

using namespace fp8;

constexpr int kRows = 128;
constexpr int kSum = 256;                             // threads that add up
constexpr int kThreads = kSum + 128;                  // and the warps that copy, multiply and hold tensor memory
constexpr int kRegsSum = 224, kRegsRest = 56;         // 2 x 224 + 56 = 3 x 168, what the block is launched with
constexpr int kOutBytes = 32 * 128;                   // of a warp: 32 rows of 128 bytes

#ifdef CGDR_DEBUG_CHECKS
constexpr bool kInside = false;                       // every store is tested
#else
constexpr bool kInside = true;
#endif

template <int BN> struct Shape {
    static constexpr int stages = BN == 256 ? 4 : 6, sums = 512 / BN;
    static constexpr int a = kRows * kBlockK, b = BN * kBlockK, stage = a + b;
    static constexpr int out = stages * stage, bars = out + kSum / 32 * kOutBytes;
    enum { full, empty = full + stages, ready = empty + stages, taken = ready + sums, drain = taken + sums, never, count };
    static constexpr int bytes = bars + count * 8 + 1024;    // and the room to align to 1024 bytes
};

template <int BN>
__global__ void __launch_bounds__(kThreads, 1) matmul_tiles_kernel(const __grid_constant__ MatmulParams p) {
    using S = Shape<BN>;
    constexpr int kCols = BN / 2;                     // of a thread
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_stop;                   // a wait gave up: everybody leaves
    __shared__ uint32_t s_issued;                     // copies of this block (index-checking build)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    auto bar = [&](int i) { return base + S::bars + 8 * i; };
    const int tiles_m = (p.n + kRows - 1) / kRows, tiles_n = (p.N + BN - 1) / BN, tiles = tiles_m * tiles_n;

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
        mbar_init(bar(S::never), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kThreads / 32 - 1) tmem_alloc(smem_u32(&s_tmem), 512);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    wait_for_inputs();
    const uint32_t tmem = s_tmem;
    auto wait = [&](int which, uint32_t parity) -> bool {
        if (mbar_try_wait(bar(which), parity)) return true;
        return keep_waiting(bar(which), parity, &s_stop, p.status, p.polls);
    };

    if (warp < kSum / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSum));
        // ---------------------------------------------------------------- sums: a thread a row and half of the columns
        const int half = warp / 4, r = 32 * (warp & 3) + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + half * kCols;
        const uint32_t out = base + S::out + warp * kOutBytes;
        uint32_t at = 0;                              // sums taken so far
        bool go = true;
        const float *xs, *ws;
        float xn, wn;                                 // scales of the next block
        auto scales_of = [&](int tile) {
            const int row = tile % tiles_m * kRows + r, c = tile / tiles_m * BN + half * kCols;
            xs = p.xs + (int64_t)min(row, p.n - 1) * p.blocks;
            ws = p.ws + (int64_t)min(c / kBlockK, (p.N - 1) / kBlockK) * p.blocks;
            xn = *xs;
            wn = *ws;
        };
        scales_of(blockIdx.x);
        for (int tile = blockIdx.x; tile < tiles && go; tile += gridDim.x) {
            const int m0 = tile % tiles_m * kRows, c0 = tile / tiles_m * BN + half * kCols;
            f32x2 acc[kCols / 2];
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) acc[c] = both(0.f);
            for (int b = 0; b < p.blocks; ++b, ++at) {
                const f32x2 s = both(xn * wn);
                if (b + 1 < p.blocks) {
                    xn = xs[b + 1];
                    wn = ws[b + 1];
                }
                const int sum = at % S::sums;
                go = __all_sync(0xffffffffu, p.inject ? wait(S::never, 0) : wait(S::ready + sum, (at / S::sums) & 1));
                if (!go) break;
                fence_after_sync();
                uint32_t d[2][16];
                const uint32_t from = t_lane + sum * BN;
                ask16(from, d[0]);
#pragma unroll
                for (int c = 0; c < kCols; c += 16) {
                    uint32_t (&now)[16] = d[c / 16 & 1];
                    there();
                    pin(now);
                    if (c + 16 < kCols) ask16(from + c + 16, d[c / 16 + 1 & 1]);
                    else {
                        fence_before_sync();
                        __syncwarp();
                        if (lane == 0) arrive(bar(S::taken + sum));
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 2)
                        acc[(c + e) / 2] = fma2(pair(__uint_as_float(now[e]), __uint_as_float(now[e + 1])), s, acc[(c + e) / 2]);
                }
            }
            if (!go) break;
            if (tile + gridDim.x < tiles) scales_of(tile + gridDim.x);
            // a warp's 32 rows leave through shared memory, 128 bytes of each at a time
            const int osz = p.o_f32 ? 4 : 2;
#pragma unroll
            for (int part = 0; part < kCols / 32; ++part) {
                if (!p.o_f32 && part % 2) continue;
#pragma unroll
                for (int c = 0; c < 8; ++c) {         // 16 bytes each, at their number xor the row's
                    uint32_t w[4];
                    if (p.o_f32) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 f = split(acc[part * 16 + 2 * c + e]);
                            w[2 * e] = __float_as_uint(f.x);
                            w[2 * e + 1] = __float_as_uint(f.y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int i = part * 16 + 4 * c + e;
                            const float2 f = split(acc[i < kCols / 2 ? i : 0]);
                            w[e] = pack_bf16x2(f.x, f.y);
                        }
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(out + lane * 128 + ((c ^ (lane & 7)) << 4)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                                 "r"(w[3]) : "memory");
                }
                __syncwarp();
                const int to = m0 + 32 * (warp & 3) + (lane >> 3), n = 16 / osz, col = c0 + part * 32 + (lane & 7) * n;
                const int64_t e0 = (int64_t)to * p.o_st + col;
                unsigned char *dst = static_cast<unsigned char *>(p.o) + e0 * osz;
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int rr = 4 * i + (lane >> 3);
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w) : "r"(out + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4)));
                }
                if (kInside && m0 + 32 * (warp & 3) + 32 <= p.n && c0 + part * 32 + 8 * n <= p.N) {      // all of it
#pragma unroll
                    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4 *>(dst + 4 * i * p.o_st * osz) = v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (to + 4 * i >= p.n || col >= p.N || !range_in_bounds(e0 + 4 * i * p.o_st, min(n, p.N - col), p.eo, p.status, nullptr)) continue;
                        unsigned char *row = dst + 4 * i * p.o_st * osz;
                        if (col + n <= p.N) *reinterpret_cast<uint4 *>(row) = v[i];
                        else {
                            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                            for (int e = 0; e < p.N - col; ++e) {
                                if (p.o_f32) reinterpret_cast<uint32_t *>(row)[e] = e == 0 ? w[0] : e == 1 ? w[1] : w[2];
                                else reinterpret_cast<uint16_t *>(row)[e] = (uint16_t)((e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3]) >> (16 * (e & 1)));
                            }
                        }
                    }
                }
                __syncwarp();
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == kSum / 32) {
            // ---------------------------------------------------------------- copies
            uint32_t at = 0;
            bool go = true;
            for (int tile = blockIdx.x; tile < tiles && go; tile += gridDim.x) {
                const int m0 = tile % tiles_m * kRows, n0 = tile / tiles_m * BN;
                for (int b = 0; b < p.blocks; ++b, ++at) {
                    const int st = at % S::stages;
                    if (at >= S::stages) go = __all_sync(0xffffffffu, wait(S::empty + st, (at / S::stages - 1) & 1));
                    if (!go) break;
                    copy_boxes(base + st * S::stage, S::a, S::stage, &p.mx, m0, &p.mw, n0, b * kBlockK, bar(S::full + st));
                }
            }
            copies_land<S::stages>(bar(S::full), at);
            if (lane == 0) s_issued = at;
        } else if (warp == kSum / 32 + 1) {
            // ---------------------------------------------------------------- products
            uint32_t at = 0;
            bool go = true;
            for (int tile = blockIdx.x; tile < tiles && go; tile += gridDim.x) {
                for (int b = 0; b < p.blocks; ++b, ++at) {
                    const int st = at % S::stages, sum = at % S::sums;
                    go = wait(S::full + st, (at / S::stages) & 1) && (at < S::sums || wait(S::taken + sum, (at / S::sums - 1) & 1));
                    go = __all_sync(0xffffffffu, go);
                    if (!go) break;
                    fence_after_sync();
                    mma_block<BN>(tmem + sum * BN, base + st * S::stage, base + st * S::stage + S::a);
                    commit_warp(bar(S::ready + sum));
                    commit_warp(bar(S::empty + st));
                }
            }
            products_end(bar(S::drain));
        }
    }
    __syncwarp();
    fence_before_sync();
    __syncthreads();
    if (tid == 0) check_over<S::stages>(bar(S::full), s_issued, bar(S::drain), p.status);
    if (warp == kThreads / 32 - 1) {
        fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

cgdr_status check(const cgdr_matmul_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->n < 0 || a->N < 0 || a->K <= 0 || a->path < CGDR_MATMUL_AUTO || a->path > CGDR_MATMUL_TILES) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->o_dtype) || a->n > kMaxTokens || a->N > kMaxTokens || a->K > kMaxTokens) return CGDR_ERR_UNSUPPORTED;
    if ((int64_t)groups_of(a->n) * groups_of(a->N) > INT32_MAX / 2) return CGDR_ERR_UNSUPPORTED;
    if (a->n == 0 || a->N == 0) return CGDR_OK;
    if (!a->x || !a->x_scale || !a->w || !a->w_scale || !a->o || a->o == a->x || a->o == a->w) return CGDR_ERR_INVALID_ARG;
    if (a->n > 1 && (a->o_st < a->N || a->x_st < a->K)) return CGDR_ERR_INVALID_ARG;
    if (a->N > 1 && a->w_st < a->K) return CGDR_ERR_INVALID_ARG;
    if (!aligned_to(a->x, 16) || !aligned_to(a->w, 16) || !aligned_to(a->o, 16) || !aligned_to(a->x_scale, 4) || !aligned_to(a->w_scale, 4) ||
        !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    if (!row_stride_ok(a->x_st, 1) || !row_stride_ok(a->w_st, 1) || (a->n > 1 && !row_stride_ok(a->o_st, esize(a->o_dtype)))) return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

template <int BN> cgdr_status launch(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s) {
    static SmemOnce smem_once;
    if (!smem_limit_once(smem_once, reinterpret_cast<const void *>(matmul_tiles_kernel<BN>), Shape<BN>::bytes)) return CGDR_ERR_CUDA;
    const int sms = device_sms();
    if (sms <= 0) return CGDR_ERR_CUDA;
    if (!encode_rows(p.mx, a.x, a.K, a.n, a.x_st, kRows) || !encode_rows(p.mw, a.w, a.K, a.N, a.w_st, BN)) return CGDR_ERR_ALIGNMENT;
    const int64_t tiles = (int64_t)((a.n + kRows - 1) / kRows) * ((a.N + BN - 1) / BN);
    return launch_early(matmul_tiles_kernel<BN>, (unsigned)(tiles < sms ? tiles : sms), kThreads, Shape<BN>::bytes, s, 0, p);
}

}  // namespace

bool encode_rows(CUtensorMap &m, const void *base, int64_t K, int64_t rows, int64_t stride, int box) {
    const auto encode = tensor_map_encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? stride : (K + 15) / 16 * 16)};
    const cuuint32_t boxes[2] = {kBlockK, (cuuint32_t)box}, ones[2] = {1, 1};
    return encode(&m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cgdr_status launch_matmul_tiles(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s) {
    // A tile of 256 columns takes 14.0 us of K = 4096 where there are many, one of 128 8.9: 1500 rows of 4096 x 4096 (2 rounds of the SMs against
    // 3) 31.1 us and 30.2, 2500 (3 against 5) 44.9 and 47.7, 600 (1 against 2) 16.7 and 21.0 (each forced; what is taken now takes 30.0, 44.5 and 16.6).
    const int64_t sms = device_sms() > 0 ? device_sms() : 152, rows = (a.n + kRows - 1) / kRows;
    const int64_t wide = (rows * ((a.N + 255) / 256) + sms - 1) / sms, narrow = (rows * groups_of(a.N) + sms - 1) / sms;
    return 5 * wide <= 3 * narrow ? launch<256>(a, p, s) : launch<128>(a, p, s);
}

}  // namespace cgdr

extern "C" cgdr_status cgdr_matmul(const cgdr_matmul_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->n == 0 || a->N == 0) return st;
    MatmulParams p{};
    p.n = a->n; p.N = a->N; p.K = a->K; p.blocks = groups_of(a->K);
    p.xs = a->x_scale; p.ws = a->w_scale;
    p.o = a->o; p.o_st = a->n > 1 ? a->o_st : a->N; p.eo = extent3(1, 0, a->n, p.o_st, a->N);
    p.o_f32 = a->o_dtype == CGDR_F32;
    p.status = a->status;
    p.polls = a->wait_polls > 0 ? (uint32_t)a->wait_polls : a->wait_polls < 0 ? (uint32_t)(-(int64_t)a->wait_polls) : kMatmulPolls;
    p.inject = a->wait_polls < 0;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return matmul_few(*a) ? launch_matmul_few(*a, p, s) : launch_matmul_tiles(*a, p, s);
}
