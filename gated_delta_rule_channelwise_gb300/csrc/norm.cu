// Root-mean-square norm with the residual's addition (cgdr_norm), and the 8-bit quantisers (cgdr_quantize).
//
// All of it is bound by memory.  4,001 rows of 4,096 bf16 with residual, in 8 bits (115 MB): 21.0 us, 17.0 at the copy rate.
// 128,000 heads of 128 bf16 out of packed rows (66 MB): 13.4 us, 9.7.  64 rows of 4,096: 2.3 us, a launch.  4,001 rows of 4,096 bf16
// into 8 bits (50 MB): 10.0 us, 7.3; a weight of 12288 x 4096 (151 MB): 25.0 us, 22.2.  4,001 rows of 4,096 fp32 with residual (262 MB):
// 50.8 us, 38.6; in 8 bits (213 MB) 38.4, 31.4.  Those forms, and others of fp32 with residual, spill 50 to 90 bytes a thread: the residency below was
// fitted on bf16, whose forms spill nothing.  Consecutive launches are 1.5 to 2 us apart, which
// these times include.
#include "layer.cuh"

namespace cgdr {
namespace {

struct NormParams {
    uint32_t rows;                                    // n * H
    int H, C, shift;                                  // 2^shift threads to a row
    uint64_t by_head;                                 // 2^64 / H, rounded up: row / H is the high word of the product
    float eps;
    const void *x;  int64_t x_st, x_sh;
    void *r;        int64_t r_st, r_sh;
    const float *weight;
    void *o;        int64_t o_st, o_sh;
    uint8_t *y8;    int64_t y8_st;
    float *scale;
    int64_t ex, er, eo, ey;                           // footprints (index-checking build)
    int *status;
};

// sum_i h_i^2 of a row, then h_i / sqrt(sum / C + eps) w_i.  A row is held by 2^shift threads, kVecs vectors of eight values a thread: one pass over the data.  The 16 lanes
// of a half warp hold 128 consecutive values, so a group's largest magnitude takes four shuffles.  A block stays and takes row after
// row, kRows at a time, with the weights in registers and the next rows on their way while it works on these (but for the longest
// rows, whose 1024 threads have no registers left for that): with a block for each row the first case takes 24.9 us, and 22.5 the
// second, which was bound by instructions, too, before values went in pairs.
constexpr int blocks_of(int vecs, int threads) { return threads > 256 ? 1 : vecs > 2 ? 2 : 4; }   // resident on an SM

template <typename T, int kVecs, int kRows, int kThreads, bool kResidual, bool k8>
__global__ void __launch_bounds__(kThreads, blocks_of(kVecs, kThreads)) norm_kernel(const NormParams p) {
    constexpr bool kKeep = kThreads < 1024;
    __shared__ float s_sum[2][kRows][32];
    const int tid = threadIdx.x, per = 1 << p.shift, t = tid & (per - 1);
    const uint32_t heads = p.H, side = blockDim.x >> p.shift, stride = gridDim.x * kRows * side;
    const float share = 1.f / (float)p.C;
    f32x2 w[kVecs][4];
    auto weights = [&](int j) {
        const int c = (t + (j << p.shift)) * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][e] = both(1.f);
        if (p.weight != nullptr && c < p.C) {
            Eight<float> raw;
            raw.load(p.weight + c);
            raw.unpack(w[j]);
        }
    };
    wait_for_inputs();
    if (kKeep)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) weights(j);
    Eight<T> xv[kRows][kVecs], rv[kRows][kVecs];
    auto offset = [&](uint32_t row, int64_t st, int64_t sh) {
        const uint32_t i = heads == 1 ? row : (uint32_t)__umul64hi(row, p.by_head);
        return (int64_t)i * st + (int64_t)(row - i * heads) * sh;
    };
    auto ask = [&](uint32_t first) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const uint32_t row = first + k * side;
            const int64_t x0 = offset(row, p.x_st, p.x_sh), r0 = kResidual ? offset(row, p.r_st, p.r_sh) : 0;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int c = (t + (j << p.shift)) * 8;
                xv[k][j].clear();
                rv[k][j].clear();
                if (row < p.rows && c < p.C) {
                    if (range_in_bounds(x0 + c, 8, p.ex, p.status, nullptr)) xv[k][j].load(static_cast<const T *>(p.x) + x0 + c);
                    if (kResidual && range_in_bounds(r0 + c, 8, p.er, p.status, nullptr)) rv[k][j].load(static_cast<T *>(p.r) + r0 + c);
                }
            }
        }
    };
    uint32_t first = blockIdx.x * kRows * side + (tid >> p.shift), last = blockIdx.x * kRows * side;
    if (kKeep) ask(first);
    for (int round = 0; last < p.rows; first += stride, last += stride, round ^= 1) {
        if (!kKeep) ask(first);
        f32x2 f[kRows][kVecs][4];
        float sum[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const uint32_t row = first + k * side;
            const int64_t r0 = kResidual ? offset(row, p.r_st, p.r_sh) : 0;
            f32x2 sums = both(0.f);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int c = (t + (j << p.shift)) * 8;
                xv[k][j].unpack(f[k][j]);
                if (kResidual) {
                    f32x2 g[4];
                    rv[k][j].unpack(g);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[k][j][e] = add2(f[k][j][e], g[e]);
                    if (row < p.rows && c < p.C && range_in_bounds(r0 + c, 8, p.er, p.status, nullptr)) Eight<T>::store(static_cast<T *>(p.r) + r0 + c, f[k][j]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) sums = fma2(f[k][j][e], f[k][j][e], sums);
            }
            const float2 v = split(sums);
            sum[k] = v.x + v.y;
        }
        if (kKeep) ask(first + stride);
        for (int o = min(per, 32) >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < kRows; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
        if (per > 32) {                               // always in the same order
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if ((tid & 31) == 0) s_sum[round][k][tid >> 5] = sum[k];
            __syncthreads();                          // (the other buffer is written before the next one of these)
#pragma unroll
            for (int k = 0; k < kRows; ++k) {
                sum[k] = 0.f;
                for (int i = 0; i < per / 32; ++i) sum[k] += s_sum[round][k][((tid >> p.shift) << (p.shift - 5)) + i];
            }
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const uint32_t row = first + k * side;
            const f32x2 by = both(__frsqrt_rn(sum[k] * share + p.eps));
            const int64_t o0 = k8 ? row * p.y8_st : offset(row, p.o_st, p.o_sh);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int v = t + (j << p.shift), c = v * 8;
                const bool in = row < p.rows && c < p.C;
                f32x2 y[4];
                if (!kKeep) weights(j);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(f[k][j][e], by), w[j][e]);
                if (k8) {
                    const float scale = scale_of(top_of_group(in ? top_of(y) : 0.f));
                    if (in && range_in_bounds(o0 + c, 8, p.ey, p.status, nullptr)) {
                        *reinterpret_cast<uint2 *>(p.y8 + o0 + c) = e4m3x8(y, __frcp_rn(scale));
                        if (v % 16 == 0) p.scale[(int64_t)row * ((p.C + kGroup - 1) / kGroup) + c / kGroup] = scale;
                    }
                } else if (in && range_in_bounds(o0 + c, 8, p.eo, p.status, nullptr)) {
                    Eight<T>::store(static_cast<T *>(p.o) + o0 + c, y);
                }
            }
        }
    }
}

template <typename T, int kVecs, int kRows, int kThreads, bool kResidual, bool k8>
cgdr_status launch_rows(const NormParams &p, cudaStream_t s) {
    const int per = 1 << p.shift, threads = per < 256 ? 256 : per, sms = device_sms();
    if (sms <= 0) return CGDR_ERR_CUDA;
    const uint32_t rows = kRows * (threads >> p.shift), need = (p.rows + rows - 1) / rows, most = sms * blocks_of(kVecs, kThreads);
    return launch_early(norm_kernel<T, kVecs, kRows, kThreads, kResidual, k8>, need < most ? need : most, threads, 0, s, 0, p);
}

template <typename T, int kVecs, int kRows, int kThreads>
cgdr_status launch_norm(const NormParams &p, cudaStream_t s) {
    if (p.r != nullptr)
        return p.y8 != nullptr ? launch_rows<T, kVecs, kRows, kThreads, true, true>(p, s) : launch_rows<T, kVecs, kRows, kThreads, true, false>(p, s);
    return p.y8 != nullptr ? launch_rows<T, kVecs, kRows, kThreads, false, true>(p, s) : launch_rows<T, kVecs, kRows, kThreads, false, false>(p, s);
}

template <typename T>
cgdr_status launch_vecs(NormParams &p, cudaStream_t s) {
    auto shift_for = [&](int v) {
        int sh = 4;
        while ((v * 8 << sh) < p.C) ++sh;
        return sh;
    };
    // Vectors of a thread.  4,096 columns: 21 us with two, 27 with one (512 threads a row).  128: 13.4 with two rows at a time, 14.7 with one.
    p.shift = shift_for(p.C <= 2048 ? 1 : p.C <= 4096 ? 2 : 4);
    return p.C <= 512     ? launch_norm<T, 1, 2, 256>(p, s)
           : p.C <= 2048  ? launch_norm<T, 1, 1, 256>(p, s)
           : p.C <= 4096  ? launch_norm<T, 2, 1, 256>(p, s)
           : p.C <= 8192  ? launch_norm<T, 4, 1, 256>(p, s)
           : p.C <= 16384 ? launch_norm<T, 4, 1, 512>(p, s)
                          : launch_norm<T, 4, 1, 1024>(p, s);
}

cgdr_status check(const cgdr_norm_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->n < 0 || a->H <= 0 || a->C <= 0) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->C % 8 != 0 || a->C > 32768 || a->n > kMaxTokens) return CGDR_ERR_UNSUPPORTED;
    if ((a->o != nullptr) == (a->y8 != nullptr) && a->n > 0) return CGDR_ERR_INVALID_ARG;
    if (a->y8 && a->H != 1) return CGDR_ERR_UNSUPPORTED;
    if (a->n == 0) return CGDR_OK;
    if (!a->x || (a->y8 && !a->y_scale)) return CGDR_ERR_INVALID_ARG;
    if (a->y8 && !disjoint(a->n, a->y8_st, 1, 0, a->C)) return CGDR_ERR_INVALID_ARG;
    if ((a->residual && !disjoint(a->n, a->residual_st, a->H, a->residual_sh, a->C)) || (a->o && !disjoint(a->n, a->o_st, a->H, a->o_sh, a->C)))
        return CGDR_ERR_INVALID_ARG;
    // In place: a thread reads what it holds of a row before it writes it, and no other row is there.
    if (a->o == a->x && ((a->n > 1 && a->o_st != a->x_st) || (a->H > 1 && a->o_sh != a->x_sh))) return CGDR_ERR_INVALID_ARG;
    if (a->y8 == a->x || (a->residual && (a->residual == a->x || a->residual == a->o || a->residual == a->y8))) return CGDR_ERR_INVALID_ARG;
    const int esz = esize(a->dtype);
    if (!aligned_to(a->x, 16) || !aligned_to(a->residual, 16) || !aligned_to(a->weight, 16) || !aligned_to(a->o, 16) ||
        !aligned_to(a->y8, 16) || !aligned_to(a->y_scale, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    if (!row_stride_ok(a->x_st, esz) || !row_stride_ok(a->x_sh, esz)) return CGDR_ERR_ALIGNMENT;
    if (a->residual && (!row_stride_ok(a->residual_st, esz) || !row_stride_ok(a->residual_sh, esz))) return CGDR_ERR_ALIGNMENT;
    if (a->o && (!row_stride_ok(a->o_st, esz) || !row_stride_ok(a->o_sh, esz))) return CGDR_ERR_ALIGNMENT;
    if (a->y8 && !row_stride_ok(a->y8_st, 1)) return CGDR_ERR_ALIGNMENT;
    return CGDR_OK;
}

struct QuantizeParams {
    int n, C, groups;
    const void *x; int64_t x_st, ex;
    uint8_t *y8;   int64_t y8_st, ey;
    float *scale;
    int *status;
};

constexpr int kQThreads = 256;
constexpr int kQGroups = 2;                           // groups of a half warp

// Rows: a half warp takes two groups of 128 values at a time (10.0 us in the first case above; one 11.8, four 11.3).
template <typename T>
__global__ void __launch_bounds__(kQThreads, 8) quantize_rows_kernel(const QuantizeParams p) {
    const int lane = threadIdx.x & 15, c = lane * 8;
    const int64_t units = (int64_t)p.n * p.groups, u0 = ((int64_t)blockIdx.x * kQGroups) * (kQThreads / 16) + threadIdx.x / 16;
    Eight<T> v[kQGroups];
    int64_t at[kQGroups];
    wait_for_inputs();
#pragma unroll
    for (int j = 0; j < kQGroups; ++j) {
        const int64_t u = u0 + j * (kQThreads / 16);
        v[j].clear();
        at[j] = -1;
        if (u < units) {
            const uint32_t row = (uint32_t)u / (uint32_t)p.groups, col = ((uint32_t)u - row * (uint32_t)p.groups) * kGroup + c;
            if (col < (uint32_t)p.C) {
                at[j] = row * p.y8_st + col;
                const int64_t from = row * p.x_st + col;
                if (range_in_bounds(from, 8, p.ex, p.status, nullptr)) v[j].load(static_cast<const T *>(p.x) + from);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kQGroups; ++j) {
        f32x2 f[4];
        v[j].unpack(f);
        const float scale = scale_of(top_of_group(top_of(f)));
        if (at[j] >= 0 && range_in_bounds(at[j], 8, p.ey, p.status, nullptr)) {
            *reinterpret_cast<uint2 *>(p.y8 + at[j]) = e4m3x8(f, __frcp_rn(scale));
            if (lane == 0) p.scale[u0 + j * (kQThreads / 16)] = scale;
        }
    }
}

// Weights: a block takes 128 x 128 values, eight rows a half warp.
template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_blocks_kernel(const QuantizeParams p) {
    constexpr int kRows = kGroup / (kQThreads / 16);
    __shared__ float s_top[kQThreads / 32];
    const int tid = threadIdx.x, lane = tid & 15, part = tid / 16;
    const int block = blockIdx.x / p.groups, group = blockIdx.x % p.groups, c = group * kGroup + lane * 8;
    Eight<T> v[kRows];
    wait_for_inputs();
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int row = block * kGroup + part + j * (kQThreads / 16);
        const int64_t from = row * p.x_st + c;
        v[j].clear();
        if (row < p.n && c < p.C && range_in_bounds(from, 8, p.ex, p.status, nullptr)) v[j].load(static_cast<const T *>(p.x) + from);
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        f32x2 f[4];
        v[j].unpack(f);
        top = top_of(f, top);
    }
    // of what is not below 0 the bits order as integers do, a NaN's above all
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQThreads / 32; w += 2) top = max3_nan(top, s_top[w], s_top[w + 1]);
    const float scale = scale_of(top), inverse = __frcp_rn(scale);
    if (tid == 0) p.scale[blockIdx.x] = scale;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int row = block * kGroup + part + j * (kQThreads / 16);
        f32x2 f[4];
        v[j].unpack(f);
        if (row < p.n && c < p.C && range_in_bounds(row * p.y8_st + c, 8, p.ey, p.status, nullptr))
            *reinterpret_cast<uint2 *>(p.y8 + row * p.y8_st + c) = e4m3x8(f, inverse);
    }
}

cgdr_status check(const cgdr_quantize_args *a) {
    if (!a) return CGDR_ERR_INVALID_ARG;
    if (a->n < 0 || a->C <= 0) return CGDR_ERR_INVALID_ARG;
    if (!dtype_ok(a->dtype) || a->C % 8 != 0 || a->n > kMaxTokens || (a->block_rows != 1 && a->block_rows != kGroup))
        return CGDR_ERR_UNSUPPORTED;
    if ((int64_t)a->n * groups_of(a->C) > INT32_MAX) return CGDR_ERR_UNSUPPORTED;
    if (a->n == 0) return CGDR_OK;
    if (!a->x || !a->y8 || !a->y_scale || a->y8 == a->x || !disjoint(a->n, a->y8_st, 1, 0, a->C)) return CGDR_ERR_INVALID_ARG;
    if (!aligned_to(a->x, 16) || !aligned_to(a->y8, 16) || !aligned_to(a->y_scale, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    return row_stride_ok(a->x_st, esize(a->dtype)) && row_stride_ok(a->y8_st, 1) ? CGDR_OK : CGDR_ERR_ALIGNMENT;
}

template <typename T>
cgdr_status launch_quantize(const QuantizeParams &p, int block_rows, cudaStream_t s) {
    if (block_rows == 1) {
        const int64_t units = (int64_t)p.n * p.groups, per = (kQThreads / 16) * kQGroups;
        return launch_early(quantize_rows_kernel<T>, (unsigned)((units + per - 1) / per), kQThreads, 0, s, 0, p);
    }
    return launch_early(quantize_blocks_kernel<T>, (unsigned)(groups_of(p.n) * (int64_t)p.groups), kQThreads, 0, s, 0, p);
}

}  // namespace
}  // namespace cgdr

extern "C" cgdr_status cgdr_norm(const cgdr_norm_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->n == 0) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int most = INT32_MAX / a->H;                // tokens of a launch: rows are numbered in 32 bits
    const int esz = esize(a->dtype);
    auto from = [&](const void *base, int64_t at) { return const_cast<char *>(static_cast<const char *>(base)) + at; };
    for (int64_t t = 0; t < a->n; t += most) {
        const int n = a->n - t < most ? (int)(a->n - t) : most;
        NormParams p{};
        p.rows = (uint32_t)n * a->H; p.H = a->H; p.C = a->C;
        p.by_head = ~0ull / a->H + 1;
        p.eps = a->eps < 0.f ? 1e-6f : a->eps;
        p.x = from(a->x, t * a->x_st * esz); p.x_st = a->x_st; p.x_sh = a->x_sh; p.ex = extent3(n, a->x_st, a->H, a->x_sh, a->C);
        if (a->residual) p.r = from(a->residual, t * a->residual_st * esz);
        p.r_st = a->residual_st; p.r_sh = a->residual_sh; p.er = extent3(n, a->residual_st, a->H, a->residual_sh, a->C);
        p.weight = a->weight;
        if (a->o) p.o = from(a->o, t * a->o_st * esz);
        p.o_st = a->o_st; p.o_sh = a->o_sh; p.eo = extent3(n, a->o_st, a->H, a->o_sh, a->C);
        if (a->y8) { p.y8 = static_cast<uint8_t *>(a->y8) + t * a->y8_st; p.scale = a->y_scale + t * groups_of(a->C); }
        p.y8_st = a->y8_st; p.ey = extent3(1, 0, n, a->y8_st, a->C);
        p.status = a->status;
        const cgdr_status done = a->dtype == CGDR_BF16 ? launch_vecs<__nv_bfloat16>(p, s) : launch_vecs<float>(p, s);
        if (done != CGDR_OK) return done;
    }
    return CGDR_OK;
}

extern "C" cgdr_status cgdr_quantize(const cgdr_quantize_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->n == 0) return st;
    QuantizeParams p{};
    p.n = a->n; p.C = a->C; p.groups = groups_of(a->C);
    p.x = a->x; p.x_st = a->x_st; p.ex = extent3(1, 0, a->n, a->x_st, a->C);
    p.y8 = static_cast<uint8_t *>(a->y8); p.y8_st = a->y8_st; p.ey = extent3(1, 0, a->n, a->y8_st, a->C);
    p.scale = a->y_scale;
    p.status = a->status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == CGDR_BF16 ? launch_quantize<__nv_bfloat16>(p, a->block_rows, s) : launch_quantize<float>(p, a->block_rows, s);
}
