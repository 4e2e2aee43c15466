// Root-mean-square norm with the residual's addition (cgdr_norm), and the 8-bit quantisers (cgdr_quantize).
#include "layer.cuh"

namespace cgdr {
namespace {

struct NormParams {
    int64_t rows;                                     // n * H
    int H, C, shift;                                  // 2^shift threads to a row
    float eps;
    const void *x;  int64_t x_st, x_sh;
    void *r;        int64_t r_st, r_sh;
    const float *weight;
    void *o;        int64_t o_st, o_sh;
    uint8_t *y8;    int64_t y8_st;
    float *scale;
    int64_t ex, er, eo, ey;                               // footprints (index-checking build)
    int *status;
};

// A row is held by 2^shift threads, kVecs vectors of eight values a thread: one pass over the data.  The 16 lanes
// of a half warp hold 128 consecutive values, so a group's largest magnitude takes four shuffles.
template <typename T, int kVecs, bool kResidual, bool k8>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
    __shared__ float s_sum[32];
    const int tid = threadIdx.x, per = 1 << p.shift, t = tid & (per - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> p.shift) + (tid >> p.shift);
    const bool live = row < p.rows;
    const int64_t i = p.H == 1 ? row : row / p.H, h = p.H == 1 ? 0 : row % p.H;
    const int64_t x0 = i * p.x_st + h * p.x_sh, r0 = i * p.r_st + h * p.r_sh;
    const int nv = p.C / 8;

    Eight<T> xv[kVecs], rv[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int c = (t + (j << p.shift)) * 8;
        xv[j].clear();
        rv[j].clear();
        if (live && c < p.C) {
            if (range_in_bounds(x0 + c, 8, p.ex, p.status, nullptr)) xv[j].load(static_cast<const T *>(p.x) + x0 + c);
            if (kResidual && range_in_bounds(r0 + c, 8, p.er, p.status, nullptr)) rv[j].fetch(static_cast<T *>(p.r) + r0 + c);
        }
    }
    float f[kVecs][8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int c = (t + (j << p.shift)) * 8;
        xv[j].unpack(f[j]);
        if (kResidual) {
            float g[8];
            rv[j].unpack(g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[j][e] += g[e];
            if (live && c < p.C && range_in_bounds(r0 + c, 8, p.er, p.status, nullptr)) Eight<T>::store(static_cast<T *>(p.r) + r0 + c, f[j]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(f[j][e], f[j][e], sum);
    }
    for (int o = min(per, 32) >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (per > 32) {                                   // always in the same order
        if ((tid & 31) == 0) s_sum[tid >> 5] = sum;
        __syncthreads();
        sum = 0.f;
        for (int w = 0; w < per / 32; ++w) sum += s_sum[((tid >> p.shift) << (p.shift - 5)) + w];
    }
    const float by = __frsqrt_rn(sum / (float)p.C + p.eps);

#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
        const int v = t + (j << p.shift), c = v * 8;
        const bool in = live && v < nv;
        float w[8];
        if (p.weight != nullptr && in) {
            Eight<float> raw;
            raw.load(p.weight + c);
            raw.unpack(w);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[j][e] = in ? f[j][e] * by * (p.weight != nullptr ? w[e] : 1.f) : 0.f;
        if (k8) {
            const float scale = scale_of(top_of_group(top_of(f[j])));
            if (in && range_in_bounds(row * p.y8_st + c, 8, p.ey, p.status, nullptr)) {
                *reinterpret_cast<uint2 *>(p.y8 + row * p.y8_st + c) = e4m3x8(f[j], __frcp_rn(scale));
                if (v % 16 == 0) p.scale[row * ((p.C + kGroup - 1) / kGroup) + c / kGroup] = scale;
            }
        } else {
            const int64_t at = i * p.o_st + h * p.o_sh + c;
            if (in && range_in_bounds(at, 8, p.eo, p.status, nullptr)) Eight<T>::store(static_cast<T *>(p.o) + at, f[j]);
        }
    }
}

template <typename T, int kVecs>
cgdr_status launch_norm(const NormParams &p, cudaStream_t s) {
    const int per = 1 << p.shift, threads = per < 256 ? 256 : per, rows = threads / per;
    const int64_t blocks = (p.rows + rows - 1) / rows;
    if (blocks > INT32_MAX) return CGDR_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks);
    if (p.r != nullptr)
        p.y8 != nullptr ? norm_kernel<T, kVecs, true, true><<<grid, threads, 0, s>>>(p) : norm_kernel<T, kVecs, true, false><<<grid, threads, 0, s>>>(p);
    else
        p.y8 != nullptr ? norm_kernel<T, kVecs, false, true><<<grid, threads, 0, s>>>(p) : norm_kernel<T, kVecs, false, false><<<grid, threads, 0, s>>>(p);
    return launched();
}

template <typename T>
cgdr_status launch_vecs(NormParams &p, cudaStream_t s) {
    const int nv = p.C / 8;
    int vecs = 1;
    auto shift_for = [&](int v) {
        int sh = 4;
        while ((v << sh) < nv) ++sh;
        return sh;
    };
    while (vecs < 4 && shift_for(vecs) > 7) vecs *= 2;
    p.shift = shift_for(vecs);
    return vecs == 1 ? launch_norm<T, 1>(p, s) : vecs == 2 ? launch_norm<T, 2>(p, s) : launch_norm<T, 4>(p, s);
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
    if ((a->residual && !disjoint(a->n, a->r_st, a->H, a->r_sh, a->C)) || (a->o && !disjoint(a->n, a->o_st, a->H, a->o_sh, a->C)))
        return CGDR_ERR_INVALID_ARG;
    const int esz = esize(a->dtype);
    if (!aligned_to(a->x, 16) || !aligned_to(a->residual, 16) || !aligned_to(a->weight, 16) || !aligned_to(a->o, 16) ||
        !aligned_to(a->y8, 16) || !aligned_to(a->y_scale, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    if (!row_stride_ok(a->x_st, esz) || !row_stride_ok(a->x_sh, esz)) return CGDR_ERR_ALIGNMENT;
    if (a->residual && (!row_stride_ok(a->r_st, esz) || !row_stride_ok(a->r_sh, esz))) return CGDR_ERR_ALIGNMENT;
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
constexpr int kQGroups = 4;                           // groups of a half warp

// Rows: a half warp takes a group of 128 values, several at a time.
template <typename T>
__global__ void __launch_bounds__(kQThreads) quantize_rows_kernel(const QuantizeParams p) {
    const int lane = threadIdx.x & 15, c = lane * 8;
    const int64_t units = (int64_t)p.n * p.groups, u0 = ((int64_t)blockIdx.x * kQGroups) * (kQThreads / 16) + threadIdx.x / 16;
    Eight<T> v[kQGroups];
    int64_t at[kQGroups];
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
        float f[8];
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
    __shared__ uint32_t s_top[kQThreads / 32];
    const int tid = threadIdx.x, lane = tid & 15, part = tid / 16;
    const int block = blockIdx.x / p.groups, group = blockIdx.x % p.groups, c = group * kGroup + lane * 8;
    Eight<T> v[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int row = block * kGroup + part + j * (kQThreads / 16);
        const int64_t from = row * p.x_st + c;
        v[j].clear();
        if (row < p.n && c < p.C && range_in_bounds(from, 8, p.ex, p.status, nullptr)) v[j].load(static_cast<const T *>(p.x) + from);
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        float f[8];
        v[j].unpack(f);
        top = max(top, top_of(f));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQThreads / 32; ++w) top = max(top, s_top[w]);
    const float scale = scale_of(top), inverse = __frcp_rn(scale);
    if (tid == 0) p.scale[blockIdx.x] = scale;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const int row = block * kGroup + part + j * (kQThreads / 16);
        float f[8];
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
    if (!a->x || !a->y8 || !a->y_scale || !disjoint(a->n, a->y8_st, 1, 0, a->C)) return CGDR_ERR_INVALID_ARG;
    if (!aligned_to(a->x, 16) || !aligned_to(a->y8, 16) || !aligned_to(a->y_scale, 4) || !aligned_to(a->status, 4))
        return CGDR_ERR_ALIGNMENT;
    return row_stride_ok(a->x_st, esize(a->dtype)) && row_stride_ok(a->y8_st, 1) ? CGDR_OK : CGDR_ERR_ALIGNMENT;
}

template <typename T>
cgdr_status launch_quantize(const QuantizeParams &p, int block_rows, cudaStream_t s) {
    if (block_rows == 1) {
        const int64_t units = (int64_t)p.n * p.groups, per = (kQThreads / 16) * kQGroups;
        quantize_rows_kernel<T><<<(unsigned)((units + per - 1) / per), kQThreads, 0, s>>>(p);
    } else {
        quantize_blocks_kernel<T><<<(unsigned)(groups_of(p.n) * (int64_t)p.groups), kQThreads, 0, s>>>(p);
    }
    return launched();
}

}  // namespace
}  // namespace cgdr

extern "C" cgdr_status cgdr_norm(const cgdr_norm_args *a, void *stream) {
    using namespace cgdr;
    const cgdr_status st = check(a);
    if (st != CGDR_OK || a->n == 0) return st;
    NormParams p{};
    p.rows = (int64_t)a->n * a->H; p.H = a->H; p.C = a->C;
    p.eps = a->eps < 0.f ? 1e-6f : a->eps;
    p.x = a->x; p.x_st = a->x_st; p.x_sh = a->x_sh;
    p.r = a->residual; p.r_st = a->r_st; p.r_sh = a->r_sh;
    p.weight = a->weight;
    p.o = a->o; p.o_st = a->o_st; p.o_sh = a->o_sh;
    p.y8 = static_cast<uint8_t *>(a->y8); p.y8_st = a->y8_st; p.scale = a->y_scale;
    p.ey = extent3(1, 0, a->n, a->y8_st, a->C);
    p.ex = extent3(a->n, a->x_st, a->H, a->x_sh, a->C);
    p.er = extent3(a->n, a->r_st, a->H, a->r_sh, a->C);
    p.eo = extent3(a->n, a->o_st, a->H, a->o_sh, a->C);
    p.status = a->status;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a->dtype == CGDR_BF16 ? launch_vecs<__nv_bfloat16>(p, s) : launch_vecs<float>(p, s);
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
