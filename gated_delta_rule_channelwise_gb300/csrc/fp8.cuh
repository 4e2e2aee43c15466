// What the two kernels of the 8-bit matrix product share: parameters, copies, products, bounded waits.
#pragma once

#include "layer.cuh"
#include "tc05.cuh"

namespace cgdr {

struct MatmulParams {
    CUtensorMap mx, mw;                               // first: 64-byte aligned
    int n, N, K, blocks;                              // blocks of 128 along K
    const float *xs, *ws;
    void *o;
    int64_t o_st, eo;                                 // and its footprint (index-checking build)
    int o_f32;
    int *status;
    uint32_t polls;
    int inject;
};

bool matmul_few(const cgdr_matmul_args &a);           // whether the kernel for few rows takes the call
cgdr_status launch_matmul_few(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s);
cgdr_status launch_matmul_tiles(const cgdr_matmul_args &a, MatmulParams &p, cudaStream_t s);
// A tensor map of [rows, K] bytes with boxes of 128 bytes by `box` rows, swizzled by 128 bytes.
bool encode_rows(CUtensorMap &m, const void *base, int64_t K, int64_t rows, int64_t stride, int box);

// Polls of a wait, before it gives up (args.wait_polls, 0).  The longest wait of a call that goes well is for a few blocks of K, or for the
// other parts of a cluster, which began together: microseconds.
constexpr uint32_t kMatmulPolls = 1u << 18;
constexpr int kBlockK = 128;                          // bytes of a row in a stage: the values of a scale

namespace fp8 {

using namespace tc05;

// What follows is called by a whole warp, and one lane of it, always the same, does it: operands that the code's form shows to be
// the same for the warp are where these instructions take them from.  Behind a branch to one lane two waits, a block's four products
// and two commits take 700 cycles, so 570; 4,001 x 12,288 x 4,096 163 us and 154, 512 x 4,096 x 4,096 15.2 and 11.3.

// D[128 x N] (+)= A[128 x 32] B[N x 32]^T, e4m3 both, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_e4m3(int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p, one;\nelect.sync _|one, 0xffffffff;\nsetp.ne.u32 p, %4, 0;\n"
        "@one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// A block of K: four products of 32.
template <int N>
__device__ __forceinline__ void mma_block(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem) {
    const uint64_t ad = smem_desc(a_smem), bd = smem_desc(b_smem);
#pragma unroll
    for (int k = 0; k < kBlockK / 32; ++k) mma_e4m3(d_tmem, ad + 2 * k, bd + 2 * k, idesc_e4m3(N), k > 0);
}

// Arrives at the barrier when the products so far are done.
__device__ __forceinline__ void commit_warp(uint32_t bar) {
    asm volatile("{\n.reg .pred one;\nelect.sync _|one, 0xffffffff;\n"
                 "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar) : "memory");
}
// Copies two boxes to dst and dst + first, whose bytes the barrier then waits for.
__device__ __forceinline__ void copy_boxes(uint32_t dst, uint32_t first, uint32_t bytes, const CUtensorMap *a, int row_a, const CUtensorMap *b, int row_b, int k, uint32_t bar) {
    asm volatile(
        "{\n.reg .pred one;\nelect.sync _|one, 0xffffffff;\n"
        "@one mbarrier.arrive.expect_tx.shared::cta.b64 _, [%7], %8;\n"
        "@one cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%2, {%6, %3}], [%7];\n"
        "@one cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%1], [%4, {%6, %5}], [%7];\n}\n"
        ::"r"(dst), "r"(dst + first), "l"(reinterpret_cast<uint64_t>(a)), "r"(row_a), "l"(reinterpret_cast<uint64_t>(b)), "r"(row_b), "r"(k), "r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16 columns of this thread's lane: asked for, and (later) there.
__device__ __forceinline__ void ask16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// All loads asked for so far are there; their registers pass through, so that no use of them moves up.
__device__ __forceinline__ void there() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
template <int N> __device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// The slow part of a wait: until the phase is over, another wait has given up, or this one does.  (Inlined: the threads that
// add up have no registers to spare for a call.)
__device__ __forceinline__ bool keep_waiting(uint32_t bar, uint32_t parity, volatile int *stop, int *status, uint32_t polls) {
    for (uint32_t it = 0; it < polls; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*stop) return false;
    }
    *stop = 1;
    if (status != nullptr) atomicExch(status, (int)CGDR_ERR_TIMEOUT);
    return false;
}

// What a block leaves must be over, whichever wait gave up and whichever warp had issued all that it had to: its memory and its tensor
// memory go to the next block.  The copying warp waits for its last uses of every stage, the issuing one for all its products.  Both
// are over before the last sums are taken in any other case, so these waits cost nothing there.
template <int kStages>
__device__ __forceinline__ void copies_land(uint32_t first_bar, uint32_t issued) {
    for (uint32_t u = issued > kStages ? issued - kStages : 0; u < issued; ++u)
        mbar_wait(first_bar + 8 * (u % kStages), (u / kStages) & 1, kMatmulPolls);
}
__device__ __forceinline__ void products_end(uint32_t bar) {
    commit_warp(bar);
    mbar_wait(bar, 0, kMatmulPolls);
}
// Index-checking build, one thread, after every warp has come to its end: CGDR_ERR_BOUNDS if that did not hold.
template <int kStages>
__device__ __forceinline__ void check_over(uint32_t full, uint32_t issued, uint32_t drain, int *status) {
#ifdef CGDR_DEBUG_CHECKS
    bool over = mbar_try_wait(drain, 0);
    for (uint32_t u = issued > kStages ? issued - kStages : 0; u < issued; ++u) over = over && mbar_try_wait(full + 8 * (u % kStages), (u / kStages) & 1);
    in_bounds(over ? 0 : -1, 1, status, nullptr);
#else
    (void)full; (void)issued; (void)drain; (void)status;
#endif
}

}  // namespace fp8
}  // namespace cgdr
