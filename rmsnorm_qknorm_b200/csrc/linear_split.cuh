// Fused linear layer for some hundred rows: K split over the CTA pairs of a cluster.
//
// Included by linear.cu only (one translation unit: its device error word).
//
// Between the two other kernels: with 100 to 500 rows a few dozen 256-row tiles
// leave most pairs of linear_pair.cuh without work, and the narrow tiles of
// linear_rows.cuh bring every operand so often from L2 (128 x 128 per CTA: 64
// KiB for what 256 x 256 on a pair does with 32 KiB per CTA) that its
// throughput bounds them.  Here a cluster of S pairs takes one 256 x 256 (or
// 128) tile, each pair a part of K with the MMAs of linear_pair.cuh.  Every
// CTA leaves its 128 fp32 rows in shared memory (over the ring, 16-byte chunks
// turned by the row so that neither side meets in a bank), and the rows are
// shared out among the CTAs that hold partials of them, which add those in
// rank order over distributed shared memory and run the epilogue, as the
// kernel for few rows does.  No workspace, no atomics: the same bits every time.
// Measured against the better of the other two (gelu): 729 x 1760 x 9432 50 -> 29
// us, 3250 x 176 x 6720 26 -> 16, 1008 x 1048 x 8784 35 -> 23, 384 x 4096 x 12288
// 54 -> 48; dx of 2511 x 11880 x 72 30 -> 20, of 419 x 4096 x 2456 19 -> 15.
//
// Roles (320 threads): warp 0 TMA producer, warp 1 MMA issuer (even CTAs),
// warps 2-9 take the accumulator out of tensor memory; all ten add up and store.
// Every wait is bounded and records a failure in g_linear_error.
#pragma once

namespace lin {
namespace split {

constexpr int BM = pair::BM, BK = pair::BK, THREADS = 320;
constexpr int kMaxPairs = 4;  // of a cluster

template <int BN> struct Shape {
    static constexpr int BN_CTA = BN / 2;
    static constexpr int STAGE_BYTES = pair::A_BYTES + BN_CTA * BK * 2;
    static constexpr int STAGES = (227 * 1024 - 2048) / STAGE_BYTES;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;
    static_assert(BM * BN * 4 <= STAGES * STAGE_BYTES && (2 * STAGES + 2) * 8 <= 256, "shared memory budget");
};

template <bool A_MN, bool B_MN, int BN, int ACT>
__global__ void __launch_bounds__(THREADS, 1)
linear_split_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                    const rows::Args g, const int pm_blocks) {
    using S = Shape<BN>;
    constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES), *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank(), side = rank & 1, even = rank & ~1u;
    const int ranks = (int)cluster_size() / 2, part = (int)rank / 2;  // pairs that share the tile, this one
    const int tile = (int)blockIdx.x / (2 * ranks);
    const int m0 = tile % pm_blocks * 2 * BM + (int)side * BM, n0 = tile / pm_blocks * BN;
    const int kb0 = (int)((int64_t)g.k_blocks * part / ranks), kb1 = (int)((int64_t)g.k_blocks * (part + 1) / ranks);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);   // even CTA: its producer's arrive + both CTAs' bytes
            mbar_init(smem_u32(&empty[s]), 1);  // the even CTA's commit
        }
        mbar_init(smem_u32(acc_full), 1);       // the even CTA's commit
        mbar_init_fence();
    }
    if (warp == 1) {  // whole warp, in both CTAs: the pair's tensor memory
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(BN) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    gemm::tc_fence_before();
    cluster_sync();  // the barriers exist before any remote arrive or copy
    gemm::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the previous kernel on the stream has finished before any global memory is touched
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer (both CTAs)
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        const uint32_t fb0 = map_to_rank(smem_u32(&full[0]), even);  // the even CTA's stage barriers
        int at = kb0 + tile * 5 % (kb1 - kb0);  // tiles start elsewhere in their part of K (see linear_rows.cuh)
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, &g_linear_error)) break;
            if (side == 0) elect_expect_tx(smem_u32(&full[stage]), 2 * STAGE_BYTES);
            const uint32_t fb = fb0 + (uint32_t)stage * 8u, sa = smem_u32(smem + stage * STAGE_BYTES);
            pair::load_operand<A_MN, BM>(sa, &tmap_a, m0, at * BK, fb);
            pair::load_operand<B_MN, S::BN_CTA>(sa + pair::A_BYTES, &tmap_b, n0 + (int)side * S::BN_CTA, at * BK, fb);
            if (++at == kb1) at = kb0;
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        // no copy of either CTA may still be writing when the ring is reused or the CTA exits
        // (immediate on the normal path; the odd CTA learns of it at the cluster's barriers)
        if (side == 0)
            for (int s = 0; s < STAGES; ++s)
                if (armed & (1u << s)) mbar_wait(smem_u32(&full[s]), (armed_parity >> s) & 1u, &g_linear_error);
        __syncwarp();
    } else if (warp == 1 && side == 0) {
        // ---------------------------------------------------------------- MMA issuer (even CTA)
        const uint32_t peer_empty0 = map_to_rank(smem_u32(&empty[0]), rank + 1);
        const uint64_t a0 = pair::operand_desc<A_MN>(smem_u32(smem)), b0 = pair::operand_desc<B_MN>(smem_u32(smem + pair::A_BYTES));
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(smem_u32(&full[stage]), phase, &g_linear_error)) break;
            gemm::tc_fence_after();
            const uint64_t at = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < BK / gemm::UMMA_K; ++k)
                elect_umma<2, pair::instr_desc<A_MN, B_MN, BN>()>(tmem_base, a0 + at + k * pair::k_step<A_MN>(),
                                                                  b0 + at + k * pair::k_step<B_MN>(),
                                                                  (kb != kb0 || k != 0) ? 1u : 0u);
            elect_commit<2>(smem_u32(&empty[stage]));
            elect_commit<2>(peer_empty0 + (uint32_t)stage * 8u);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        elect_commit<2>(smem_u32(acc_full));  // every MMA issued here has completed
        elect_commit<2>(map_to_rank(smem_u32(acc_full), rank + 1));
        __syncwarp();
    }
    // every thread: the accumulator is complete and no MMA reads either CTA's ring any more
    mbar_wait_cluster(smem_u32(acc_full), 0u, &g_linear_error, product_timeout(kb1 - kb0));
    gemm::tc_fence_after();
    __syncwarp();  // tensor memory is read by whole warps
    __syncthreads();
    // this CTA's rows of the partial tile: [128][BN] fp32, chunk c of row i at c ^ (i & 7)
    const uint32_t mine = smem_u32(smem);
    if (warp >= 2) {
        const int quarter = warp & 3, half = (warp - 2) >> 2, row = quarter * 32 + lane;
        const uint32_t at = mine + (uint32_t)row * (BN * 4u);
#pragma unroll 1
        for (int c = 0; c < BN / 2; c += 32) {
            uint32_t v[32];
            gemm::tmem_ld_32cols(tmem_base + ((uint32_t)(quarter * 32) << 16) + half * (BN / 2) + c, v);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                             ::"r"(at + (uint32_t)((((half * (BN / 2) + c) / 4 + q) ^ (row & 7)) * 16)),
                               "r"(v[4 * q]), "r"(v[4 * q + 1]), "r"(v[4 * q + 2]), "r"(v[4 * q + 3]) : "memory");
        }
        gemm::tc_fence_before();
    }
    cluster_sync();
    // Rows part, part + ranks, ... of this side's 128, whose partials lie in the CTAs of the same side
    const int valid = min(BM, g.M - m0);
#pragma unroll 1
    for (int h = 0; h < BN / 128; ++h) {
        const int n = n0 + 128 * h + 4 * lane;
        float bias[4];
        rows::load_bias(g, n, bias);
        auto partial = [&](int i, int s) {
            return map_to_rank(mine + (uint32_t)i * (BN * 4u) + (uint32_t)(((32 * h + lane) ^ (i & 7)) * 16), 2u * (uint32_t)s + side);
        };
        if (ranks <= 2) rows::finish<ACT, 2, 4, THREADS>(g, partial, bias, n, m0, valid, part, ranks);
        else rows::finish<ACT, kMaxPairs, 2, THREADS>(g, partial, bias, n, m0, valid, part, ranks);
    }
    cluster_sync();  // the other CTAs have read this one's rows
    if (warp == 1) {
        gemm::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(BN) : "memory");
    }
}

// ---------------------------------------------------------------- host side

template <bool A_MN, bool B_MN, int BN, int ACT>
qkn_status launch_bn(const pair::Matrix &x, const pair::Matrix &W, const rows::Args &a, int parts, cudaStream_t s) {
    const auto kernel = linear_split_kernel<A_MN, B_MN, BN, ACT>;
    CUtensorMap ta, tb;
    if (qkn_status st = make_tmap_pitched(&ta, x.p, x.rows, x.inner, x.pitch, BK, A_MN ? BK : BM)) return st;
    if (qkn_status st = make_tmap_pitched(&tb, W.p, W.rows, W.inner, W.pitch, BK, B_MN ? BK : BN / 2)) return st;
    static std::atomic<bool> attr_set[64];  // per device: the attribute has been set
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (!known || !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<BN>::SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(linear_split_kernel)");
        if (known) attr_set[dev].store(true, std::memory_order_release);
    }
    const int pm_blocks = (a.M + 2 * BM - 1) / (2 * BM), n_blocks = (a.N + BN - 1) / BN;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = Shape<BN>::SMEM_BYTES;
    cfg.gridDim = dim3((unsigned)(pm_blocks * n_blocks * 2 * parts), 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)(2 * parts);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, a, pm_blocks);
    if (e != cudaSuccess) return cuda_fail(e, "linear_split_kernel launch");
    return check_launch("linear_split_kernel launch");
}

// Clusters of `parts` pairs that the device holds at once (33, 22 and 15 of two, three and four pairs
// on 148 SMs; one more and the kernel takes twice as long).
inline int64_t clusters_of(int parts) {
    static std::atomic<int> held[64][kMaxPairs + 1];  // per device, 0 until asked
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    int n = known ? held[dev][parts].load(std::memory_order_acquire) : 0;
    if (n > 0) return n - 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = Shape<256>::SMEM_BYTES;
    cfg.gridDim = dim3(2u * parts, 1, 1);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2u * parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const auto kernel = linear_split_kernel<false, false, 256, QKN_ACT_NONE>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<256>::SMEM_BYTES) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 0;  // the other kernels serve the call
    }
    if (known) held[dev][parts].store(n + 1, std::memory_order_release);
    return n;
}

// About how long the kernel takes, in ns, with the tile's columns and the pairs of a cluster.
// Measured at 256 rows, K 4096 and 12288: 16 tiles of 256 columns in three parts 17 us, 32 of 128 in
// two 14.7, of 256 in two 21.3.
inline int64_t cost(int64_t M, int64_t N, int64_t K, int bn, int parts) {
    const int64_t kb = (K + BK - 1) / BK;
    const int64_t tiles = ((M + 2 * BM - 1) / (2 * BM)) * ((N + bn - 1) / bn);
    if (kb < 4 * parts || 2 * parts * tiles > sm_count() || tiles > clusters_of(parts)) return INT64_MAX;
    return bn == 256 ? 8800 + (kb + parts - 1) / parts * 370 : 6500 + (kb + parts - 1) / parts * 256;
}

// Columns and pairs for a product, 0 columns where the other kernels, estimated at `others` ns, serve it.
struct Choice { int columns, parts; };
inline Choice choose(int64_t M, int64_t N, int64_t K, int64_t others) {
    Choice best = {0, 0};
    for (int parts = 2; parts <= kMaxPairs; ++parts)
        for (int bn = 128; bn <= 256; bn += 128)
            if (const int64_t c = cost(M, N, K, bn, parts); c < others) {
                others = c;
                best = {bn, parts};
            }
    return best;
}

// y = epilogue of the product of A and B, as pair::launch.
template <bool A_MN, bool B_MN, int ACT>
qkn_status launch(const pair::Matrix &a, const pair::Matrix &b, const pair::Matrix &y, const pair::Matrix *res,
                  const pair::Matrix *z, const Epilogue &epi, int64_t K, Choice c, cudaStream_t s) {
    const rows::Args g = rows::args_of(y, res, z, epi, K);
    return c.columns == 128 ? launch_bn<A_MN, B_MN, 128, ACT>(a, b, g, c.parts, s)
                            : launch_bn<A_MN, B_MN, 256, ACT>(a, b, g, c.parts, s);
}

}  // namespace split
}  // namespace lin
