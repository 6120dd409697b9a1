// Matrix product of the fused linear layer and its gradients on CTA pairs.
//
// Included by linear.cu only (one translation unit: its device error word).
//
//   C[m][n] = sum_k A(m, k) B(n, k),  256 x 256 tiles of C, bf16 in, fp32
// accumulated in tensor memory by tcgen05.mma.cta_group::2.  An operand is
// K-major (rows of consecutive k: x and W of the forward product) or MN-major
// (consecutive m or n: W in dx = dz W, dz and x in dW = dz^T x), read where it
// lies: no operand is transposed in memory.  A stage holds 64 k of 128 rows
// of each operand per CTA, as 128-byte-swizzled rows of 64 k, or as two
// blocks of 64 (k) rows of 64 m.
//
// Roles per CTA (192 threads) as in the FlashNorm projection: warp 0 moves
// tiles with TMA, one lane of the even CTA's warp 1 issues the MMAs, warps
// 2-5 run the epilogue of a tile while the MMAs of the next one run into the
// other accumulator.  The epilogue works on 32 x 32 blocks: accumulator
// -> times the row's scale, plus bias -> z (stored where asked) -> activation
// -> plus residual -> y.  A residual block is brought by TMA into the buffer
// that y leaves from, one block ahead, and each thread overwrites the bytes
// it read.
// Every wait is bounded and records a failure in g_linear_error.
#pragma once

namespace lin {
namespace pair {

constexpr int BM = 128, BN = 256, BN_CTA = 128, BK = 64;
constexpr int STAGES = 6;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN_CTA * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int PAIR_STAGE_BYTES = 2 * STAGE_BYTES;
constexpr int ACC_COLS = BN, TMEM_COLS = 2 * ACC_COLS;
constexpr int THREADS = 192;
constexpr int BLOCK_BYTES = 2048;                  // a 32 x 32 bf16 block
constexpr int EPI_BYTES = 4 * 4 * BLOCK_BYTES;     // per epilogue warp: two blocks of y (residual first), two of z
constexpr int BAR_BYTES = 256;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + BAR_BYTES + 1024;
constexpr int GROUP_M = 16;  // pair row blocks walked together down each column block (operands shared in L2)
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

struct Args {
    Epilogue epi;
    int M, N;              // of C
    int pm_blocks, n_blocks, k_blocks, num_tiles;
};

__device__ __forceinline__ void tile_coords(int tile, const Args &g, int &pm, int &n) {
    const int group_tiles = GROUP_M * g.n_blocks;
    const int group = tile / group_tiles;
    const int first = group * GROUP_M;
    const int rows_in_group = min(g.pm_blocks - first, GROUP_M);
    const int in_group = tile - group * group_tiles;
    pm = first + in_group % rows_in_group;
    n = in_group / rows_in_group;
}

// Instruction descriptor: bf16 A and B, fp32 D, M = 256 (the pair), N = 256;
// bits 15 and 16 mark MN-major operands.
template <bool A_MN, bool B_MN> constexpr uint32_t instr_desc() {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) |
           ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(2 * BM >> 4) << 24);
}

// Shared-memory descriptor of an operand's 128 rows x 64 k, 128-byte swizzle.
// K-major: as in gemm_tc.cuh.  MN-major: blocks of 64 m x 64 k, 128-byte rows
// of one k each; 8 k are 1024 bytes apart (stride byte offset), the next 64 m
// 8192 bytes (leading byte offset).
template <bool MN> __device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    if constexpr (!MN) return gemm::sw128_kmajor_desc(saddr);
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// 16 k further: 32 bytes along a K-major row, two groups of 8 k MN-major.
template <bool MN> constexpr uint64_t k_step() { return MN ? 2048u >> 4 : 32u >> 4; }

template <uint32_t IDESC>
__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(IDESC), "r"(accumulate));
}

// One operand's 128 rows x 64 k into a stage of this CTA.
template <bool MN>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int row, int k, uint32_t bar) {
    if constexpr (MN) {
        qkn::pair::tma_load_2d_pair(dst, map, row, k, bar);
        qkn::pair::tma_load_2d_pair(dst + 8192u, map, row + 64, k, bar);
    } else {
        qkn::pair::tma_load_2d_pair(dst, map, k, row, bar);
    }
}

template <bool A_MN, bool B_MN, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                   const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_res,
                   const __grid_constant__ CUtensorMap tmap_z, const Args g) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES + EPI_BYTES);
    uint64_t *full = bars, *empty = bars + STAGES;
    uint64_t *acc_full = bars + 2 * STAGES, *acc_empty = bars + 2 * STAGES + 2;
    uint64_t *drained = bars + 2 * STAGES + 4;
    uint64_t *res_full = bars + 2 * STAGES + 5;  // [4 warps][2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 13);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = rank == 0;
    const int pair_id = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);   // even CTA: its producer's arrive + both CTAs' bytes
            mbar_init(smem_u32(&empty[s]), 1);  // the even CTA's commit
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&acc_full[a]), 1);   // the even CTA's commit
            mbar_init(smem_u32(&acc_empty[a]), 8);  // even CTA: four epilogue warps of each CTA
        }
        mbar_init(smem_u32(drained), 1);
        for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&res_full[i]), 1);
        mbar_init_fence();
    }
    if (warp == 1) {  // whole warp, in both CTAs: the pair's tensor memory
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    gemm::tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before any remote arrive or copy
    gemm::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer (both CTAs)
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            uint32_t armed = 0, armed_parity = 0;  // per stage: loads issued; parity of the phase they complete
            bool ok = true;
            const uint32_t fb0 = map_to_rank(smem_u32(&full[0]), 0);  // the even CTA's stage barriers
            for (int tile = pair_id; ok && tile < g.num_tiles; tile += num_pairs) {
                int pm, n;
                tile_coords(tile, g, pm, n);
                for (int kb = 0; kb < g.k_blocks; ++kb) {
                    if (!mbar_wait_fast(smem_u32(&empty[stage]), phase ^ 1u, &g_linear_error)) { ok = false; break; }
                    if (leader) mbar_arrive_expect_tx(smem_u32(&full[stage]), PAIR_STAGE_BYTES);
                    const uint32_t fb = fb0 + (uint32_t)stage * 8u;
                    const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                    load_operand<A_MN>(sa, &tmap_a, pm * 2 * BM + (int)rank * BM, kb * BK, fb);
                    load_operand<B_MN>(sa + A_BYTES, &tmap_b, n * BN + (int)rank * BN_CTA, kb * BK, fb);
                    armed |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            // no copy of either CTA is in flight when the pair exits (the odd CTA stays until the
            // cluster barrier below; immediate on the normal path)
            if (leader)
                for (int s2 = 0; s2 < STAGES; ++s2)
                    if (armed & (1u << s2))
                        mbar_wait(smem_u32(&full[s2]), (armed_parity >> s2) & 1u, &g_linear_error);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer (even CTA)
        if (leader && lane == 0) {
            const uint32_t peer_empty0 = map_to_rank(smem_u32(&empty[0]), 1);
            const uint32_t peer_acc_full0 = map_to_rank(smem_u32(&acc_full[0]), 1);
            const uint64_t a_desc0 = operand_desc<A_MN>(smem_u32(smem));
            const uint64_t b_desc0 = operand_desc<B_MN>(smem_u32(smem + A_BYTES));
            int stage = 0;
            uint32_t phase = 0;
            int it = 0;
            bool ok = true;
            for (int tile = pair_id; ok && tile < g.num_tiles; tile += num_pairs, ++it) {
                const int acc = it & 1;
                const uint32_t acc_phase = (it >> 1) & 1;
                if (!mbar_wait_cluster(smem_u32(&acc_empty[acc]), acc_phase ^ 1u, &g_linear_error)) break;
                gemm::tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
                for (int kb = 0; kb < g.k_blocks; ++kb) {
                    if (!mbar_wait_fast(smem_u32(&full[stage]), phase, &g_linear_error)) { ok = false; break; }
                    gemm::tc_fence_after();
                    const uint64_t at = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
                    for (int k = 0; k < BK / gemm::UMMA_K; ++k)
                        umma<instr_desc<A_MN, B_MN>()>(d_tmem, a_desc0 + at + k * k_step<A_MN>(),
                                                       b_desc0 + at + k * k_step<B_MN>(), (kb | k) != 0 ? 1u : 0u);
                    // the stage is free in both CTAs once these MMAs have read it
                    qkn::pair::umma_commit_pair(smem_u32(&empty[stage]));
                    qkn::pair::umma_commit_pair(peer_empty0 + (uint32_t)stage * 8u);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                qkn::pair::umma_commit_pair(smem_u32(&acc_full[acc]));
                qkn::pair::umma_commit_pair(peer_acc_full0 + (uint32_t)acc * 8u);
            }
            // tensor memory is released only after every MMA issued here has completed
            qkn::pair::umma_commit_pair(smem_u32(drained));
            mbar_wait(smem_u32(drained), 0u, &g_linear_error);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- epilogue (warps 2..5, both CTAs)
        const int quarter = warp & 3;  // TMEM lanes this warp may access: 32 * quarter ...
        const uint32_t ybuf = smem_u32(smem + STAGES * STAGE_BYTES) + (uint32_t)quarter * 4u * BLOCK_BYTES;
        const uint32_t zbuf = ybuf + 2u * BLOCK_BYTES;
        const uint32_t rbar = smem_u32(&res_full[2 * quarter]);
        const uint32_t acc_empty_leader0 = map_to_rank(smem_u32(&acc_empty[0]), 0);
        const bool has_res = g.epi.has_res != 0, has_z = g.epi.has_z != 0;
        uint32_t blk = 0, res_issued = 0, res_taken = 0;  // blocks so far; residual blocks asked for, arrived
        bool ok = true;
        int it = 0;
        // lane 0: the residual block at (col, row) into the y buffer of the res_issued-th block,
        // once the stores issued so far have read their buffers
        auto fetch = [&](int col, int row) {
            bulk_wait_read0();
            const uint32_t bar = rbar + (res_issued & 1u) * 8u;
            mbar_arrive_expect_tx(bar, BLOCK_BYTES);
            tma_load_2d(ybuf + (res_issued & 1u) * BLOCK_BYTES, &tmap_res, col, row, bar);
        };
        for (int tile = pair_id; ok && tile < g.num_tiles; tile += num_pairs, ++it) {
            int pm, n;
            tile_coords(tile, g, pm, n);
            const int acc = it & 1;
            const uint32_t acc_phase = (it >> 1) & 1;
            const int row0 = pm * 2 * BM + (int)rank * BM + quarter * 32;
            const int row = row0 + lane;
            // 32-column blocks of this warp inside C
            const int blocks = row0 < g.M ? min(BN / 32, (g.N - n * BN + 31) / 32) : 0;
            if (has_res && blocks > 0) {
                if (lane == 0) fetch(n * BN, row0);
                ++res_issued;
            }
            if (!mbar_wait(smem_u32(&acc_full[acc]), acc_phase, &g_linear_error)) break;
            gemm::tc_fence_after();
            const float r = g.epi.inv_rms != nullptr && row < g.M ? __ldg(g.epi.inv_rms + row) : 1.f;
            const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * ACC_COLS;
#pragma unroll 1
            for (int c = 0; c < blocks; ++c, ++blk) {
                const int col0 = n * BN + c * 32;
                const uint32_t yb = ybuf + (blk & 1u) * BLOCK_BYTES, zb = zbuf + (blk & 1u) * BLOCK_BYTES;
                if (has_res) {
                    if (c + 1 < blocks) {
                        if (lane == 0) fetch(col0 + 32, row0);
                        ++res_issued;
                    }
                    ok = mbar_wait_fast(rbar + (blk & 1u) * 8u, (blk >> 1) & 1u, &g_linear_error);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    ++res_taken;
                } else if (lane == 0 && blk >= 2) {
                    bulk_wait_read1();  // the stores that used these buffers have read them
                }
                __syncwarp();
                uint32_t v[32];
                gemm::tmem_ld_32cols(tbase + c * 32, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t at = (uint32_t)lane * 64u + (uint32_t)((j ^ ((lane >> 1) & 3)) * 16);
                    float b[8], f[8];
                    if (col0 + 8 * j < g.N) load_bias8(g.epi, col0 + 8 * j, b);
                    else
#pragma unroll
                        for (int e = 0; e < 8; ++e) b[e] = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = fmaf(__uint_as_float(v[8 * j + e]), r, b[e]);
                    if (has_z) {
                        const uint4 o = Chunk<__nv_bfloat16>::pack(f);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                     ::"r"(zb + at), "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w) : "memory");
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = activate<ACT>(f[e]);
                    if (has_res) {
                        uint4 q;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(yb + at) : "memory");
                        float s[8];
                        Chunk<__nv_bfloat16>::unpack(q, s);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] += s[e];
                    }
                    const uint4 o = Chunk<__nv_bfloat16>::pack(f);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 ::"r"(yb + at), "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w) : "memory");
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (has_z) tma_store_2d(&tmap_z, zb, col0, row0);
                    tma_store_2d(&tmap_y, yb, col0, row0);
                    bulk_commit();
                }
            }
            gemm::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_leader0 + (uint32_t)acc * 8u);
        }
        // no copy into or out of the staging blocks is in flight at the exit
        if (lane == 0) {
            for (; res_taken < res_issued; ++res_taken)
                mbar_wait(rbar + (res_taken & 1u) * 8u, (res_taken >> 1) & 1u, &g_linear_error);
            bulk_wait_all();
        }
        __syncwarp();
    }

    gemm::tc_fence_before();
    __syncthreads();
    cluster_sync();  // the even CTA's MMAs and copies, which use both CTAs' memory, are done
    if (warp == 1) {
        gemm::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

// ---------------------------------------------------------------- host side

// An operand or result in memory: `rows` rows of `inner` consecutive bf16, `pitch` elements apart.
struct Matrix {
    const void *p;
    int64_t rows, inner, pitch;
};

template <bool A_MN, bool B_MN, int ACT>
qkn_status launch(const Matrix &a, const Matrix &b, const Matrix &y, const Matrix *res, const Matrix *z,
                  const Epilogue &epi, int64_t K, cudaStream_t s) {
    const auto kernel = linear_pair_kernel<A_MN, B_MN, ACT>;
    CUtensorMap ta, tb, ty, tr, tz;
    if (qkn_status st = make_tmap_pitched(&ta, a.p, a.rows, a.inner, a.pitch, BK, A_MN ? BK : BM, 128)) return st;
    if (qkn_status st = make_tmap_pitched(&tb, b.p, b.rows, b.inner, b.pitch, BK, B_MN ? BK : BN_CTA, 128)) return st;
    if (qkn_status st = make_tmap_pitched(&ty, y.p, y.rows, y.inner, y.pitch, 32, 32, 64)) return st;
    tr = tz = ty;
    if (res != nullptr)
        if (qkn_status st = make_tmap_pitched(&tr, res->p, res->rows, res->inner, res->pitch, 32, 32, 64)) return st;
    if (z != nullptr)
        if (qkn_status st = make_tmap_pitched(&tz, z->p, z->rows, z->inner, z->pitch, 32, 32, 64)) return st;
    Args g;
    g.epi = epi;
    g.epi.has_res = res != nullptr;
    g.epi.has_z = z != nullptr;
    g.M = (int)y.rows;
    g.N = (int)y.inner;
    g.pm_blocks = (int)((y.rows + 2 * BM - 1) / (2 * BM));
    g.n_blocks = (int)((y.inner + BN - 1) / BN);
    g.k_blocks = (int)((K + BK - 1) / BK);
    if ((int64_t)g.pm_blocks * g.n_blocks > 0x7fffffffLL) return fail(QKN_ERR_SHAPE, "linear_pair_kernel: too many tiles");
    g.num_tiles = g.pm_blocks * g.n_blocks;
    static std::atomic<int> max_pairs[64];  // per device: resident clusters of two (0 until measured)
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    int pairs = known ? max_pairs[dev].load(std::memory_order_acquire) : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    if (pairs == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(linear_pair_kernel)");
        cfg.gridDim = dim3(2 * (unsigned)(sm_count() / 2), 1, 1);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess || n <= 0) return cuda_fail(e, "cudaOccupancyMaxActiveClusters(linear_pair_kernel)");
        pairs = n;
        if (known) max_pairs[dev].store(n, std::memory_order_release);
    }
    cfg.gridDim = dim3(2 * (unsigned)(g.num_tiles < pairs ? g.num_tiles : pairs), 1, 1);
    cfg.stream = s;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, ty, tr, tz, g);
    if (e != cudaSuccess) return cuda_fail(e, "linear_pair_kernel launch");
    return check_launch("linear_pair_kernel launch");
}

}  // namespace pair
}  // namespace lin
