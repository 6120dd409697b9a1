// Matrix product of the fused linear layer and its gradients on CTA pairs.
//
// Included by linear.cu only (one translation unit: its device error word).
//
//   C[m][n] = sum_k A(m, k) B(n, k),  256 x 256 (or 128) tiles of C, bf16 in, fp32
// accumulated in tensor memory by tcgen05.mma.cta_group::2.  An operand is
// K-major (rows of consecutive k: x and W of the forward product) or MN-major
// (consecutive m or n: W in dx = dz W, dz and x in dW = dz^T x), read where it
// lies: no operand is transposed in memory.  A stage holds 64 k of 128 rows
// of each operand per CTA, as 128-byte-swizzled rows of 64 k, or as two
// blocks of 64 (k) rows of 64 m.
//
// Roles per CTA (320 threads): warp 0 moves tiles with TMA, one lane of the
// even CTA's warp 1 issues the MMAs, warps 2-9 run the epilogue of a tile
// while the MMAs of the next one run into the other accumulator: a quarter of
// the rows and half of the columns per warp, a row per thread, 32 columns at
// a time: accumulator -> times the row's scale, plus bias -> z (stored where
// asked) -> activation -> plus residual -> y.  Residual, z and y are read and
// written where they lie, whole 32-byte sectors per thread (16 bytes where
// the rows are not 32-byte aligned); the residual is asked for before the
// accumulator is waited for.  (Staged through shared memory and TMA by four
// warps, a block was a chain of waits: 27 us for a call of one tile.)
// Every wait is bounded and records a failure in g_linear_error.
#pragma once

namespace lin {
namespace pair {

constexpr int BM = 128, BK = 64;                   // rows per CTA (256 per pair), k per stage
constexpr int A_BYTES = BM * BK * 2;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int BAR_BYTES = 256;

// The tile's columns: 256, or 128 where the wider tiles leave pairs without work.
template <int BN> struct Shape {
    static constexpr int BN_CTA = BN / 2;          // rows of B that each CTA loads
    static constexpr int B_BYTES = BN_CTA * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = (226 * 1024 - BAR_BYTES - 1024) / STAGE_BYTES;
    static constexpr int PAIR_STAGE_BYTES = 2 * STAGE_BYTES;
    static constexpr int TMEM_COLS = 2 * BN;       // two accumulators
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + BAR_BYTES + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024 && (2 * STAGES + 6) * 8 <= BAR_BYTES, "shared memory budget");
};
constexpr int GROUP_M = 16;  // pair row blocks walked together down each column block (operands shared in L2)

struct Args {
    Epilogue epi;
    const __nv_bfloat16 *res;
    __nv_bfloat16 *y, *z;
    int64_t ldr, ldy, ldz;
    int wide;              // residual, z and y rows are 32-byte aligned
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

// Instruction descriptor: bf16 A and B, fp32 D, M = 256 (the pair), N = BN;
// bits 15 and 16 mark MN-major operands.
template <bool A_MN, bool B_MN, int BN> constexpr uint32_t instr_desc() {
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

// ROWS rows x 64 k of an operand into a stage of this CTA.
template <bool MN, int ROWS>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int row, int k, uint32_t bar) {
    if constexpr (MN) {
#pragma unroll
        for (int h = 0; h < ROWS / 64; ++h) elect_tma_load_pair(dst + h * 8192u, map, row + 64 * h, k, bar);
    } else {
        elect_tma_load_pair(dst, map, k, row, bar);
    }
}

// 16 bf16 of a row, as far as they lie inside it: 32 bytes at once where the rows allow.
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, bool wide, int left, uint32_t (&w)[8]) {
    if (wide && left >= 16) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p) : "memory");
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (left > 8 * h) v = *reinterpret_cast<const uint4 *>(p + 8 * h);
        w[4 * h] = v.x;
        w[4 * h + 1] = v.y;
        w[4 * h + 2] = v.z;
        w[4 * h + 3] = v.w;
    }
}

__device__ __forceinline__ void store16(__nv_bfloat16 *p, bool wide, int left, const float (&f)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    if (wide && left >= 16) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (left > 8 * h) *reinterpret_cast<uint4 *>(p + 8 * h) = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
}

template <bool A_MN, bool B_MN, int BN, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                   const Args g) {
    using S = Shape<BN>;
    constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, BN_CTA = S::BN_CTA;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES);
    uint64_t *full = bars, *empty = bars + STAGES;
    uint64_t *acc_full = bars + 2 * STAGES, *acc_empty = bars + 2 * STAGES + 2;
    uint64_t *drained = bars + 2 * STAGES + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * STAGES + 5);

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
            mbar_init(smem_u32(&acc_empty[a]), 2 * EPI_WARPS);  // even CTA: the epilogue warps of both
        }
        mbar_init(smem_u32(drained), 1);
        mbar_init_fence();
    }
    if (warp == 1) {  // whole warp, in both CTAs: the pair's tensor memory
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(S::TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    gemm::tc_fence_before();
    cluster_sync();  // both CTAs' barriers exist before any remote arrive or copy
    gemm::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the previous kernel on the stream has finished before any global memory is touched
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer (both CTAs)
        int stage = 0;
        uint32_t phase = 0;
        uint32_t armed = 0, armed_parity = 0;  // per stage: loads issued; parity of the phase they complete
        bool ok = true;
        const uint32_t fb0 = map_to_rank(smem_u32(&full[0]), 0);  // the even CTA's stage barriers
        for (int tile = pair_id; ok && tile < g.num_tiles; tile += num_pairs) {
            int pm, n;
            tile_coords(tile, g, pm, n);
            const int row = pm * 2 * BM + (int)rank * BM, col = n * BN + (int)rank * BN_CTA;
            for (int kb = 0; kb < g.k_blocks; ++kb) {
                if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, &g_linear_error)) { ok = false; break; }
                if (leader) elect_expect_tx(smem_u32(&full[stage]), S::PAIR_STAGE_BYTES);
                const uint32_t fb = fb0 + (uint32_t)stage * 8u;
                const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                load_operand<A_MN, BM>(sa, &tmap_a, row, kb * BK, fb);
                load_operand<B_MN, BN_CTA>(sa + A_BYTES, &tmap_b, col, kb * BK, fb);
                armed |= 1u << stage;
                armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        // no copy of either CTA is in flight when the pair exits (the odd CTA stays until the
        // cluster barrier below; immediate on the normal path)
        if (leader)
            for (int s2 = 0; s2 < STAGES; ++s2)
                if (armed & (1u << s2)) mbar_wait(smem_u32(&full[s2]), (armed_parity >> s2) & 1u, &g_linear_error);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer (even CTA)
        if (leader) {
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
                if (!__all_sync(0xffffffffu, mbar_wait_cluster(smem_u32(&acc_empty[acc]), acc_phase ^ 1u, &g_linear_error))) break;
                gemm::tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * BN;
                for (int kb = 0; kb < g.k_blocks; ++kb) {
                    if (!warp_wait(smem_u32(&full[stage]), phase, &g_linear_error)) { ok = false; break; }
                    gemm::tc_fence_after();
                    const uint64_t at = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
                    for (int k = 0; k < BK / gemm::UMMA_K; ++k)
                        elect_umma<2, instr_desc<A_MN, B_MN, BN>()>(d_tmem, a_desc0 + at + k * k_step<A_MN>(),
                                                                    b_desc0 + at + k * k_step<B_MN>(), (kb | k) != 0 ? 1u : 0u);
                    // the stage is free in both CTAs once these MMAs have read it
                    elect_commit<2>(smem_u32(&empty[stage]));
                    elect_commit<2>(peer_empty0 + (uint32_t)stage * 8u);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                elect_commit<2>(smem_u32(&acc_full[acc]));
                elect_commit<2>(peer_acc_full0 + (uint32_t)acc * 8u);
            }
            // tensor memory is released only after every MMA issued here has completed
            elect_commit<2>(smem_u32(drained));
            mbar_wait(smem_u32(drained), 0u, &g_linear_error);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- epilogue (warps 2..9, both CTAs)
        const int quarter = warp & 3;       // TMEM lanes this warp may access: 32 * quarter ...
        const int half = (warp - 2) >> 2;   // its half of the columns
        const uint32_t acc_empty_leader0 = map_to_rank(smem_u32(&acc_empty[0]), 0);
        const bool wide = g.wide != 0;
        int it = 0;
        for (int tile = pair_id; tile < g.num_tiles; tile += num_pairs, ++it) {
            int pm, n;
            tile_coords(tile, g, pm, n);
            const int acc = it & 1;
            const uint32_t acc_phase = (it >> 1) & 1;
            const int row = pm * 2 * BM + (int)rank * BM + quarter * 32 + lane;
            const int col0 = n * BN + half * (BN / 2);
            const bool in = row < g.M;
            const __nv_bfloat16 *res = g.res != nullptr && in ? g.res + row * g.ldr : nullptr;
            __nv_bfloat16 *y = g.y + row * g.ldy, *z = g.z != nullptr && in ? g.z + row * g.ldz : nullptr;
            uint32_t q[2][8];
            if (res != nullptr)
#pragma unroll
                for (int h = 0; h < 2; ++h) load16(res + col0 + 16 * h, wide, g.N - col0 - 16 * h, q[h]);
            const float r = g.epi.inv_rms != nullptr && in ? __ldg(g.epi.inv_rms + row) : 1.f;
            if (!mbar_wait(smem_u32(&acc_full[acc]), acc_phase, &g_linear_error)) break;
            gemm::tc_fence_after();
            const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN + half * (BN / 2);
#pragma unroll 1
            for (int c = 0; c < BN / 64; ++c) {
                const int col = col0 + c * 32;
                uint32_t v[32];
                gemm::tmem_ld_32cols(tbase + c * 32, v);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int at = col + 16 * h, left = g.N - at;
                    float f[16];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float b[8];
                        if (left > 8 * k) load_bias8(g.epi, at + 8 * k, b);
                        else
#pragma unroll
                            for (int e = 0; e < 8; ++e) b[e] = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[8 * k + e] = fmaf(__uint_as_float(v[16 * h + 8 * k + e]), r, b[e]);
                    }
                    if (z != nullptr) store16(z + at, wide, left, f);
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = activate<ACT>(f[e]);
                    if (res != nullptr) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            f[2 * e] += bf16lo(q[h][e]);
                            f[2 * e + 1] += bf16hi(q[h][e]);
                        }
                        // the next block's residual (the bytes of y written here are not among them)
                        if (c + 1 < BN / 64) load16(res + at + 32, wide, left - 32, q[h]);
                    }
                    if (in) store16(y + at, wide, left, f);
                }
            }
            gemm::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_leader0 + (uint32_t)acc * 8u);
        }
    }

    gemm::tc_fence_before();
    __syncthreads();
    cluster_sync();  // the even CTA's MMAs and copies, which use both CTAs' memory, are done
    if (warp == 1) {
        gemm::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(S::TMEM_COLS)
                     : "memory");
    }
}

// ---------------------------------------------------------------- host side

// An operand or result in memory: `rows` rows of `inner` consecutive bf16, `pitch` elements apart.
struct Matrix {
    const void *p;
    int64_t rows, inner, pitch;
};

template <bool A_MN, bool B_MN, int BN, int ACT>
qkn_status launch_bn(const Matrix &a, const Matrix &b, Args &g, int64_t K, cudaStream_t s) {
    using S = Shape<BN>;
    const auto kernel = linear_pair_kernel<A_MN, B_MN, BN, ACT>;
    CUtensorMap ta, tb;
    if (qkn_status st = make_tmap_pitched(&ta, a.p, a.rows, a.inner, a.pitch, BK, A_MN ? BK : BM, 128)) return st;
    if (qkn_status st = make_tmap_pitched(&tb, b.p, b.rows, b.inner, b.pitch, BK, B_MN ? BK : S::BN_CTA, 128)) return st;
    g.pm_blocks = (int)(((int64_t)g.M + 2 * BM - 1) / (2 * BM));
    g.n_blocks = (int)(((int64_t)g.N + BN - 1) / BN);
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
    cfg.dynamicSmemBytes = S::SMEM_BYTES;
    if (pairs == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM_BYTES);
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
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, g);
    if (e != cudaSuccess) return cuda_fail(e, "linear_pair_kernel launch");
    return check_launch("linear_pair_kernel launch");
}

template <bool A_MN, bool B_MN, int ACT>
qkn_status launch(const Matrix &a, const Matrix &b, const Matrix &y, const Matrix *res, const Matrix *z,
                  const Epilogue &epi, int64_t K, cudaStream_t s) {
    Args g;
    g.epi = epi;
    g.y = static_cast<__nv_bfloat16 *>(const_cast<void *>(y.p));
    g.ldy = y.pitch;
    g.res = res ? static_cast<const __nv_bfloat16 *>(res->p) : nullptr;
    g.ldr = res ? res->pitch : 0;
    g.z = z ? static_cast<__nv_bfloat16 *>(const_cast<void *>(z->p)) : nullptr;
    g.ldz = z ? z->pitch : 0;
    g.wide = aligned(g.y, 32) && g.ldy % 16 == 0 && aligned(g.res, 32) && g.ldr % 16 == 0 && aligned(g.z, 32) &&
             g.ldz % 16 == 0;
    g.M = (int)y.rows;
    g.N = (int)y.inner;
    const int64_t pm = (y.rows + 2 * BM - 1) / (2 * BM), pairs = sm_count() / 2;
    const int64_t w256 = (pm * ((y.inner + 255) / 256) + pairs - 1) / pairs, w128 = (pm * ((y.inner + 127) / 128) + pairs - 1) / pairs;
    bool narrow = 8 * w128 < 13 * w256;
    if (const char *v = getenv("LIN_BN")) narrow = atoi(v) == 128;
    return narrow ? launch_bn<A_MN, B_MN, 128, ACT>(a, b, g, K, s) : launch_bn<A_MN, B_MN, 256, ACT>(a, b, g, K, s);
}

}  // namespace pair
}  // namespace lin
