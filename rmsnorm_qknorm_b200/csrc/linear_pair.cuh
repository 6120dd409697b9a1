// Matrix product of the fused linear layer and its gradients on CTA pairs.
//
// Included by linear.cu only (one translation unit: its device error word).
//
//   C[m][n] = sum_k A(m, k) B(n, k),  256 x 256 (192, 128) tiles of C, bf16 in, fp32
// accumulated in tensor memory by tcgen05.mma.cta_group::2.  An operand is
// K-major (rows of consecutive k: x and W of the forward product) or MN-major
// (consecutive m or n: W in dx = dz W, dz and x in dW = dz^T x), read where it
// lies: no operand is transposed in memory.  A stage holds 64 k of 128 rows
// of each operand per CTA, as 128-byte-swizzled rows of 64 k, or as two
// blocks of 64 (k) rows of 64 m.
//
// Roles per CTA (320 threads): warp 0 moves tiles with TMA, the even CTA's
// warp 1 issues the MMAs (both as whole warps with an elected lane, see
// linear_issue.cuh), warps 2-9 run the epilogue of a tile
// while the MMAs of the next one run into the other accumulator: a quarter of
// the rows and every other 64 columns per warp, a row per thread: accumulator
// -> times the row's scale, plus bias -> z (stored where asked) -> activation
// -> plus residual -> y.  y leaves through 32 x 64 boxes in shared memory and
// TMA stores; the residual comes by TMA into the box that y then overwrites
// in place, one box ahead.  (Both read and written by the threads, a 32-byte
// sector of another row per lane, the requests to L2 alone took 2.6 us per
// tile and operand.)  z, which only training asks for, is written that way.
// Eight epilogue warps against sixteen, with gelu and a residual: 2048 x 8192 x
// 512 31.9 and 29.6 us, 8192 x 12288 x 4096 536 and 575-603.
// Every wait is bounded and records a failure in g_linear_error.
#pragma once

namespace lin {
namespace pair {

constexpr int BM = 128, BK = 64;                   // rows per CTA (256 per pair), k per stage
constexpr int A_BYTES = BM * BK * 2;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int BAR_BYTES = 320;

constexpr int BOX_COLS = 64, BOX_BYTES = 32 * BOX_COLS * 2;  // an epilogue warp's staging box: 32 rows

// The tile's columns: 256, or 192 or 128 where wider tiles leave pairs without work.
template <int BN> struct Shape {
    static constexpr int EPI_BYTES = EPI_WARPS * 2 * BOX_BYTES;
    static constexpr int BN_CTA = BN / 2;          // rows of B that each CTA loads
    static constexpr int B_BYTES = BN_CTA * BK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int BIAS_BYTES = 4 * BOX_COLS * 4;
    static constexpr int STAGES = (227 * 1024 - BAR_BYTES - 1024 - EPI_BYTES - BIAS_BYTES) / STAGE_BYTES;
    static constexpr int PAIR_STAGE_BYTES = 2 * STAGE_BYTES;
    static constexpr int TMEM_COLS = BN > 128 ? 512 : 256;  // two accumulators
    static constexpr int BOXES = BN / BOX_COLS;    // of a row of the tile
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EPI_BYTES + BIAS_BYTES + BAR_BYTES + 1024;
    static_assert(SMEM_BYTES <= 227 * 1024 && (2 * STAGES + 6 + 2 * EPI_WARPS) * 8 <= BAR_BYTES, "shared memory budget");
};
constexpr int GROUP_M = 16;  // pair row blocks walked together down each column block (operands shared in L2)

struct Args {
    Epilogue epi;
    __nv_bfloat16 *z;
    int64_t ldz;
    int wide;              // the rows of z are 32-byte aligned
    int has_res;
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
__device__ __forceinline__ void store16(__nv_bfloat16 *p, bool wide, int left, const float2 *f) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(f[i].x, f[i].y);
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
                   const __grid_constant__ CUtensorMap tmap_y, const __grid_constant__ CUtensorMap tmap_res, const Args g) {
    using S = Shape<BN>;
    constexpr int STAGES = S::STAGES, STAGE_BYTES = S::STAGE_BYTES, BN_CTA = S::BN_CTA;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES + S::EPI_BYTES + S::BIAS_BYTES);
    uint64_t *full = bars, *empty = bars + STAGES;
    uint64_t *acc_full = bars + 2 * STAGES, *acc_empty = bars + 2 * STAGES + 2;
    uint64_t *drained = bars + 2 * STAGES + 4;
    uint64_t *res_full = bars + 2 * STAGES + 5;  // [EPI_WARPS][2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(res_full + 2 * EPI_WARPS);

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
        for (int i = 0; i < 2 * EPI_WARPS; ++i) mbar_init(smem_u32(&res_full[i]), 1);
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
                const uint32_t d_tmem = tmem_base + acc * (S::TMEM_COLS / 2);
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
        const int half = (warp - 2) >> 2;   // its boxes of the tile: half, half + 2
        const int own = (S::BOXES + 1 - half) / 2;
        const uint32_t acc_empty_leader0 = map_to_rank(smem_u32(&acc_empty[0]), 0);
        const uint32_t boxes = smem_u32(smem + STAGES * STAGE_BYTES) + (uint32_t)(warp - 2) * 2u * BOX_BYTES;
        const uint32_t rbar = smem_u32(&res_full[2 * (warp - 2)]);
        float *bias = reinterpret_cast<float *>(smem + STAGES * STAGE_BYTES + S::EPI_BYTES) + half * 2 * BOX_COLS;
        const bool wide = g.wide != 0, has_res = g.has_res != 0;
        uint32_t box = 0, asked = 0;  // boxes stored so far, residual boxes asked for
        bool ok = true;
        // corner of this warp's j-th box of a tile; false when it lies outside C
        auto corner = [&](int tile, int j, int &row0, int &col0) {
            int pm, n;
            tile_coords(tile, g, pm, n);
            row0 = pm * 2 * BM + (int)rank * BM + quarter * 32;
            col0 = n * BN + (half + 2 * j) * BOX_COLS;
            return row0 < g.M && col0 < g.N;
        };
        // the residual of a box into the buffer its y leaves from; the stores issued so far have
        // been read by then
        auto fetch = [&](int row0, int col0) {
            const uint32_t bar = rbar + (asked & 1u) * 8u;
            if (lane == 0) {
                bulk_wait_read0();
                mbar_arrive_expect_tx(bar, BOX_BYTES);
                tma_load_2d(boxes + (asked & 1u) * BOX_BYTES, &tmap_res, col0, row0, bar);
            }
            ++asked;
        };
        int it = 0;
        // after a wait that gave up (!ok) a warp still meets the others at every barrier
        for (int tile = pair_id; tile < g.num_tiles; tile += num_pairs, ++it) {
            int row0, col0;
            if (corner(tile, 0, row0, col0) && has_res && ok && asked == box) fetch(row0, col0);
            const int acc = it & 1;
            const uint32_t acc_phase = (it >> 1) & 1;
            const int row = row0 + lane;
            const bool in = row < g.M;
            __nv_bfloat16 *z = g.z != nullptr && in ? g.z + row * g.ldz : nullptr;
            // the columns' bias, which the four warps of these boxes share
            asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + half) : "memory");
            if (const int i = quarter * 32 + lane; i < own * BOX_COLS) {
                const int c = col0 + i + (i >= BOX_COLS ? BOX_COLS : 0);
                float b = 0.f;
                if (g.epi.bias != nullptr && c < g.N)
                    b = g.epi.bias_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(g.epi.bias)[c])
                                        : static_cast<const float *>(g.epi.bias)[c];
                bias[i] = b;
            }
            const float r = g.epi.inv_rms != nullptr && in ? __ldg(g.epi.inv_rms + row) : 1.f;
            asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + half) : "memory");
            if (ok) ok = warp_wait(smem_u32(&acc_full[acc]), acc_phase, &g_linear_error, product_timeout(g.k_blocks));
            gemm::tc_fence_after();
            const uint32_t tbase = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * (S::TMEM_COLS / 2) + half * BOX_COLS;
            for (int j = 0; ok && j < own; ++j) {
                const int col = col0 + 2 * j * BOX_COLS;
                if (row0 >= g.M || col >= g.N) break;  // the boxes behind it lie outside, too
                const uint32_t buf = boxes + (box & 1u) * BOX_BYTES;
                if (has_res) {
                    ok = warp_wait(rbar + (box & 1u) * 8u, (box >> 1) & 1u, &g_linear_error);
                    if (!ok) break;
                } else if (lane == 0 && box >= 2) {
                    bulk_wait_read1();  // the store that used this buffer has read it
                }
                __syncwarp();
#pragma unroll 1
                for (int c = 0; c < BOX_COLS / 32; ++c) {
                    uint32_t v[32];
                    __syncwarp();  // rows behind the last store no z, one lane asks for the residual
                    gemm::tmem_ld_32cols(tbase + 2 * j * BOX_COLS + c * 32, v);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 f[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 b = *reinterpret_cast<const float4 *>(bias + j * BOX_COLS + c * 32 + h * 16 + 4 * e);
                            f[2 * e] = __ffma2_rn(make_float2(__uint_as_float(v[16 * h + 4 * e]), __uint_as_float(v[16 * h + 4 * e + 1])),
                                                  pair_of(r), make_float2(b.x, b.y));
                            f[2 * e + 1] = __ffma2_rn(make_float2(__uint_as_float(v[16 * h + 4 * e + 2]), __uint_as_float(v[16 * h + 4 * e + 3])),
                                                      pair_of(r), make_float2(b.z, b.w));
                        }
                        const int at = col + c * 32 + h * 16;
                        if (z != nullptr) store16(z + at, wide, g.N - at, f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = activate2<ACT>(f[e]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            // 16-byte chunk of the box's 128-byte row, at its place in the 128-byte swizzle
                            const uint32_t p = buf + (uint32_t)lane * 128u + (uint32_t)(((c * 4 + h * 2 + k) ^ (lane & 7)) * 16);
                            if (has_res) {
                                uint4 q;
                                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(p) : "memory");
                                f[4 * k] = __fadd2_rn(f[4 * k], make_float2(bf16lo(q.x), bf16hi(q.x)));
                                f[4 * k + 1] = __fadd2_rn(f[4 * k + 1], make_float2(bf16lo(q.y), bf16hi(q.y)));
                                f[4 * k + 2] = __fadd2_rn(f[4 * k + 2], make_float2(bf16lo(q.z), bf16hi(q.z)));
                                f[4 * k + 3] = __fadd2_rn(f[4 * k + 3], make_float2(bf16lo(q.w), bf16hi(q.w)));
                            }
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                         ::"r"(p), "r"(pack_bf16x2(f[4 * k].x, f[4 * k].y)),
                                         "r"(pack_bf16x2(f[4 * k + 1].x, f[4 * k + 1].y)),
                                         "r"(pack_bf16x2(f[4 * k + 2].x, f[4 * k + 2].y)),
                                         "r"(pack_bf16x2(f[4 * k + 3].x, f[4 * k + 3].y)) : "memory");
                        }
                    }
                    if (has_res && c == 0) {  // the next box's residual, into the other buffer
                        int r1, c1;
                        const bool more = j + 1 < own && col + 2 * BOX_COLS < g.N;
                        if (more ? corner(tile, j + 1, r1, c1) : tile + num_pairs < g.num_tiles && corner(tile + num_pairs, 0, r1, c1))
                            fetch(r1, c1);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&tmap_y, buf, col, row0);
                    bulk_commit();
                }
                ++box;
            }
            gemm::tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acc_empty_leader0 + (uint32_t)acc * 8u);
        }
        // no copy into or out of the boxes is in flight at the exit
        if (lane == 0) {
            for (; box < asked; ++box) mbar_wait(rbar + (box & 1u) * 8u, (box >> 1) & 1u, &g_linear_error);
            bulk_wait_all();
        }
        __syncwarp();
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
qkn_status launch_bn(const Matrix &a, const Matrix &b, const Matrix &y, const Matrix *res, Args &g, int64_t K,
                     cudaStream_t s) {
    using S = Shape<BN>;
    const auto kernel = linear_pair_kernel<A_MN, B_MN, BN, ACT>;
    CUtensorMap ta, tb, ty, tr;
    if (qkn_status st = make_tmap_pitched(&ty, y.p, y.rows, y.inner, y.pitch, BOX_COLS, 32)) return st;
    tr = ty;
    if (res != nullptr)
        if (qkn_status st = make_tmap_pitched(&tr, res->p, res->rows, res->inner, res->pitch, BOX_COLS, 32)) return st;
    if (qkn_status st = make_tmap_pitched(&ta, a.p, a.rows, a.inner, a.pitch, BK, A_MN ? BK : BM)) return st;
    if (qkn_status st = make_tmap_pitched(&tb, b.p, b.rows, b.inner, b.pitch, BK, B_MN ? BK : S::BN_CTA)) return st;
    g.pm_blocks = (int)(((int64_t)g.M + 2 * BM - 1) / (2 * BM));
    g.n_blocks = (int)(((int64_t)g.N + BN - 1) / BN);
    g.k_blocks = (int)((K + BK - 1) / BK);
    if ((int64_t)g.pm_blocks * g.n_blocks > 0x7fff0000LL) return fail(QKN_ERR_SHAPE, "linear_pair_kernel: too many tiles");
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, ty, tr, g);
    if (e != cudaSuccess) return cuda_fail(e, "linear_pair_kernel launch");
    return check_launch("linear_pair_kernel launch");
}

// About how long the kernel takes, in ns: 4 us, and for every round of tiles over the pairs its
// products (64 k: 340 ns at 256 columns, 290 at 192, 240 at 128) or, for short K, its epilogue,
// which an activation, a residual or a kept z makes longer (`plain` without them).  Measured with
// 512 .. 12288 columns, K 512 .. 12288 and 128 .. 2048 rows, gelu and a residual: within a tenth of
// it, e.g. 512 x 4096 x 4096 27.6 us (256 columns, 32 of 74 pairs) against 20.7 (128), 2048 x 4096 x
// 4096 52.8 against 70.2; without them 4096 x 4096 x 64 15.6; 192 columns against the better of the
// others: 512 x 12288 x 4096 47 and 57, 1536 x 4096 x 12288 120 and 137.
inline int64_t cost(int64_t M, int64_t N, int64_t K, int bn, bool plain) {
    const int64_t pairs = sm_count() > 1 ? sm_count() / 2 : 1, kb = (K + BK - 1) / BK;
    const int64_t tiles = ((M + 2 * BM - 1) / (2 * BM)) * ((N + bn - 1) / bn);
    const int64_t round = bn == 256   ? std::max<int64_t>(plain ? 3000 : 7000, 2500 + 340 * kb)
                          : bn == 192 ? std::max<int64_t>(plain ? 3000 : 7000, 2500 + 290 * kb)
                                      : std::max<int64_t>(plain ? 2000 : 4400, 1500 + 240 * kb);
    return 4000 + (tiles + pairs - 1) / pairs * round;
}

// The columns of the tile.  MN-major operands come in blocks of 64, of which each CTA takes half a
// tile's: 256 or 128.
inline int columns_of(int64_t M, int64_t N, int64_t K, bool k_major, bool plain) {
    int best = 256;
    if (k_major && cost(M, N, K, 192, plain) < cost(M, N, K, best, plain)) best = 192;
    if (cost(M, N, K, 128, plain) < cost(M, N, K, best, plain)) best = 128;
    return best;
}

template <bool A_MN, bool B_MN, int ACT>
qkn_status launch(const Matrix &a, const Matrix &b, const Matrix &y, const Matrix *res, const Matrix *z,
                  const Epilogue &epi, int64_t K, cudaStream_t s) {
    Args g;
    g.epi = epi;
    g.has_res = res != nullptr;
    g.z = z ? static_cast<__nv_bfloat16 *>(const_cast<void *>(z->p)) : nullptr;
    g.ldz = z ? z->pitch : 0;
    g.wide = aligned(g.z, 32) && g.ldz % 16 == 0;
    g.M = (int)y.rows;
    g.N = (int)y.inner;
    const bool plain = ACT == QKN_ACT_NONE && res == nullptr && z == nullptr;
    const int bn = columns_of(g.M, g.N, K, !A_MN && !B_MN, plain);
    if constexpr (!A_MN && !B_MN)
        if (bn == 192) return launch_bn<A_MN, B_MN, 192, ACT>(a, b, y, res, g, K, s);
    if (bn == 128) return launch_bn<A_MN, B_MN, 128, ACT>(a, b, y, res, g, K, s);
    return launch_bn<A_MN, B_MN, 256, ACT>(a, b, y, res, g, K, s);
}

}  // namespace pair
}  // namespace lin
