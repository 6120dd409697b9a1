// Fused linear layer for few rows: serving a token or a small batch.
//
// Included by linear.cu only (one translation unit: its device error word).
//
// With few rows the weights are the traffic: the kernel has to keep enough of
// W in flight on every SM, and the tensor cores have to take W as the operand
// of 128 rows (a tile of rows of x would be mostly padding).  So the product
// is formed transposed, D[feature][token] = sum_k W[n][k] x[m][k], with 128
// features by BT tokens per CTA (BT = 16, 32, 64 or 128, rows behind the last
// token read as zero), and K is split over the S CTAs of a cluster so that
// about two CTAs per SM stream W at once, each through a ring of some 100 KiB
// filled by TMA.  The S partial tiles stay on chip: every CTA leaves its fp32
// tile in shared memory, and the tokens of the tile are shared out among the
// CTAs, which add the S partials in rank order over distributed shared memory
// and run the epilogue.  No workspace, no atomics: the same bits every time.
//
// The gradients' products take the same shape where tiles are few and K is
// long: dx = dz W has W's columns as features, dW = dz^T x the columns of x,
// with dz's as tokens.  An operand whose features (or tokens) are contiguous in
// memory is MN-major, as in linear_pair.cuh.
//
// Roles (192 threads): warp 0 TMA producer, warp 1 MMA issuer, warps 2-5 take
// the accumulator out of tensor memory; all six add up and store.
// Every wait is bounded and records a failure in g_linear_error.
#pragma once

namespace lin {
namespace rows {

constexpr int BF = 128;                    // features per CTA
constexpr int BK = 64;
constexpr int THREADS = 192;
constexpr int W_BYTES = BF * BK * 2;       // 16 KiB
constexpr int kMaxCluster = 8;
constexpr int kMinBlocks = 4;              // blocks of k per CTA at least, where K is split
template <int BT> constexpr int stage_bytes() { return W_BYTES + BT * BK * 2; }
// two CTAs per SM: at most 113 KiB each
template <int BT> constexpr int stages() { return (112 * 1024 - 2048) / stage_bytes<BT>(); }
template <int BT> constexpr int smem_bytes() { return stages<BT>() * stage_bytes<BT>() + 1024 + 256; }

struct Args {
    Epilogue epi;
    const __nv_bfloat16 *res;
    __nv_bfloat16 *y, *z;
    int64_t ldr, ldy, ldz;
    int M, N, k_blocks;
};

// bf16 A and B, fp32 D, M = 128, N = BT; bits 15 and 16 mark MN-major operands.
template <int BT, bool F_MN, bool T_MN> constexpr uint32_t instr_desc() {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((F_MN ? 1u : 0u) << 15) | ((T_MN ? 1u : 0u) << 16) |
           ((uint32_t)(BT >> 3) << 17) | ((uint32_t)(BF >> 4) << 24);
}

// ROWS rows x 64 k of an operand into a stage.
template <bool MN, int ROWS>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int row, int k, uint32_t bar) {
    if constexpr (MN) {
#pragma unroll
        for (int h = 0; h < ROWS / 64; ++h) elect_tma_load(dst + h * 8192u, map, row + 64 * h, k, bar);
    } else {
        elect_tma_load(dst, map, k, row, bar);
    }
}

__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// The bias of features n .. n + 3 (zero where there is none).
__device__ __forceinline__ void load_bias(const Args &g, int n, float (&bias)[4]) {
    bias[0] = bias[1] = bias[2] = bias[3] = 0.f;
    if (g.epi.bias == nullptr || n >= g.N) return;
    if (g.epi.bias_bf16) load_weights_batched<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16 *>(g.epi.bias) + n, bias);
    else load_weights_batched<float, 4>(static_cast<const float *>(g.epi.bias) + n, bias);
}

// Adds up the partials of a CTA's tokens (rank, rank + ranks, ... of the tile's
// `valid`) and runs the epilogue: a warp of the block's NTHREADS per token, the
// features n .. n + 3 per thread, TOKENS tokens at a time.  partial(t, s) is
// the cluster address of token t's four features in rank s.
template <int ACT, int MAX_RANKS, int TOKENS, int NTHREADS, typename Partial>
__device__ __forceinline__ void finish(const Args &g, const Partial &partial, const float (&bias)[4], int n, int t0,
                                       int valid, int rank, int ranks) {
    constexpr int kStep = NTHREADS / 32;
    const int warp = threadIdx.x >> 5;
    if (n >= g.N) return;  // N is a multiple of 8
    for (int i = warp; rank + i * ranks < valid; i += TOKENS * kStep) {
        float4 part[TOKENS][MAX_RANKS];
        uint2 q[TOKENS];
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            const int t = rank + (i + u * kStep) * ranks;
            q[u] = make_uint2(0u, 0u);
            if (t >= valid) continue;
#pragma unroll
            for (int s = 0; s < MAX_RANKS; ++s)
                if (s < ranks) part[u][s] = ld_cluster_f32x4(partial(t, s));
            if (g.res != nullptr) q[u] = *reinterpret_cast<const uint2 *>(g.res + (int64_t)(t0 + t) * g.ldr + n);  // may be y itself
        }
#pragma unroll
        for (int u = 0; u < TOKENS; ++u) {
            const int t = rank + (i + u * kStep) * ranks;
            if (t >= valid) continue;
            float v[4] = {part[u][0].x, part[u][0].y, part[u][0].z, part[u][0].w};
#pragma unroll
            for (int s = 1; s < MAX_RANKS; ++s)
                if (s < ranks) {
                    v[0] += part[u][s].x;
                    v[1] += part[u][s].y;
                    v[2] += part[u][s].z;
                    v[3] += part[u][s].w;
                }
            const int64_t m = t0 + t;
            const float r = g.epi.inv_rms != nullptr ? __ldg(g.epi.inv_rms + m) : 1.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = fmaf(v[e], r, bias[e]);
            if (g.z != nullptr)
                *reinterpret_cast<uint2 *>(g.z + m * g.ldz + n) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            const float2 lo = activate2<ACT>(make_float2(v[0], v[1])), hi = activate2<ACT>(make_float2(v[2], v[3]));
            v[0] = lo.x;
            v[1] = lo.y;
            v[2] = hi.x;
            v[3] = hi.y;
            if (g.res != nullptr) {
                v[0] += bf16lo(q[u].x);
                v[1] += bf16hi(q[u].x);
                v[2] += bf16lo(q[u].y);
                v[3] += bf16hi(q[u].y);
            }
            *reinterpret_cast<uint2 *>(g.y + m * g.ldy + n) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
    }
}

// F_MN, T_MN: the operand of features, of tokens, is MN-major (tokens: 64 or 128 per tile).
template <int BT, int ACT, bool F_MN, bool T_MN>
__global__ void __launch_bounds__(THREADS, 2)
linear_rows_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x, const Args g) {
    constexpr int STAGES = stages<BT>(), STAGE_BYTES = stage_bytes<BT>();
    constexpr int TMEM_COLS = BT < 32 ? 32 : BT;
    static_assert(!T_MN || BT % 64 == 0, "an MN-major operand comes in blocks of 64");
    static_assert(BT * BF * 4 <= STAGES * STAGE_BYTES, "the partial tile reuses the ring");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * STAGE_BYTES), *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_full + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int n0 = (int)(blockIdx.x / ranks) * BF, t0 = (int)blockIdx.y * BT;
    const int kb0 = (int)((int64_t)g.k_blocks * rank / ranks), kb1 = (int)((int64_t)g.k_blocks * (rank + 1) / ranks);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(acc_full), 1);
        mbar_init_fence();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    gemm::tc_fence_before();
    __syncthreads();
    gemm::tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // the previous kernel on the stream has finished before any global memory is touched
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == 0) {
        // ---------------------------------------------------------------- TMA producer
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        // every tile of features starts elsewhere in its part of K: the CTAs then read other columns
        // of W and other parts of x at any one time (12288 x 4096, one token: 21.7 -> 20.8 us)
        int at = kb0 + (int)(blockIdx.x / ranks) * 5 % (kb1 - kb0);
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(smem_u32(&empty[stage]), phase ^ 1u, &g_linear_error)) break;
            const uint32_t fb = smem_u32(&full[stage]), sa = smem_u32(smem + stage * STAGE_BYTES);
            elect_expect_tx(fb, STAGE_BYTES);
            load_operand<F_MN, BF>(sa, &tmap_w, n0, at * BK, fb);
            load_operand<T_MN, BT>(sa + W_BYTES, &tmap_x, t0, at * BK, fb);
            if (++at == kb1) at = kb0;
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        // no copy may still be writing when the ring is reused (immediate on the normal path)
        for (int s = 0; s < STAGES; ++s)
            if (armed & (1u << s)) mbar_wait(smem_u32(&full[s]), (armed_parity >> s) & 1u, &g_linear_error);
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- MMA issuer
        const uint64_t a0 = pair::operand_desc<F_MN>(smem_u32(smem)), b0 = pair::operand_desc<T_MN>(smem_u32(smem + W_BYTES));
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!warp_wait(smem_u32(&full[stage]), phase, &g_linear_error)) break;
            gemm::tc_fence_after();
            const uint64_t at = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < BK / gemm::UMMA_K; ++k)
                elect_umma<1, instr_desc<BT, F_MN, T_MN>()>(tmem_base, a0 + at + k * pair::k_step<F_MN>(),
                                                            b0 + at + k * pair::k_step<T_MN>(), (kb != kb0 || k != 0) ? 1u : 0u);
            elect_commit<1>(smem_u32(&empty[stage]));
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
        elect_commit<1>(smem_u32(acc_full));  // every MMA issued here has completed
        __syncwarp();
    }
    float bias[4];  // of this thread's four features in the last step
    load_bias(g, n0 + 4 * lane, bias);
    // every thread: the accumulator is complete and no MMA reads the ring any more
    mbar_wait(smem_u32(acc_full), 0u, &g_linear_error, product_timeout(kb1 - kb0));
    gemm::tc_fence_after();
    __syncwarp();  // lanes come from the bias and the wait; tensor memory is read by whole warps
    __syncthreads();
    float *tile = reinterpret_cast<float *>(smem);  // [BT tokens][BF features]
    if (warp >= 2) {
        const int quarter = warp & 3;
#pragma unroll 1
        for (int c = 0; c < BT / 16; ++c) {
            uint32_t v[16];
            tmem_ld_16cols(tmem_base + ((uint32_t)(quarter * 32) << 16) + c * 16, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) tile[(c * 16 + i) * BF + quarter * 32 + lane] = __uint_as_float(v[i]);
        }
        gemm::tc_fence_before();
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    // Tokens rank, rank + ranks, ... of the tile: up to 16 partials of a thread's four features
    // are asked for before the first is added
    const uint32_t at = smem_u32(tile);
    const int n = n0 + 4 * lane, valid = min(BT, g.M - t0);
    auto partial = [&](int t, int s) { return map_to_rank(at + (uint32_t)(t * BF + 4 * lane) * 4u, (uint32_t)s); };
    if (ranks <= 2) finish<ACT, 2, 8, THREADS>(g, partial, bias, n, t0, valid, rank, ranks);
    else if (ranks <= 4) finish<ACT, 4, 4, THREADS>(g, partial, bias, n, t0, valid, rank, ranks);
    else finish<ACT, kMaxCluster, 2, THREADS>(g, partial, bias, n, t0, valid, rank, ranks);
    __syncwarp();  // lanes whose features lie behind the last have left `finish` before the others
    if (ranks > 1) cluster_sync();  // the other CTAs have read this one's tile
    else __syncthreads();
    if (warp == 1) {
        gemm::tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS) : "memory");
    }
}

// ---------------------------------------------------------------- host side

// CTAs that share a tile's K: up to one CTA per SM over kMinBlocks blocks of k each, or up to two,
// less an eighth that clusters cannot use, over four times as many.  One token: 12288 x 4096 21.6 us
// over 192 CTAs, 24.9 over 96 and 29.9 over 288, more than run at once; 4096 x 12288 18.9 split in
// 8, 19.6 in 4; 4096 x 4096 9.1 split in 8, 8.8 in 4.
inline int64_t split_of(int64_t tiles, int64_t k_blocks) {
    const int64_t sms = sm_count();
    const int64_t one = std::min<int64_t>(k_blocks / kMinBlocks, sms / tiles);
    const int64_t two = std::min<int64_t>(k_blocks / (4 * kMinBlocks), 7 * sms / 4 / tiles);
    const int64_t s = std::min<int64_t>(kMaxCluster, std::max(one, two));
    return s < 1 ? 1 : s;
}

template <int BT, int ACT, bool F_MN, bool T_MN>
qkn_status launch_bt(const pair::Matrix &x, const pair::Matrix &W, const Args &a, cudaStream_t s) {
    const auto kernel = linear_rows_kernel<BT, ACT, F_MN, T_MN>;
    CUtensorMap tw, tx;
    if (qkn_status st = make_tmap_pitched(&tw, W.p, W.rows, W.inner, W.pitch, BK, F_MN ? BK : BF)) return st;
    if (qkn_status st = make_tmap_pitched(&tx, x.p, x.rows, x.inner, x.pitch, BK, T_MN ? BK : BT)) return st;
    static std::atomic<bool> attr_set[64];  // per device: the attribute has been set
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (!known || !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<BT>());
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(linear_rows_kernel)");
        if (known) attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (a.N + BF - 1) / BF, token_tiles = (a.M + BT - 1) / BT;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes<BT>();
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    const int64_t split = split_of(tiles * token_tiles, a.k_blocks);
    cfg.numAttrs = 2;
    cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)token_tiles, 1);
    attr[0].val.clusterDim.x = (unsigned)split;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tw, tx, a);
    if (e != cudaSuccess) return cuda_fail(e, "linear_rows_kernel launch");
    return check_launch("linear_rows_kernel launch");
}

// About how long the kernel takes with bt tokens per tile, in ns: 3.5 us, and for each of the CTAs
// that share an SM its blocks of 64 k (c below) and the 25 ns a token takes in the last step.
// Measured like pair::cost; it leaves out the weights' way from DRAM, which is the same for
// every bt and sets the time of few tokens and many features, and how many clusters the device holds
// at once: 768 x 1024 x 1024, 48 tiles in clusters of three, takes 10.5 us with gelu where this says
// 7.4 (512 rows in clusters of four 7.9 and 6.2, 1024 rows by the split kernel 9.5).
inline int64_t cost(int64_t M, int64_t N, int64_t K, int bt) {
    const int64_t sms = sm_count(), kb = (K + BK - 1) / BK, tiles = ((N + BF - 1) / BF) * ((M + bt - 1) / bt);
    const int64_t c = bt == 16 ? 190 : bt == 32 ? 200 : bt == 64 ? 300 : 480;
    const int64_t split = split_of(tiles, kb);
    return 3500 + (tiles * split + sms - 1) / sms * ((kb + split - 1) / split * c + 25 * std::min<int64_t>(bt, M) / split);
}

// Tokens per tile (`least` or more) for a product of M tokens, N features and K, 0 where the pair
// kernel is estimated faster.  Forward products of up to 64 rows, where the weights are the
// traffic, it always serves; e.g. 256 x 4096 x 4096 19.3 us against 20.6 by the pair kernel, 128 x
// 12288 x 4096 36.7 against 32.1, 1024 x 1024 x 1024 9.2 against 9.3, 512 x 4096 x 4096 31.3 against
// 20.7.
inline int tokens_per_tile(int64_t M, int64_t N, int64_t K, bool forward, bool plain, int least) {
    int best = least;
    for (int bt = 2 * least; bt <= 128; bt *= 2)
        if (cost(M, N, K, bt) < cost(M, N, K, best)) best = bt;
    if ((M + best - 1) / best > 65535) return 0;  // the grid's second dimension
    if (!(forward && M <= 64) && cost(M, N, K, best) >= pair::cost(M, N, K, pair::columns_of(M, N, K, forward, plain), plain)) return 0;
    return best;
}

inline Args args_of(const pair::Matrix &y, const pair::Matrix *res, const pair::Matrix *z, const Epilogue &epi, int64_t K) {
    Args a;
    a.epi = epi;
    a.res = res ? static_cast<const __nv_bfloat16 *>(res->p) : nullptr;
    a.z = z ? static_cast<__nv_bfloat16 *>(const_cast<void *>(z->p)) : nullptr;
    a.y = static_cast<__nv_bfloat16 *>(const_cast<void *>(y.p));
    a.ldr = res ? res->pitch : 0;
    a.ldz = z ? z->pitch : 0;
    a.ldy = y.pitch;
    a.M = (int)y.rows;
    a.N = (int)y.inner;
    a.k_blocks = (int)((K + BK - 1) / BK);
    return a;
}

// y[token][feature] = epilogue of sum_k F(feature, k) T(token, k).
template <int ACT, bool F_MN, bool T_MN>
qkn_status launch(const pair::Matrix &t, const pair::Matrix &f, const pair::Matrix &y, const pair::Matrix *res,
                  const pair::Matrix *z, const Epilogue &epi, int64_t K, int tokens, cudaStream_t s) {
    const Args a = args_of(y, res, z, epi, K);
    if constexpr (!T_MN) {
        if (tokens == 16) return launch_bt<16, ACT, F_MN, false>(t, f, a, s);
        if (tokens == 32) return launch_bt<32, ACT, F_MN, false>(t, f, a, s);
    }
    if (tokens == 64) return launch_bt<64, ACT, F_MN, T_MN>(t, f, a, s);
    return launch_bt<128, ACT, F_MN, T_MN>(t, f, a, s);
}

}  // namespace rows
}  // namespace lin
