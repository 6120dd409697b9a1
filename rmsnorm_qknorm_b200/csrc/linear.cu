// Fused linear layer: y = act(r (x W^T) + b) + residual, and its gradients.
//
//   z = r_m sum_k x[m][k] W[n][k] + b[n],  y = act(z) + residual
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz
// The products run on the tensor cores (linear_rows.cuh for few rows,
// linear_pair.cuh for many, linear_split.cuh between) with everything else in
// their epilogue; dz is formed once (and rounded to bf16, the products'
// operand type) by an element-wise pass that adds up db in fp32 on the way.
// That rounding takes dx and dW from 1.7 x 10^-3 of their norm off the 64-bit
// result (their own rounding alone) to 2.3 x 10^-3 at 4096 x 12288 x 4096; dz as
// a sum of two bf16 parts would double the time of both products.
#include <algorithm>
#include <atomic>
#include <cuda.h>
#include <math.h>

#include "gemm_tc.cuh"
#include "linear_issue.cuh"
#include "linear_math.cuh"
#include "pair_tc.cuh"
#include "qkn_common.cuh"
#include "qkn_sync.cuh"

namespace qkn {

// Set by a bounded wait of the linear kernels that gave up (see qkn_check_device).
__device__ int g_linear_error = 0;

#include "linear_pair.cuh"
#include "linear_rows.cuh"
#include "linear_split.cuh"

namespace lin {

// ---------------------------------------------------------------- dz and db

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// dz = dy act'(z) and the partial column sums of dz: a block walks the rows of
// its slice over 256 columns, a 16-byte chunk per thread, eight rows side by
// side and four of those groups at a time, all their loads issued before any
// arithmetic; the eight rows' sums meet in shared memory in row order.  The
// slices' sums go to part, for linear_db_kernel, or (db given: few rows, the
// slices of 256 columns are a cluster) meet in the first slice's block, in
// slice order, which saves the second launch.
constexpr int kDzCols = 256, kDzThreads = 256, kDzRows = 8, kDzUnroll = 4;

template <int ACT>
__global__ void __launch_bounds__(kDzThreads) linear_dz_kernel(const __nv_bfloat16 *__restrict__ dy,
                                                               const __nv_bfloat16 *__restrict__ z,
                                                               __nv_bfloat16 *__restrict__ dz, float *__restrict__ part,
                                                               float *__restrict__ db, int64_t M, int N, int64_t lddy, int64_t ldz, int slices) {
    __shared__ float red[kDzRows][kDzCols + 4], total[kDzCols];
    const int chunk = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int col = blockIdx.x * kDzCols + chunk * 8;
    const bool in = col < N;
    float2 sum[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = pair_of(0.f);
    const int64_t step = (int64_t)slices * kDzRows;
    for (int64_t row0 = (int64_t)blockIdx.y * kDzRows + rl; in && row0 < M; row0 += kDzUnroll * step) {
        uint4 g[kDzUnroll], v[kDzUnroll];
#pragma unroll
        for (int u = 0; u < kDzUnroll; ++u) {
            const int64_t row = row0 + u * step;
            g[u] = v[u] = make_uint4(0u, 0u, 0u, 0u);
            if (row < M) {
                g[u] = ld_stream(dy + row * lddy + col);
                if constexpr (ACT != QKN_ACT_NONE) v[u] = ld_stream(z + row * ldz + col);
            }
        }
#pragma unroll
        for (int u = 0; u < kDzUnroll; ++u) {
            const int64_t row = row0 + u * step;
            if (row >= M) continue;
            float2 f[4] = {make_float2(bf16lo(g[u].x), bf16hi(g[u].x)), make_float2(bf16lo(g[u].y), bf16hi(g[u].y)),
                           make_float2(bf16lo(g[u].z), bf16hi(g[u].z)), make_float2(bf16lo(g[u].w), bf16hi(g[u].w))};
            if constexpr (ACT != QKN_ACT_NONE) {
                f[0] = __fmul2_rn(f[0], slope2<ACT>(make_float2(bf16lo(v[u].x), bf16hi(v[u].x))));
                f[1] = __fmul2_rn(f[1], slope2<ACT>(make_float2(bf16lo(v[u].y), bf16hi(v[u].y))));
                f[2] = __fmul2_rn(f[2], slope2<ACT>(make_float2(bf16lo(v[u].z), bf16hi(v[u].z))));
                f[3] = __fmul2_rn(f[3], slope2<ACT>(make_float2(bf16lo(v[u].w), bf16hi(v[u].w))));
                *reinterpret_cast<uint4 *>(dz + row * N + col) =
                    make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                               pack_bf16x2(f[3].x, f[3].y));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = __fadd2_rn(sum[e], f[e]);
        }
    }
    if (part == nullptr && db == nullptr) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        red[rl][chunk * 8 + 2 * e] = sum[e].x;
        red[rl][chunk * 8 + 2 * e + 1] = sum[e].y;
    }
    __syncthreads();
    const int c = blockIdx.x * kDzCols + threadIdx.x;
    float s = red[0][threadIdx.x];
#pragma unroll
    for (int j = 1; j < kDzRows; ++j) s += red[j][threadIdx.x];
    if (db == nullptr) {
        if (c < N) part[(int64_t)blockIdx.y * N + c] = s;
        return;
    }
    total[threadIdx.x] = s;
    cluster_sync();
    if (blockIdx.y == 0 && c < N) {
        for (int r = 1; r < slices; ++r) s += ld_cluster_f32(map_to_rank(smem_u32(&total[threadIdx.x]), (uint32_t)r));
        db[c] = s;
    }
    cluster_sync();  // the first block has read this one's sums
}

// db[c] = sum over slices of part[slice][c], in a fixed order.
__global__ void __launch_bounds__(256) linear_db_kernel(const float *__restrict__ part, float *__restrict__ db, int N,
                                                        int slices) {
    __shared__ float red[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    float s = 0.f;
    if (col < N)
        for (int i = k; i < slices; i += 8) s += part[(int64_t)i * N + col];
    red[k][threadIdx.x & 31] = s;
    __syncthreads();
    if (k == 0 && col < N) {
        float v = red[0][threadIdx.x];
#pragma unroll
        for (int j = 1; j < 8; ++j) v += red[j][threadIdx.x];
        db[col] = v;
    }
}

// Slices of a cluster, where the columns' sums are asked for and the rows so few that each block has
// one round of loads; 0 for more rows.  A gradient call 28.4 -> 26.2 us on the host, the pass 3.4 ->
// 3.8 us on the device (64 x 256); with 1024 rows it would take 8.5 us against 4.6.
constexpr int kDzCluster = 8;
int dz_cluster(int64_t M) {
    return M > kDzCluster * kDzRows * kDzUnroll ? 0 : (int)std::min<int64_t>(kDzCluster, (M + kDzRows - 1) / kDzRows);
}

// Row slices of the pass otherwise: about six 256-thread blocks per SM in all, at least a row group each.
int dz_slices(int64_t M, int64_t N) {
    const int64_t cols = (N + kDzCols - 1) / kDzCols, groups = (M + kDzRows - 1) / kDzRows;
    int64_t s = 6 * (int64_t)sm_count() / cols;
    if (s < 1) s = 1;
    if (s > groups) s = groups;
    return (int)s;
}

size_t dz_bytes(int64_t M, int64_t N, int act) {
    return act == QKN_ACT_NONE ? 0 : ((size_t)M * (size_t)N * 2 + 255) / 256 * 256;
}

// dz (with an activation) and db (where given).
template <int ACT>
qkn_status launch_dz(const __nv_bfloat16 *dy, const __nv_bfloat16 *z, __nv_bfloat16 *dz, float *part, float *db, int64_t M,
                     int64_t N, int64_t lddy, int64_t ldz, cudaStream_t s) {
    const unsigned cols = (unsigned)((N + kDzCols - 1) / kDzCols);
    if (const int slices = db != nullptr ? dz_cluster(M) : 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(cols, (unsigned)slices, 1);
        cfg.blockDim = dim3(kDzThreads, 1, 1);
        cfg.stream = s;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = attr.val.clusterDim.z = 1;
        attr.val.clusterDim.y = (unsigned)slices;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, linear_dz_kernel<ACT>, dy, z, dz, (float *)nullptr, db, M, (int)N, lddy,
                                                 ldz, slices);
        return e == cudaSuccess ? check_launch("linear_dz_kernel launch") : cuda_fail(e, "linear_dz_kernel launch");
    }
    const int slices = dz_slices(M, N);
    linear_dz_kernel<ACT><<<dim3(cols, (unsigned)slices), kDzThreads, 0, s>>>(dy, z, dz, db ? part : nullptr, nullptr, M, (int)N,
                                                                             lddy, ldz, slices);
    qkn_status st = check_launch("linear_dz_kernel launch");
    if (st == QKN_OK && db != nullptr) {
        linear_db_kernel<<<(unsigned)((N + 31) / 32), 256, 0, s>>>(part, db, (int)N, slices);
        st = check_launch("linear_db_kernel launch");
    }
    return st;
}

// One product by the kernel with the least estimated time.  Forward: x [M][K], W [N][K].  dx: dz and
// W (MN-major), dW: dz and x (both MN-major).
template <bool A_MN, bool B_MN, int ACT>
qkn_status product(const pair::Matrix &a, const pair::Matrix &b, const pair::Matrix &y, const pair::Matrix *res,
                   const pair::Matrix *z, const Epilogue &epi, int64_t K, cudaStream_t s) {
    constexpr bool kForward = !A_MN && !B_MN;
    const bool plain = ACT == QKN_ACT_NONE && !res && !z;
    const int64_t M = y.rows, N = y.inner;
    const int tokens = rows::tokens_per_tile(M, N, K, kForward, plain, A_MN ? 64 : 16);
    if (M > 64) {
        const int64_t others = tokens ? rows::cost(M, N, K, tokens)
                                      : pair::cost(M, N, K, pair::columns_of(M, N, K, kForward, plain), plain);
        if (const split::Choice c = split::choose(M, N, K, others); c.columns)
            return split::launch<A_MN, B_MN, ACT>(a, b, y, res, z, epi, K, c, s);
    }
    if (tokens) return rows::launch<ACT, B_MN, A_MN>(a, b, y, res, z, epi, K, tokens, s);
    return pair::launch<A_MN, B_MN, ACT>(a, b, y, res, z, epi, K, s);
}

bool pitch_ok(int64_t ld, int64_t width) { return ld >= width && ld % 8 == 0; }

Span span_of(const pair::Matrix &m) { return {m.p, m.rows, m.inner * 2, m.pitch * 2}; }

// Whether the rows of a bf16 result share memory with those of another matrix, or with a vector.
bool meets(const pair::Matrix &y, const pair::Matrix &m) { return rows_overlap(span_of(y), span_of(m)); }
bool meets(const pair::Matrix &y, const Span &v) { return rows_overlap(span_of(y), v); }

}  // namespace lin

qkn_status read_linear_error(int *flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_linear_error, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "reading the linear kernels' device error word");
    if (*flag) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_linear_error, &zero, sizeof zero);
    }
    return QKN_OK;
}

}  // namespace qkn

using namespace qkn;

// Rows and columns at most, so that a tile behind the last one still has 32-bit coordinates.
static constexpr int64_t kMaxSize = 0x7ffffe00LL;

extern "C" QKN_API qkn_status linear_fused(const void *x, const void *W, void *y, int64_t M, int64_t N, int64_t K,
                                           int64_t ldx, int64_t ldw, int64_t ldy, const void *bias, qkn_dtype bias_dt,
                                           qkn_activation act, const void *residual, int64_t ldr, const float *inv_rms,
                                           void *preact, int64_t ldz, void *stream) {
    const char *fn = "linear_fused";
    if (M < 0 || N < 1 || K < 1 || M > kMaxSize || N > kMaxSize || K > kMaxSize)
        return fail(QKN_ERR_SHAPE, "%s: bad sizes M=%lld N=%lld K=%lld", fn, (long long)M, (long long)N, (long long)K);
    if (K % 8 != 0 || N % 8 != 0)
        return fail(QKN_ERR_SHAPE, "%s: K=%lld and N=%lld must be multiples of 8", fn, (long long)K, (long long)N);
    if (!lin::pitch_ok(ldx, K) || !lin::pitch_ok(ldw, K) || !lin::pitch_ok(ldy, N) ||
        (residual && !lin::pitch_ok(ldr, N)) || (preact && !lin::pitch_ok(ldz, N)))
        return fail(QKN_ERR_SHAPE, "%s: leading dimensions must be multiples of 8 and at least the row width", fn);
    if (bias && !valid_dtype(bias_dt)) return fail(QKN_ERR_DTYPE, "%s: unknown bias dtype %d", fn, (int)bias_dt);
    if ((int)act < QKN_ACT_NONE || (int)act > QKN_ACT_GELU_TANH)
        return fail(QKN_ERR_UNSUPPORTED, "%s: unknown activation %d", fn, (int)act);
    if (M == 0) return QKN_OK;
    if (x == nullptr || W == nullptr || y == nullptr) return fail(QKN_ERR_NULL, "%s: x, W and y are required", fn);
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(y, 16) || !aligned(bias, 16) || !aligned(residual, 16) ||
        !aligned(preact, 16) || !aligned(inv_rms, 4))
        return fail(QKN_ERR_ALIGN, "%s: x, W, y, bias, residual and preact must be 16-byte aligned", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const lin::pair::Matrix mx = {x, M, K, ldx}, mw = {W, N, K, ldw}, my = {y, M, N, ldy}, mr = {residual, M, N, ldr},
                            mz = {preact, M, N, ldz};
    const Span vb = flat(bias, N * (int64_t)dtype_size(bias_dt)), vr = flat(inv_rms, 4 * M);
    const bool in_place = residual == y && (M == 1 || ldr == ldy);
    if (lin::meets(my, mx) || lin::meets(my, mw) || lin::meets(my, mz) || (lin::meets(my, mr) && !in_place) ||
        lin::meets(mz, mx) || lin::meets(mz, mw) || lin::meets(mz, mr) || lin::meets(my, vb) || lin::meets(my, vr) ||
        lin::meets(mz, vb) || lin::meets(mz, vr))
        return fail(QKN_ERR_UNSUPPORTED, "%s: y or preact shares memory with an input or with one another", fn);
    const lin::pair::Matrix *res = residual ? &mr : nullptr, *z = preact ? &mz : nullptr;
    lin::Epilogue e{};
    e.inv_rms = inv_rms;
    e.bias = bias;
    e.bias_bf16 = bias_dt == QKN_BF16;
    switch (act) {
    case QKN_ACT_RELU: return lin::product<false, false, QKN_ACT_RELU>(mx, mw, my, res, z, e, K, s);
    case QKN_ACT_SILU: return lin::product<false, false, QKN_ACT_SILU>(mx, mw, my, res, z, e, K, s);
    case QKN_ACT_GELU: return lin::product<false, false, QKN_ACT_GELU>(mx, mw, my, res, z, e, K, s);
    case QKN_ACT_GELU_TANH: return lin::product<false, false, QKN_ACT_GELU_TANH>(mx, mw, my, res, z, e, K, s);
    default: return lin::product<false, false, QKN_ACT_NONE>(mx, mw, my, res, z, e, K, s);
    }
}

extern "C" QKN_API size_t linear_fused_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, qkn_activation act) {
    if (M < 0 || N < 1 || K < 1 || M > kMaxSize || N > kMaxSize || K > kMaxSize || (int)act < QKN_ACT_NONE ||
        (int)act > QKN_ACT_GELU_TANH)
        return 0;
    return lin::dz_bytes(M, N, act) + (M ? (size_t)lin::dz_slices(M, N) * (size_t)N * 4 : 0) + 16;
}

extern "C" QKN_API qkn_status linear_fused_backward(const void *dy, const void *preact, const void *x, const void *W,
                                                    void *dx, void *dW, float *dbias, int64_t M, int64_t N, int64_t K,
                                                    int64_t lddy, int64_t ldz, int64_t ldx, int64_t ldw, int64_t lddx,
                                                    int64_t lddw, qkn_activation act, void *workspace,
                                                    size_t workspace_bytes, void *stream) {
    const char *fn = "linear_fused_backward";
    if (M < 0 || N < 1 || K < 1 || M > kMaxSize || N > kMaxSize || K > kMaxSize)
        return fail(QKN_ERR_SHAPE, "%s: bad sizes M=%lld N=%lld K=%lld", fn, (long long)M, (long long)N, (long long)K);
    if (K % 8 != 0 || N % 8 != 0)
        return fail(QKN_ERR_SHAPE, "%s: K=%lld and N=%lld must be multiples of 8", fn, (long long)K, (long long)N);
    if ((int)act < QKN_ACT_NONE || (int)act > QKN_ACT_GELU_TANH)
        return fail(QKN_ERR_UNSUPPORTED, "%s: unknown activation %d", fn, (int)act);
    const bool has_z = act != QKN_ACT_NONE;
    if (!lin::pitch_ok(lddy, N) || (has_z && !lin::pitch_ok(ldz, N)) || (dW && !lin::pitch_ok(ldx, K)) ||
        (dx && !lin::pitch_ok(ldw, K)) || (dx && !lin::pitch_ok(lddx, K)) || (dW && !lin::pitch_ok(lddw, K)))
        return fail(QKN_ERR_SHAPE, "%s: leading dimensions must be multiples of 8 and at least the row width", fn);
    if (dx == nullptr && dW == nullptr && dbias == nullptr) return QKN_OK;
    if (M > 0) {
        if (dy == nullptr || (has_z && preact == nullptr) || (dW && x == nullptr) || (dx && W == nullptr))
            return fail(QKN_ERR_NULL, "%s: dy, preact (with an activation), x (for dW) and W (for dx) are required", fn);
        if (!aligned(dy, 16) || !aligned(preact, 16) || !aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16))
            return fail(QKN_ERR_ALIGN, "%s: dy, preact, x, W and dx must be 16-byte aligned", fn);
    }
    if (!aligned(dW, 16) || !aligned(dbias, 4))
        return fail(QKN_ERR_ALIGN, "%s: dW must be 16-byte aligned, dbias 4-byte aligned", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t need = linear_fused_backward_workspace_bytes(M, N, K, act);
    if (workspace != nullptr) {
        if (workspace_bytes < need)
            return fail(QKN_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
        if (!aligned(workspace, 16)) return fail(QKN_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    }
    if (M == 0) {  // no rows: the gradients of W and b are empty sums
        cudaError_t e = cudaSuccess;
        if (dW != nullptr) e = cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)K * 2, (size_t)N, s);
        if (e == cudaSuccess && dbias != nullptr) e = cudaMemsetAsync(dbias, 0, (size_t)N * 4, s);
        return e == cudaSuccess ? QKN_OK : cuda_fail(e, "linear_fused_backward: clearing the gradients");
    }
    {
        const lin::pair::Matrix results[2] = {{dx, M, K, lddx}, {dW, N, K, lddw}};
        const lin::pair::Matrix inputs[4] = {{dy, M, N, lddy}, {has_z ? preact : nullptr, M, N, ldz},
                                             {dW ? x : nullptr, M, K, ldx}, {dx ? W : nullptr, N, K, ldw}};
        bool met = lin::meets(results[0], results[1]);
        for (const lin::pair::Matrix &r : results)
            for (const lin::pair::Matrix &m : inputs) met = met || lin::meets(r, m);
        const Span sums = flat(dbias, 4 * N);
        for (const lin::pair::Matrix &r : results) met = met || lin::meets(r, sums);
        for (const lin::pair::Matrix &m : inputs) met = met || lin::meets(m, sums);
        if (met) return fail(QKN_ERR_UNSUPPORTED, "%s: dx, dW or dbias shares memory with an input or with one another", fn);
        const Span ws = flat(workspace, (int64_t)need);  // written before the products read their operands
        met = rows_overlap(ws, sums);
        for (const lin::pair::Matrix &r : results) met = met || lin::meets(r, ws);
        for (const lin::pair::Matrix &m : inputs) met = met || lin::meets(m, ws);
        if (met) return fail(QKN_ERR_UNSUPPORTED, "%s: the workspace shares memory with an input or a result", fn);
    }
    void *own = nullptr;
    if (workspace == nullptr && (has_z || dbias != nullptr)) {
        const cudaError_t e = cudaMallocAsync(&own, need, s);
        if (e != cudaSuccess) return cuda_fail(e, "linear_fused_backward: workspace");
        workspace = own;
    }
    const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(dy);
    int64_t ldg = lddy;
    qkn_status st = QKN_OK;
    if (has_z || dbias != nullptr) {
        __nv_bfloat16 *dz = static_cast<__nv_bfloat16 *>(workspace);
        float *part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + lin::dz_bytes(M, N, act));
        const __nv_bfloat16 *z = static_cast<const __nv_bfloat16 *>(preact);
        switch (act) {
        case QKN_ACT_RELU: st = lin::launch_dz<QKN_ACT_RELU>(g, z, dz, part, dbias, M, N, lddy, ldz, s); break;
        case QKN_ACT_SILU: st = lin::launch_dz<QKN_ACT_SILU>(g, z, dz, part, dbias, M, N, lddy, ldz, s); break;
        case QKN_ACT_GELU: st = lin::launch_dz<QKN_ACT_GELU>(g, z, dz, part, dbias, M, N, lddy, ldz, s); break;
        case QKN_ACT_GELU_TANH: st = lin::launch_dz<QKN_ACT_GELU_TANH>(g, z, dz, part, dbias, M, N, lddy, ldz, s); break;
        default: st = lin::launch_dz<QKN_ACT_NONE>(g, z, dz, part, dbias, M, N, lddy, ldz, s);
        }
        if (has_z) {
            g = dz;
            ldg = N;
        }
    }
    const lin::pair::Matrix mg = {g, M, N, ldg}, mx = {x, M, K, ldx}, mw = {W, N, K, ldw};
    const lin::Epilogue e{};
    if (st == QKN_OK && dx != nullptr) {
        const lin::pair::Matrix out = {dx, M, K, lddx};
        st = lin::product<false, true, QKN_ACT_NONE>(mg, mw, out, nullptr, nullptr, e, N, s);
    }
    if (st == QKN_OK && dW != nullptr) {
        const lin::pair::Matrix out = {dW, N, K, lddw};
        st = lin::product<true, true, QKN_ACT_NONE>(mg, mx, out, nullptr, nullptr, e, M, s);
    }
    if (own != nullptr) {
        const cudaError_t f = cudaFreeAsync(own, s);
        if (f != cudaSuccess && st == QKN_OK) st = cuda_fail(f, "linear_fused_backward: releasing the workspace");
    }
    return st;
}
