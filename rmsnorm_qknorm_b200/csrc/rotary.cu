// Rotary positions on query and key rows, alone or after QK-Norm in the same
// pass, and the gradients of the two.
//
// Row t has position p_t.  In every head of D elements the first r are
// rotated as r / 2 pairs; pair i turns by theta = p_t * f_i:
//   c = m cos(theta), s = m sin(theta)
//   y_a = x_a c - x_b s,  y_b = x_b c + x_a s       (inverse: s -> -s)
// with (a, b) = (i, i + r/2) in the half layout and (2i, 2i + 1) in the
// interleaved one; elements r .. D - 1 are copied.  With QK-Norm x is
// n = (x * rsqrt(mean(x^2) + eps)) * w over the FULL row, unrounded.
// Gradients for dy, with R the (linear) rotation and inv the row's factor:
//   g = R^T dy,  dw = sum_rows g x inv,
//   dx = inv (w g - x inv^2 mean(w g x))
// Sums and statistics are fp32; each output is rounded once.
//
// The angle is formed in fp64 as turns, p_t * (f_i / 2 pi), of which only the
// fraction is kept: three roundings (1 / 2 pi, f / 2 pi and the product), an
// error of 3 x 2^-53 of the angle, below fp32 resolution up to 10^8 radians,
// where an fp32 angle is off by 0.06 rad at position 10^6.  The fraction, half
// a turn at most, is rounded to fp32 for sincospif (pi 2^-25 rad at most), one
// rounding like those of the fp32 products behind it and far below bf16's 2^-8:
// fp32 rows are off by 5.5 x 10^-8 of their norm, 4.2 x 10^-8 with cos and sin
// taken in fp64.
#include <atomic>
#include <math.h>

#include "qkn_common.cuh"
#include "qkn_sync.cuh"

namespace qkn {
namespace rot {

constexpr int kMaxRotary = 1024;      // rotated elements per head at most (the cos / sin table of a row)
constexpr int kBlock = 256;
constexpr int64_t kMaxWidth = 0x3ffffff0;  // of a row: columns of q and k, rounded up to blocks of 32, stay below 2^31

// One tensor of the call: query or key rows.
struct Job {
    const uint8_t *x;      // rows (the rows to rotate; for gradients the rows that were normalised)
    const uint8_t *g;      // gradients of the outputs (gradients only)
    uint8_t *y;            // results
    const void *w;         // norm weights [d] (unused without the norm)
    float *dw;             // gradients of the weights [d]
    int64_t ldx, ldg, ldy; // pitches in bytes
    int d;
};

struct Args {
    Job job[2];
    int njobs;
    int64_t T;
    int D, r;              // head width, rotated elements (r == 0: no rotation)
    int layout;            // qkn_rotary_layout
    const void *pos;
    int pos64;             // positions are int64 (else int32)
    const double *freq;    // [r / 2]
    float mscale, sign;    // sign of the sine: -1 rotates back
    float eps;
    float *part;           // gradients: [slices][dq + dk] partial weight gradients
    float *inv;            // gradients, element-wise kernel: [njobs][T] row factors
    int slices;
};

__device__ __forceinline__ Job pick(const Args &a, int which) {
    const Job &p = a.job[0], &q = a.job[1];
    Job J;
    J.x = which ? q.x : p.x;
    J.g = which ? q.g : p.g;
    J.y = which ? q.y : p.y;
    J.w = which ? q.w : p.w;
    J.dw = which ? q.dw : p.dw;
    J.ldx = which ? q.ldx : p.ldx;
    J.ldg = which ? q.ldg : p.ldg;
    J.ldy = which ? q.ldy : p.ldy;
    J.d = which ? q.d : p.d;
    return J;
}

__device__ __forceinline__ int64_t position(const Args &a, int64_t row) {
    return a.pos64 ? __ldg(static_cast<const long long *>(a.pos) + row)
                   : (int64_t)__ldg(static_cast<const int *>(a.pos) + row);
}

constexpr double kInvTwoPi = 0.15915494309189533576888;  // 1 / (2 pi)

// c and s of one pair at one position.  turns = f / (2 pi).
__device__ __forceinline__ void cos_sin(int64_t p, double turns, float mscale, float sign, float &c, float &s) {
    const double t = (double)p * turns;
    const float half_turns = (float)(2.0 * (t - rint(t)));
    sincospif(half_turns, &s, &c);
    c *= mscale;
    s *= mscale * sign;
}

// Sum over the block, the same on every thread; red holds 2 x 8 floats.
__device__ __forceinline__ float2 block_sum2(float2 v, float *red) {
    for (int off = 16; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        red[threadIdx.x >> 5] = v.x;
        red[8 + (threadIdx.x >> 5)] = v.y;
    }
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) {
        s.x += red[w];
        s.y += red[8 + w];
    }
    return s;
}

// An item of a row: a rotated pair (elements ia, ib, table entry f) or a
// single copied element (ia, f < 0).  A head holds D - r / 2 items.
struct Item { int ia, ib, f; };
__device__ __forceinline__ Item item(int i, int D, int r, int layout) {
    const int half = r >> 1, per = D - half;
    const int h = i / per, p = i - h * per;
    Item t;
    if (p < half) {
        t.f = p;
        t.ia = h * D + (layout == QKN_ROTARY_HALF ? p : 2 * p);
        t.ib = layout == QKN_ROTARY_HALF ? t.ia + half : t.ia + 1;
    } else {
        t.f = -1;
        t.ia = t.ib = h * D + p + half;
    }
    return t;
}

enum Mode { kRotate, kNorm, kNormBack };

// Element-wise kernel, any width, alignment and pitch: one block per row at a
// time, an item per thread and step.  It serves rows the unit kernel does not
// take; each row is read twice with the norm (the second time from L2).
template <typename TA, typename TW, int MODE>
__global__ void __launch_bounds__(kBlock) rotary_scalar_kernel(const Args a) {
    __shared__ float2 table[kMaxRotary / 2];
    __shared__ float red[16];
    const int64_t total = a.T * a.njobs;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int which = b >= a.T ? 1 : 0;
        const int64_t row = which ? b - a.T : b;
        const Job J = pick(a, which);
        const TA *x = reinterpret_cast<const TA *>(J.x + row * J.ldx);
        const TA *g = reinterpret_cast<const TA *>(J.g + row * J.ldg);
        TA *y = reinterpret_cast<TA *>(J.y + row * J.ldy);
        const TW *w = static_cast<const TW *>(J.w);
        const int D = a.r ? a.D : J.d;
        const int items = J.d / D * (D - (a.r >> 1));
        __syncthreads();  // the previous row's table has been read
        if (a.r) {
            const int64_t p = position(a, row);
            for (int f = threadIdx.x; f < (a.r >> 1); f += kBlock) {
                float c, s;
                cos_sin(p, __ldg(a.freq + f) * kInvTwoPi, a.mscale, a.sign, c, s);
                table[f] = make_float2(c, s);
            }
        }
        __syncthreads();
        float inv = 1.f, coef = 0.f;
        if constexpr (MODE != kRotate) {
            float2 acc = make_float2(0.f, 0.f);  // sum x^2, sum w g x
            for (int i = threadIdx.x; i < items; i += kBlock) {
                const Item t = item(i, D, a.r, a.layout);
                const float xa = to_f32<TA>(x[t.ia]), xb = t.f >= 0 ? to_f32<TA>(x[t.ib]) : 0.f;
                acc.x = fmaf(xa, xa, fmaf(xb, xb, acc.x));
                if constexpr (MODE == kNormBack) {
                    float ga = to_f32<TA>(g[t.ia]), gb = 0.f;
                    if (t.f >= 0) {
                        const float2 cs = table[t.f];
                        const float da = ga, db = to_f32<TA>(g[t.ib]);
                        ga = da * cs.x - db * cs.y;
                        gb = db * cs.x + da * cs.y;
                        acc.y = fmaf(xb * gb, to_f32<TW>(w[t.ib]), acc.y);
                    }
                    acc.y = fmaf(xa * ga, to_f32<TW>(w[t.ia]), acc.y);
                }
            }
            acc = block_sum2(acc, red);
            inv = rsqrtf(acc.x / (float)J.d + a.eps);
            coef = inv * inv * (acc.y / (float)J.d);
            if (MODE == kNormBack && threadIdx.x == 0) a.inv[b] = inv;
        }
        for (int i = threadIdx.x; i < items; i += kBlock) {
            const Item t = item(i, D, a.r, a.layout);
            const TA *src = MODE == kNormBack ? g : x;
            float va = to_f32<TA>(src[t.ia]), vb = t.f >= 0 ? to_f32<TA>(src[t.ib]) : 0.f;
            if constexpr (MODE == kNorm) {
                va = (va * inv) * to_f32<TW>(w[t.ia]);
                if (t.f >= 0) vb = (vb * inv) * to_f32<TW>(w[t.ib]);
            }
            if (t.f >= 0) {
                const float2 cs = table[t.f];
                const float ra = va * cs.x - vb * cs.y, rb = vb * cs.x + va * cs.y;
                va = ra;
                vb = rb;
            }
            if constexpr (MODE == kNormBack) {
                va = inv * (to_f32<TW>(w[t.ia]) * va - to_f32<TA>(x[t.ia]) * coef);
                if (t.f >= 0) vb = inv * (to_f32<TW>(w[t.ib]) * vb - to_f32<TA>(x[t.ib]) * coef);
            }
            y[t.ia] = from_f32<TA>(va);
            if (t.f >= 0) y[t.ib] = from_f32<TA>(vb);
        }
    }
}

// Weight gradients beside rotary_scalar_kernel<kNormBack>: a thread owns an
// item's columns and walks the rows of its slice in order; blockIdx.y is the
// slice, blockIdx.z the tensor.  The partial sums go to part[slice][column].
// x and g are read again here, after the kernel above wrote dx: dx must not
// overlap them.
template <typename TA, typename TW>
__global__ void __launch_bounds__(kBlock) rotary_scalar_dw_kernel(const Args a) {
    const int which = blockIdx.z;
    const Job J = pick(a, which);
    const int D = a.r ? a.D : J.d;
    const int items = J.d / D * (D - (a.r >> 1));
    const int i = blockIdx.x * kBlock + threadIdx.x;
    if (i >= items) return;
    const Item t = item(i, D, a.r, a.layout);
    const double turns = t.f >= 0 ? __ldg(a.freq + t.f) * kInvTwoPi : 0.0;
    float da = 0.f, db = 0.f;
    for (int64_t row = blockIdx.y; row < a.T; row += a.slices) {
        const TA *x = reinterpret_cast<const TA *>(J.x + row * J.ldx);
        const TA *g = reinterpret_cast<const TA *>(J.g + row * J.ldg);
        const float inv = a.inv[(int64_t)which * a.T + row];
        float ga = to_f32<TA>(g[t.ia]);
        if (t.f >= 0) {
            const float gb = to_f32<TA>(g[t.ib]);
            float c, s;
            cos_sin(position(a, row), turns, a.mscale, a.sign, c, s);
            const float ra = ga * c - gb * s, rb = gb * c + ga * s;
            ga = ra;
            db = fmaf(rb, to_f32<TA>(x[t.ib]) * inv, db);
        }
        da = fmaf(ga, to_f32<TA>(x[t.ia]) * inv, da);
    }
    float *part = a.part + (int64_t)blockIdx.y * (a.job[0].d + (a.njobs > 1 ? a.job[1].d : 0)) + (which ? a.job[0].d : 0);
    part[t.ia] = da;
    if (t.f >= 0) part[t.ib] = db;
}

// dw[c] = sum over slices of part[slice][c], in a fixed order: 8 threads take
// every 8th slice of a column, their sums are added in thread order.
__global__ void __launch_bounds__(kBlock) dw_reduce_kernel(const float *__restrict__ part, float *__restrict__ dwq,
                                                           float *__restrict__ dwk, int dq, int dk, int slices) {
    __shared__ float red[8][33];
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    const int d = dq + dk;
    // launched as a programmatic dependent: its blocks may start while the partial sums are formed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    if (col < d)
#pragma unroll 4
        for (int i = k; i < slices; i += 8) s += part[(int64_t)i * d + col];
    red[k][threadIdx.x & 31] = s;
    __syncthreads();
    if (k == 0 && col < d) {
        float v = red[0][threadIdx.x];
#pragma unroll
        for (int j = 1; j < 8; ++j) v += red[j][threadIdx.x];
        if (col < dq) dwq[col] = v;
        else dwk[col - dq] = v;
    }
}

}  // namespace rot
}  // namespace qkn

#include "rotary_rows.cuh"

namespace qkn {
namespace rot {

// ---------------------------------------------------------------- host side

constexpr int kScalarSlices = 64;

qkn_status launch_dw_reduce(const Args &a, int slices, cudaStream_t s) {
    const int dq = a.job[0].d, dk = a.njobs > 1 ? a.job[1].d : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((dq + dk + 31) / 32), 1, 1);
    cfg.blockDim = dim3(kBlock, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dw_reduce_kernel, (const float *)a.part, a.job[0].dw, a.job[1].dw, dq, dk,
                                             slices);
    if (e != cudaSuccess) return cuda_fail(e, "dw_reduce_kernel launch");
    return check_launch("dw_reduce_kernel launch");
}

template <typename TA, typename TW, int MODE>
qkn_status launch_scalar(Args &a, cudaStream_t s) {
    const int64_t total = a.T * a.njobs, cap = 8 * (int64_t)sm_count();
    rotary_scalar_kernel<TA, TW, MODE><<<(unsigned)(total < cap ? total : cap), kBlock, 0, s>>>(a);
    if (qkn_status st = check_launch("rotary_scalar_kernel launch")) return st;
    if constexpr (MODE == kNormBack) {
        a.slices = (int)(a.T < kScalarSlices ? a.T : kScalarSlices);
        const int dq = a.job[0].d, dk = a.njobs > 1 ? a.job[1].d : 0;
        const int widest = dq > dk ? dq : dk;
        const dim3 grid((unsigned)((widest + kBlock - 1) / kBlock), (unsigned)a.slices, (unsigned)a.njobs);
        rotary_scalar_dw_kernel<TA, TW><<<grid, kBlock, 0, s>>>(a);
        if (qkn_status st = check_launch("rotary_scalar_dw_kernel launch")) return st;
        return launch_dw_reduce(a, a.slices, s);
    }
    return QKN_OK;
}

template <typename TA, typename TW, int MODE>
qkn_status launch(Args &a, cudaStream_t s) {
    bool taken = false;
    int grid = 0;
    const qkn_status st = unit::launch<TA, TW, MODE>(a, &taken, &grid, s);
    if (st != QKN_OK) return st;
    if (taken) return MODE == kNormBack ? launch_dw_reduce(a, grid, s) : QKN_OK;
    return launch_scalar<TA, TW, MODE>(a, s);
}

template <int MODE>
qkn_status launch_types(Args &a, qkn_dtype act, qkn_dtype wdt, cudaStream_t s) {
    if constexpr (MODE == kRotate) {
        return act == QKN_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, MODE>(a, s) : launch<float, float, MODE>(a, s);
    } else {
        if (act == QKN_BF16)
            return wdt == QKN_BF16 ? launch<__nv_bfloat16, __nv_bfloat16, MODE>(a, s)
                                   : launch<__nv_bfloat16, float, MODE>(a, s);
        return wdt == QKN_BF16 ? launch<float, __nv_bfloat16, MODE>(a, s) : launch<float, float, MODE>(a, s);
    }
}

// The checks the three entry points share; fills what they have in common.
qkn_status check_rotary(const char *fn, int64_t T, int64_t dq, int64_t dk, int64_t head_dim, int64_t rotary_dim,
                        int pos_bits, int layout, float mscale, qkn_dtype act, qkn_dtype wdt) {
    if (!valid_dtype(act) || !valid_dtype(wdt))
        return fail(QKN_ERR_DTYPE, "%s: unknown dtype (act=%d, wdt=%d)", fn, (int)act, (int)wdt);
    if (T < 0 || dq < 1 || dk < 0 || dq > kMaxWidth || dk > kMaxWidth || T > 0x7fffffffLL)
        return fail(QKN_ERR_SHAPE, "%s: bad sizes T=%lld dq=%lld dk=%lld", fn, (long long)T, (long long)dq,
                    (long long)dk);
    if (rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > kMaxRotary)
        return fail(QKN_ERR_SHAPE, "%s: rotary_dim=%lld must be even and at most %d", fn, (long long)rotary_dim,
                    kMaxRotary);
    if (rotary_dim > 0) {
        if (head_dim < rotary_dim || dq % head_dim != 0 || dk % head_dim != 0)
            return fail(QKN_ERR_SHAPE,
                        "%s: head_dim=%lld must be at least rotary_dim=%lld and divide dq=%lld and dk=%lld", fn,
                        (long long)head_dim, (long long)rotary_dim, (long long)dq, (long long)dk);
        if (layout != QKN_ROTARY_HALF && layout != QKN_ROTARY_INTERLEAVED)
            return fail(QKN_ERR_UNSUPPORTED, "%s: unknown layout %d", fn, layout);
        if (pos_bits != 32 && pos_bits != 64)
            return fail(QKN_ERR_DTYPE, "%s: positions are 32- or 64-bit integers (pos_bits=%d)", fn, pos_bits);
        if (!(fabsf(mscale) <= 3.4e38f)) return fail(QKN_ERR_SHAPE, "%s: mscale must be finite", fn);
    }
    return QKN_OK;
}

void fill(Args &a, int64_t T, int64_t head_dim, const void *positions, int pos_bits, const double *inv_freq,
          int64_t rotary_dim, int layout, float mscale, bool inverse, float eps) {
    a.T = T;
    a.D = (int)head_dim;
    a.r = (int)rotary_dim;
    a.layout = layout;
    a.pos = positions;
    a.pos64 = pos_bits == 64;
    a.freq = inv_freq;
    a.mscale = mscale;
    a.sign = inverse ? -1.f : 1.f;
    a.eps = eps;
}

qkn_status check_rotary_pointers(const char *fn, const void *positions, int pos_bits, const double *inv_freq,
                                 int64_t rotary_dim) {
    if (rotary_dim == 0) return QKN_OK;
    if (positions == nullptr || inv_freq == nullptr)
        return fail(QKN_ERR_NULL, "%s: positions and inv_freq are required", fn);
    if (!aligned(positions, pos_bits / 8) || !aligned(inv_freq, 8))
        return fail(QKN_ERR_ALIGN, "%s: positions and inv_freq must be aligned to their element size", fn);
    return QKN_OK;
}

// The results are the operand's own rows (in place) or rows that share nothing with any operand,
// and not one another's: rows are read ahead of the ones that are written.  Nor do they share anything
// with the weights (of ws bytes), positions and frequencies, which other blocks may read later, or
// with the workspace.
qkn_status check_rotary_rows(const char *fn, const Args &a, int64_t es, int64_t ws, bool inplace,
                             const void *workspace = nullptr, size_t workspace_bytes = 0) {
    const Span pos = flat(a.r ? a.pos : nullptr, a.T * (a.pos64 ? 8 : 4)), freq = flat(a.r ? a.freq : nullptr, a.r / 2 * 8);
    const Span scratch = flat(workspace, (int64_t)workspace_bytes);
    if (rows_overlap(scratch, pos) || rows_overlap(scratch, freq))
        return fail(QKN_ERR_UNSUPPORTED, "%s: the workspace shares memory with an input", fn);
    for (int i = 0; i < a.njobs; ++i) {
        const Job &j = a.job[i];
        const Span y = {j.y, a.T, j.d * es, j.ldy};
        for (int o = 0; o < a.njobs; ++o) {
            const Job &k = a.job[o];
            const Span x = {k.x, a.T, k.d * es, k.ldx}, g = {k.g, a.T, k.d * es, k.ldg}, z = {k.y, a.T, k.d * es, k.ldy};
            if ((rows_overlap(y, x) && !(inplace && o == i && same_rows(y, x))) || rows_overlap(y, g) ||
                (o > i && rows_overlap(y, z)))
                return fail(QKN_ERR_UNSUPPORTED, "%s: a result shares memory with an input or the other result", fn);
            const Span w = flat(j.dw, 4 * (int64_t)j.d), v = flat(k.dw, 4 * (int64_t)k.d);  // of gradients
            if (rows_overlap(w, x) || rows_overlap(w, g) || rows_overlap(w, z) || (o > i && rows_overlap(w, v)))
                return fail(QKN_ERR_UNSUPPORTED, "%s: the gradient of weights shares memory with rows or the other's", fn);
            const Span norm = flat(k.w, k.d * ws);
            if (rows_overlap(y, norm) || rows_overlap(w, norm))
                return fail(QKN_ERR_UNSUPPORTED, "%s: a result shares memory with weights", fn);
            if (rows_overlap(scratch, x) || rows_overlap(scratch, g) || rows_overlap(scratch, z) ||
                rows_overlap(scratch, v) || rows_overlap(scratch, norm))
                return fail(QKN_ERR_UNSUPPORTED, "%s: the workspace shares memory with an input or a result", fn);
        }
        const Span w = flat(j.dw, 4 * (int64_t)j.d);
        if (rows_overlap(y, pos) || rows_overlap(y, freq) || rows_overlap(w, pos) || rows_overlap(w, freq))
            return fail(QKN_ERR_UNSUPPORTED, "%s: a result shares memory with positions or frequencies", fn);
    }
    return QKN_OK;
}

}  // namespace rot
}  // namespace qkn

using namespace qkn;

extern "C" QKN_API qkn_status rotary_apply(const void *q, const void *k, void *q_out, void *k_out, int64_t T,
                                           int64_t dq, int64_t dk, int64_t ldq, int64_t ldk, int64_t ldq_out,
                                           int64_t ldk_out, int64_t head_dim, const void *positions, int pos_bits,
                                           const double *inv_freq, int64_t rotary_dim, qkn_rotary_layout layout,
                                           float mscale, int inverse, qkn_dtype act, void *stream) {
    const char *fn = "rotary_apply";
    if (qkn_status st = rot::check_rotary(fn, T, dq, dk, head_dim, rotary_dim, pos_bits, (int)layout, mscale, act, act))
        return st;
    if (rotary_dim < 2) return fail(QKN_ERR_SHAPE, "%s: rotary_dim must be at least 2", fn);
    const bool has_k = dk > 0;
    if (ldq < dq || (has_k && ldk < dk) || (q_out && ldq_out < dq) || (has_k && k_out && ldk_out < dk))
        return fail(QKN_ERR_SHAPE, "%s: leading dimension smaller than the row width", fn);
    if (T == 0) return QKN_OK;
    if (q == nullptr || (has_k && k == nullptr)) return fail(QKN_ERR_NULL, "%s: q (and k when dk > 0) are required", fn);
    if (qkn_status st = rot::check_rotary_pointers(fn, positions, pos_bits, inv_freq, rotary_dim)) return st;
    const size_t es = dtype_size(act);
    if (!aligned(q, es) || (q_out && !aligned(q_out, es)) || (has_k && (!aligned(k, es) || (k_out && !aligned(k_out, es)))))
        return fail(QKN_ERR_ALIGN, "%s: pointers must be aligned to their element size", fn);
    rot::Args a{};
    rot::fill(a, T, head_dim, positions, pos_bits, inv_freq, rotary_dim, (int)layout, mscale, inverse != 0, 0.f);
    const int64_t e = (int64_t)es;
    a.job[0] = {static_cast<const uint8_t *>(q), nullptr, static_cast<uint8_t *>(q_out ? q_out : const_cast<void *>(q)),
                nullptr, nullptr, ldq * e, 0, (q_out ? ldq_out : ldq) * e, (int)dq};
    a.job[1] = {static_cast<const uint8_t *>(k), nullptr, static_cast<uint8_t *>(k_out ? k_out : const_cast<void *>(k)),
                nullptr, nullptr, ldk * e, 0, (k_out ? ldk_out : ldk) * e, (int)dk};
    a.njobs = has_k ? 2 : 1;
    if (qkn_status st = rot::check_rotary_rows(fn, a, e, e, true)) return st;
    return rot::launch_types<rot::kRotate>(a, act, act, static_cast<cudaStream_t>(stream));
}

extern "C" QKN_API qkn_status qknorm_rotary(const void *q, const void *k, const void *wq, const void *wk, void *q_out,
                                            void *k_out, int64_t T, int64_t dq, int64_t dk, int64_t ldq, int64_t ldk,
                                            int64_t ldq_out, int64_t ldk_out, int64_t head_dim, const void *positions,
                                            int pos_bits, const double *inv_freq, int64_t rotary_dim,
                                            qkn_rotary_layout layout, float mscale, qkn_dtype act, qkn_dtype wdt,
                                            float eps, void *stream) {
    const char *fn = "qknorm_rotary";
    if (qkn_status st = rot::check_rotary(fn, T, dq, dk, head_dim, rotary_dim, pos_bits, (int)layout, mscale, act, wdt))
        return st;
    const bool has_k = dk > 0;
    if (ldq < dq || (has_k && ldk < dk) || (q_out && ldq_out < dq) || (has_k && k_out && ldk_out < dk))
        return fail(QKN_ERR_SHAPE, "%s: leading dimension smaller than the row width", fn);
    if (!(eps >= 0.f) || isinf(eps)) return fail(QKN_ERR_EPS, "%s: eps must be finite and >= 0", fn);
    if (T == 0) return QKN_OK;
    if (q == nullptr || wq == nullptr || (has_k && (k == nullptr || wk == nullptr)))
        return fail(QKN_ERR_NULL, "%s: q and wq (and k and wk when dk > 0) are required", fn);
    if (qkn_status st = rot::check_rotary_pointers(fn, positions, pos_bits, inv_freq, rotary_dim)) return st;
    const size_t es = dtype_size(act), ws = dtype_size(wdt);
    if (!aligned(q, es) || !aligned(wq, ws) || (q_out && !aligned(q_out, es)) ||
        (has_k && (!aligned(k, es) || !aligned(wk, ws) || (k_out && !aligned(k_out, es)))))
        return fail(QKN_ERR_ALIGN, "%s: pointers must be aligned to their element size", fn);
    rot::Args a{};
    rot::fill(a, T, head_dim, positions, pos_bits, inv_freq, rotary_dim, (int)layout, mscale, false, eps);
    const int64_t e = (int64_t)es;
    a.job[0] = {static_cast<const uint8_t *>(q), nullptr, static_cast<uint8_t *>(q_out ? q_out : const_cast<void *>(q)),
                wq, nullptr, ldq * e, 0, (q_out ? ldq_out : ldq) * e, (int)dq};
    a.job[1] = {static_cast<const uint8_t *>(k), nullptr, static_cast<uint8_t *>(k_out ? k_out : const_cast<void *>(k)),
                wk, nullptr, ldk * e, 0, (k_out ? ldk_out : ldk) * e, (int)dk};
    a.njobs = has_k ? 2 : 1;
    if (qkn_status st = rot::check_rotary_rows(fn, a, e, (int64_t)dtype_size(wdt), true)) return st;
    return rot::launch_types<rot::kNorm>(a, act, wdt, static_cast<cudaStream_t>(stream));
}

extern "C" QKN_API size_t qknorm_rotary_backward_workspace_bytes(int64_t T, int64_t dq, int64_t dk) {
    if (T < 0 || dq < 1 || dk < 0 || dq > rot::kMaxWidth || dk > rot::kMaxWidth || T > 0x7fffffffLL) return 0;
    // row factors of both tensors (element-wise kernels), then rows of partial sums: one per
    // slice of the element-wise kernel or per block of the unit kernel
    const size_t inv = ((size_t)T * 2 * 4 + 255) / 256 * 256;
    const size_t blocks = (size_t)sm_count();
    const size_t parts = blocks > (size_t)rot::kScalarSlices ? blocks : (size_t)rot::kScalarSlices;
    return inv + ((size_t)T < parts ? (size_t)T : parts) * (size_t)(dq + dk) * 4;
}

extern "C" QKN_API qkn_status qknorm_rotary_backward(
    const void *dq_out, const void *dk_out, const void *q, const void *k, const void *wq, const void *wk, void *dq_in,
    void *dk_in, float *dwq, float *dwk, int64_t T, int64_t dq, int64_t dk, int64_t ldgq, int64_t ldgk, int64_t ldq,
    int64_t ldk, int64_t lddq, int64_t lddk, int64_t head_dim, const void *positions, int pos_bits,
    const double *inv_freq, int64_t rotary_dim, qkn_rotary_layout layout, float mscale, qkn_dtype act, qkn_dtype wdt,
    float eps, void *workspace, size_t workspace_bytes, void *stream) {
    const char *fn = "qknorm_rotary_backward";
    if (qkn_status st = rot::check_rotary(fn, T, dq, dk, head_dim, rotary_dim, pos_bits, (int)layout, mscale, act, wdt))
        return st;
    const bool has_k = dk > 0;
    if (ldq < dq || ldgq < dq || lddq < dq || (has_k && (ldk < dk || ldgk < dk || lddk < dk)))
        return fail(QKN_ERR_SHAPE, "%s: leading dimension smaller than the row width", fn);
    if (!(eps >= 0.f) || isinf(eps)) return fail(QKN_ERR_EPS, "%s: eps must be finite and >= 0", fn);
    if (dwq == nullptr || (has_k && dwk == nullptr))
        return fail(QKN_ERR_NULL, "%s: dwq (and dwk when dk > 0) are required", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!aligned(dwq, 4) || (has_k && !aligned(dwk, 4)))
        return fail(QKN_ERR_ALIGN, "%s: dwq and dwk must be 4-byte aligned", fn);
    if (T > 0) {
        if (q == nullptr || wq == nullptr || dq_out == nullptr || dq_in == nullptr ||
            (has_k && (k == nullptr || wk == nullptr || dk_out == nullptr || dk_in == nullptr)))
            return fail(QKN_ERR_NULL, "%s: the rows, their gradients, the weights and the results are required", fn);
        if (qkn_status st = rot::check_rotary_pointers(fn, positions, pos_bits, inv_freq, rotary_dim)) return st;
        const size_t es = dtype_size(act), ws = dtype_size(wdt);
        if (!aligned(q, es) || !aligned(dq_out, es) || !aligned(dq_in, es) || !aligned(wq, ws) ||
            (has_k && (!aligned(k, es) || !aligned(dk_out, es) || !aligned(dk_in, es) || !aligned(wk, ws))))
            return fail(QKN_ERR_ALIGN, "%s: pointers must be aligned to their element size", fn);
    }
    const size_t need = qknorm_rotary_backward_workspace_bytes(T, dq, dk);
    if (workspace != nullptr) {
        if (workspace_bytes < need)
            return fail(QKN_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
        if (!aligned(workspace, 16)) return fail(QKN_ERR_ALIGN, "%s: workspace must be 16-byte aligned", fn);
    }
    if (T == 0) {  // no rows: the weights' gradients are empty sums
        cudaError_t e = cudaMemsetAsync(dwq, 0, (size_t)dq * 4, s);
        if (e == cudaSuccess && has_k) e = cudaMemsetAsync(dwk, 0, (size_t)dk * 4, s);
        return e == cudaSuccess ? QKN_OK : cuda_fail(e, "qknorm_rotary_backward: clearing the weight gradients");
    }
    rot::Args a{};
    rot::fill(a, T, head_dim, positions, pos_bits, inv_freq, rotary_dim, (int)layout, mscale, true, eps);
    const int64_t e = (int64_t)dtype_size(act);
    a.job[0] = {static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(dq_out), static_cast<uint8_t *>(dq_in), wq,
                dwq, ldq * e, ldgq * e, lddq * e, (int)dq};
    a.job[1] = {static_cast<const uint8_t *>(k), static_cast<const uint8_t *>(dk_out), static_cast<uint8_t *>(dk_in), wk,
                dwk, ldk * e, ldgk * e, lddk * e, (int)dk};
    a.njobs = has_k ? 2 : 1;
    if (qkn_status st = rot::check_rotary_rows(fn, a, e, (int64_t)dtype_size(wdt), false, workspace, need)) return st;
    void *own = nullptr;
    if (workspace == nullptr) {
        const cudaError_t f = cudaMallocAsync(&own, need, s);
        if (f != cudaSuccess) return cuda_fail(f, "qknorm_rotary_backward: workspace");
        workspace = own;
    }
    a.inv = static_cast<float *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + ((size_t)T * 2 * 4 + 255) / 256 * 256);
    qkn_status st = rot::launch_types<rot::kNormBack>(a, act, wdt, s);
    if (own != nullptr) {
        const cudaError_t f = cudaFreeAsync(own, s);
        if (f != cudaSuccess && st == QKN_OK) st = cuda_fail(f, "qknorm_rotary_backward: releasing the workspace");
    }
    return st;
}
