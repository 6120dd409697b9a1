// Unit kernel of the rotary entry points: rows of 16-byte chunks, persistent,
// fed by bulk copies.
//
// Included by rotary.cu only (one translation unit: its device error word,
// Args and helpers).
//
// The work is all HBM: every row is read once and written once (gradients:
// x and dy read, dx written).  A token's rows (q and k together) are handled
// by a group of G + 1 warps; a block holds NG groups that never wait for one
// another.  Each group owns a ring of stages in shared memory, one token per
// stage.  The group's last warp is its producer: it fills a stage with 1-D
// bulk copies of the token's rows and, while they fly, forms the cos and sin
// of the token's angles into the stage's table, up to `stages` tokens ahead
// of the G consumer warps.  (With the table formed by the consumers between
// their loads and the row's barrier the fp64 angle and sincospif sat on every
// token's critical path.)
//
// A consumer thread owns the same columns of every token: UPT "units" of two
// 16-byte chunks, chunk j and chunk j + r / 2E of a head (E elements per
// chunk).  In the half layout the two chunks hold the two sides of E pairs;
// in the interleaved layout each holds E / 2 whole pairs.  Either way a unit
// needs the cos and sin of two runs of E / 2 frequencies, which the table
// keeps at positions j and j + r / 2E (filled in the order the layout asks
// for), so neighbouring threads read neighbouring 16-byte words.  Chunks
// behind the rotated part form units of their own, copied (or only
// normalised).  Fixed columns keep the weights' gradients in registers over
// all tokens; the weights are read from a copy in shared memory.
//
// With the norm, consumers meet at one barrier per token: before it they read
// their chunks, add up squares, multiply by the weights and park their warp's
// sums; after it they form the row's factor, turn, scale and store.  q and k
// have warps of their own (a group of one warp adds up both).  The sums are
// double-buffered by token, which one barrier per token makes safe.  The two
// halves of a packed fp32x2 operation round like scalar ones.
#pragma once

namespace qkn {

// Set by a bounded wait of the unit kernel that gave up (see qkn_check_device).
__device__ int g_rotary_error = 0;

namespace rot {
namespace unit {

constexpr int kMaxThreads = 512;
constexpr int kSmemLimit = 227 * 1024;

struct Rows {
    const uint8_t *x, *g;
    uint8_t *y;
    const void *w;
    int64_t ldx, ldg, ldy;   // pitches in bytes
    int d, row_bytes, row_off;  // row_off: of x in a stage; the gradient's is row_off + x_bytes
    int head_chunks, units_per_head, tail_chunks, tail_units;
    int nunits;
};

struct Params {
    Rows job[2];
    int njobs;
    int64_t T;
    int r, rot_units;        // rot_units: per head, r / 2E
    const void *pos;
    int pos64;
    const double *freq;
    float mscale, sign, eps;
    float *part;             // gradients: [gridDim.x][dq + dk]
    int warps, groups;       // consumer warps per group, groups per block
    int warps0;              // consumer warps of job 0 (== warps when one warp serves both jobs)
    int stages, stage_bytes, x_bytes;
    int w_bytes;             // the block's copy of the weights, in front of the rings
    uint64_t wait_ns;
};

constexpr int kMaxWarps = 15;  // consumer warps per group
constexpr int kSlots = 16;     // sums per tensor and token

inline __host__ __device__ int table_bytes(int r) { return (r * 4 + 15) / 16 * 16; }  // cos and sin of a token
// per group: tables, 2 tokens x (sum x^2, sum w g x) x kSlots sums, full and empty barriers
inline __host__ __device__ int group_fixed(int r, int stages) {
    return stages * table_bytes(r) + 4 * kSlots * 4 + stages * 16;
}

__device__ __forceinline__ Rows pick(const Params &a, int which) {
    const Rows &p = a.job[0], &q = a.job[1];
    Rows J;
    J.x = which ? q.x : p.x;
    J.g = which ? q.g : p.g;
    J.y = which ? q.y : p.y;
    J.w = which ? q.w : p.w;
    J.ldx = which ? q.ldx : p.ldx;
    J.ldg = which ? q.ldg : p.ldg;
    J.ldy = which ? q.ldy : p.ldy;
    J.d = which ? q.d : p.d;
    J.row_bytes = which ? q.row_bytes : p.row_bytes;
    J.row_off = which ? q.row_off : p.row_off;
    J.head_chunks = which ? q.head_chunks : p.head_chunks;
    J.units_per_head = which ? q.units_per_head : p.units_per_head;
    J.tail_chunks = which ? q.tail_chunks : p.tail_chunks;
    J.tail_units = which ? q.tail_units : p.tail_units;
    J.nunits = which ? q.nunits : p.nunits;
    return J;
}

// Barrier of a group's consumers, true on every thread when any of them failed.
__device__ __forceinline__ bool group_sync_or(bool failed, int group, int warps) {
    if (warps == 1) {
        const bool any = __any_sync(0xffffffffu, failed);
        __syncwarp();
        return any;
    }
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
                 "barrier.cta.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"(group + 1), "r"(warps * 32), "r"((uint32_t)failed) : "memory");
    return r != 0;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// A 16-byte chunk as E / 2 pairs of fp32.
template <typename TA, int H> __device__ __forceinline__ void unpack2(const uint4 &v, float2 (&f)[H]) {
    if constexpr (sizeof(TA) == 4) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    } else {
        f[0] = make_float2(bf16lo(v.x), bf16hi(v.x));
        f[1] = make_float2(bf16lo(v.y), bf16hi(v.y));
        f[2] = make_float2(bf16lo(v.z), bf16hi(v.z));
        f[3] = make_float2(bf16lo(v.w), bf16hi(v.w));
    }
}
template <typename TA, int H> __device__ __forceinline__ uint4 pack2(const float2 (&f)[H]) {
    if constexpr (sizeof(TA) == 4)
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
    else
        return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y),
                          pack_bf16x2(f[3].x, f[3].y));
}

// H = E / 2 consecutive floats of the table, as pairs.
template <int H>
__device__ __forceinline__ void lds_run(uint32_t addr, float2 (&f)[H / 2]) {
    if constexpr (H == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(f[0].x), "=f"(f[0].y), "=f"(f[1].x), "=f"(f[1].y) : "r"(addr));
    else
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[0].x), "=f"(f[0].y) : "r"(addr));
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The two chunks of a unit, turned and (SCALE) multiplied by inv.
template <int H, bool HALF, bool SCALE>
__device__ __forceinline__ void turn(float2 (&a)[H], float2 (&b)[H], uint32_t cos_addr, uint32_t run, uint32_t sin_off,
                                     float inv) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float2 c[H / 2], s[H / 2];
        lds_run<H>(cos_addr + (q ? run : 0u), c);
        lds_run<H>(cos_addr + sin_off + (q ? run : 0u), s);
        if constexpr (HALF) {
#pragma unroll
            for (int p = 0; p < H / 2; ++p) {
                const int i = q * (H / 2) + p;
                const float2 x = a[i], y = b[i];
                const float2 xc = __fmul2_rn(x, c[p]), ys = __fmul2_rn(y, s[p]), yc = __fmul2_rn(y, c[p]);
                if constexpr (SCALE) {
                    a[i] = __ffma2_rn(ys, both(-inv), __fmul2_rn(xc, both(inv)));
                    b[i] = __fmul2_rn(__ffma2_rn(x, s[p], yc), both(inv));
                } else {
                    a[i] = __ffma2_rn(ys, both(-1.f), xc);
                    b[i] = __ffma2_rn(x, s[p], yc);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const float ce = (e & 1) ? c[e >> 1].y : c[e >> 1].x, se = (e & 1) ? s[e >> 1].y : s[e >> 1].x;
                const float2 v = q ? b[e] : a[e];
                float2 t = make_float2(v.x * ce - v.y * se, v.y * ce + v.x * se);
                if constexpr (SCALE) t = __fmul2_rn(t, both(inv));
                if (q) b[e] = t;
                else a[e] = t;
            }
        }
    }
}

// The weights of a chunk from shared memory, as pairs.
template <typename TW, int H>
__device__ __forceinline__ void lds_weights(uint32_t addr, float2 (&f)[H]) {
    if constexpr (sizeof(TW) * 2 * H == 32) {  // fp32 weights of 8 elements
        const uint4 a = lds128(addr), b = lds128(addr + 16);
        f[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
        f[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
        f[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
        f[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    } else if constexpr (sizeof(TW) * 2 * H == 16) {
        unpack2<TW, H>(lds128(addr), f);
    } else {  // bf16 weights of 4 elements
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
        f[0] = make_float2(bf16lo(v.x), bf16hi(v.x));
        f[1] = make_float2(bf16lo(v.y), bf16hi(v.y));
    }
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// WIDE: groups of up to 15 consumer warps; otherwise up to 10, two blocks per SM where the registers allow.
template <bool WIDE> constexpr int max_threads() { return WIDE ? 32 * (kMaxWarps + 1) : 32 * 11; }
#ifndef ROT_MINB
#define ROT_MINB 2
#endif
#ifndef ROT_MINB_BACK
#define ROT_MINB_BACK 1
#endif

template <typename TA, typename TW, int MODE, int UPT, bool HALF, bool WIDE>
__global__ void __launch_bounds__(max_threads<WIDE>(), WIDE ? 1 : MODE == kNormBack ? ROT_MINB_BACK : ROT_MINB)
rotary_unit_kernel(const Params a) {
    constexpr int E = Chunk<TA>::E, H = E / 2;
    constexpr bool NORM = MODE != kRotate, BACK = MODE == kNormBack;
    extern __shared__ __align__(128) uint8_t smem[];
    const int gthreads = (a.warps + 1) * 32;
    const int group = threadIdx.x / gthreads, gt = threadIdx.x - group * gthreads;  // thread within its group
    const int lane = threadIdx.x & 31, gw = gt >> 5;
    uint8_t *rings = smem + a.w_bytes;
    uint8_t *fix_p = rings + (size_t)a.groups * a.stages * a.stage_bytes + (size_t)group * group_fixed(a.r, a.stages);
    const uint32_t ring = smem_u32(rings + (size_t)group * a.stages * a.stage_bytes);
    const int tbytes = table_bytes(a.r);
    float *red = reinterpret_cast<float *>(fix_p + (size_t)a.stages * tbytes);
    const uint32_t full = smem_u32(red + 4 * kSlots), empty = full + 8u * a.stages;
    const int64_t step = (int64_t)gridDim.x * a.groups;
    const int64_t first_token = (int64_t)blockIdx.x * a.groups + group;

    if (gt == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full + 8u * s, 2);         // the producer's two arrivals and the copies' bytes
            mbar_init(empty + 8u * s, a.warps);  // one per consumer warp
        }
        mbar_init_fence();
    }
    for (int i = gt; i < 4 * kSlots; i += gthreads) red[i] = 0.f;
    // the previous kernel on the stream has finished before any global memory is touched
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (NORM) {  // weights word by word, at the element positions of a stage's rows
        const int d0 = a.job[0].d, words = (int)sizeof(TW) * (d0 + a.job[1].d) / 4, words0 = (int)sizeof(TW) * d0 / 4;
        for (int i = threadIdx.x; i < words; i += blockDim.x)
            reinterpret_cast<uint32_t *>(smem)[i] = i < words0 ? __ldg(static_cast<const uint32_t *>(a.job[0].w) + i)
                                                               : __ldg(static_cast<const uint32_t *>(a.job[1].w) + i - words0);
    }
    __syncthreads();

    float2 da[UPT][H], db[UPT][H];  // gradients of the weights, over this group's tokens
    int off_a[UPT], off_b[UPT], tab[UPT];  // stage offsets of a unit's chunks (-1: none), table offset (-1: not turned)
    uint32_t is_k = 0;

    if (gw == a.warps) {
        // ---------------------------------------------------------------- producer warp
        const int nf = a.r >> 1;
        // frequency f sits in run f / H; the runs are placed in the layout's order
        auto place = [&](int f) {
            const int q = f / H;
            return (HALF ? (q & 1) * a.rot_units + (q >> 1) : q) * H + f % H;
        };
        double turns[2];
        int at[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            turns[i] = lane + 32 * i < nf ? __ldg(a.freq + lane + 32 * i) * kInvTwoPi : 0.0;
            at[i] = place(lane + 32 * i);
        }
        auto pos_at = [&](int64_t n) -> int64_t {
            if (a.r == 0 || n >= a.T) return 0;
            return a.pos64 ? __ldg(static_cast<const long long *>(a.pos) + n)
                           : (int64_t)__ldg(static_cast<const int *>(a.pos) + n);
        };
        int stage = 0;
        uint32_t phase = 0, issued = 0;
        int64_t p = pos_at(first_token);
        for (int64_t n = first_token; n < a.T; n += step) {
            bool ok = mbar_wait_fast(empty + 8u * stage, phase ^ 1u, &g_rotary_error, a.wait_ns);
            if (__any_sync(0xffffffffu, !ok)) break;
            const uint32_t bar = full + 8u * stage;
            if (lane == 0) {
                const uint32_t dst = ring + (uint32_t)(stage * a.stage_bytes);
                mbar_arrive_expect_tx(bar, (uint32_t)a.stage_bytes);
                bulk_g2s(dst, a.job[0].x + n * a.job[0].ldx, a.job[0].row_bytes, bar);
                if (BACK) bulk_g2s(dst + a.x_bytes, a.job[0].g + n * a.job[0].ldg, a.job[0].row_bytes, bar);
                if (a.njobs > 1) {
                    bulk_g2s(dst + a.job[1].row_off, a.job[1].x + n * a.job[1].ldx, a.job[1].row_bytes, bar);
                    if (BACK)
                        bulk_g2s(dst + a.x_bytes + a.job[1].row_off, a.job[1].g + n * a.job[1].ldg, a.job[1].row_bytes,
                                 bar);
                }
                issued |= 1u << stage;
            }
            const int64_t next = pos_at(n + step);
            float *t = reinterpret_cast<float *>(fix_p + (size_t)stage * tbytes);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i < nf) cos_sin(p, turns[i], a.mscale, a.sign, t[at[i]], t[nf + at[i]]);
            for (int f = lane + 64; f < nf; f += 32)
                cos_sin(p, __ldg(a.freq + f) * kInvTwoPi, a.mscale, a.sign, t[place(f)], t[nf + place(f)]);
            p = next;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // no copy may still be writing when the block exits: the last phase filled on every stage
        // (on the normal path the consumers have waited for them all already)
        if (lane == 0)
            for (int s = 0; s < a.stages; ++s)
                if (issued & (1u << s)) mbar_wait(full + 8u * s, s < stage ? phase : phase ^ 1u, &g_rotary_error, a.wait_ns);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- consumer warps
        const bool mixed = a.warps0 == a.warps && a.njobs > 1;  // one warp serves both jobs
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            int which = mixed ? 0 : (gw >= a.warps0 ? 1 : 0);
            const int jw = which ? a.warps - a.warps0 : a.warps0;
            int u = gt - (which ? a.warps0 * 32 : 0) + i * jw * 32;
            if (mixed && u >= a.job[0].nunits) {
                u -= a.job[0].nunits;
                which = 1;
            }
            off_a[i] = off_b[i] = tab[i] = -1;
            if (which) is_k |= 1u << i;
            if (u >= (which ? a.job[1].nunits : a.job[0].nunits)) continue;
            const Rows J = pick(a, which);
            const int h = u / J.units_per_head, j = u - h * J.units_per_head;
            const int first = h * J.head_chunks;
            if (j < a.rot_units) {
                off_a[i] = J.row_off + (first + j) * 16;
                off_b[i] = off_a[i] + a.rot_units * 16;
                tab[i] = j * H * 4;
            } else {
                const int t = j - a.rot_units;
                off_a[i] = J.row_off + (first + 2 * a.rot_units + t) * 16;
                if (t + J.tail_units < J.tail_chunks) off_b[i] = off_a[i] + J.tail_units * 16;
            }
        }
        const bool wk = !mixed && gw >= a.warps0;  // a warp of job 1 alone
        const uint32_t w_s = smem_u32(smem);
        // a chunk's weights: 16 bytes of elements are E weights
        auto weights = [&](int off, float2 (&f)[H]) { lds_weights<TW, H>(w_s + (uint32_t)(off / 16 * (E * (int)sizeof(TW))), f); };
        if constexpr (BACK) {
#pragma unroll
            for (int i = 0; i < UPT; ++i)
#pragma unroll
                for (int p = 0; p < H; ++p) da[i][p] = db[i][p] = make_float2(0.f, 0.f);
        }
        const uint32_t sin_off = (uint32_t)a.r * 2u, run = (uint32_t)a.rot_units * H * 4u;  // bytes
        const uint32_t tables = smem_u32(fix_p);
        const float dq = (float)a.job[0].d, dk = (float)a.job[1].d;

        int stage = 0, par = 0;
        uint32_t phase = 0;
        for (int64_t n = first_token; n < a.T; n += step) {
            const bool ok = mbar_wait_fast(full + 8u * stage, phase, &g_rotary_error, a.wait_ns);
            const uint32_t src = ring + (uint32_t)(stage * a.stage_bytes);
            const uint32_t tab_s = tables + (uint32_t)(stage * tbytes);
            float2 va[UPT][H], vb[UPT][H];  // x w (forward), x (gradients)
            float2 ga[UPT][H], gb[UPT][H];  // gradients turned back
            float2 sq[2] = {both(0.f), both(0.f)}, pg[2] = {both(0.f), both(0.f)};  // per job where mixed
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                const uint4 none = make_uint4(0u, 0u, 0u, 0u);
                unpack2<TA, H>(off_a[i] >= 0 ? lds128(src + off_a[i]) : none, va[i]);
                unpack2<TA, H>(off_b[i] >= 0 ? lds128(src + off_b[i]) : none, vb[i]);
                if constexpr (NORM) {
                    float2 q = both(0.f), r = both(0.f), w[H];
                    weights(off_a[i] >= 0 ? off_a[i] : 0, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) q = __ffma2_rn(va[i][p], va[i][p], q);
#pragma unroll
                    for (int p = 0; p < H; ++p) q = __ffma2_rn(vb[i][p], vb[i][p], q);
                    if constexpr (BACK) {
                        unpack2<TA, H>(off_a[i] >= 0 ? lds128(src + a.x_bytes + off_a[i]) : none, ga[i]);
                        unpack2<TA, H>(off_b[i] >= 0 ? lds128(src + a.x_bytes + off_b[i]) : none, gb[i]);
                        if (tab[i] >= 0) turn<H, HALF, false>(ga[i], gb[i], tab_s + tab[i], run, sin_off, 1.f);
#pragma unroll
                        for (int p = 0; p < H; ++p) r = __ffma2_rn(__fmul2_rn(va[i][p], ga[i][p]), w[p], r);
                        weights(off_b[i] >= 0 ? off_b[i] : 0, w);
#pragma unroll
                        for (int p = 0; p < H; ++p) r = __ffma2_rn(__fmul2_rn(vb[i][p], gb[i][p]), w[p], r);
                    } else {
#pragma unroll
                        for (int p = 0; p < H; ++p) va[i][p] = __fmul2_rn(va[i][p], w[p]);
                        weights(off_b[i] >= 0 ? off_b[i] : 0, w);
#pragma unroll
                        for (int p = 0; p < H; ++p) vb[i][p] = __fmul2_rn(vb[i][p], w[p]);
                    }
                    if (mixed && ((is_k >> i) & 1u)) {
                        sq[1] = __fadd2_rn(sq[1], q);
                        if (BACK) pg[1] = __fadd2_rn(pg[1], r);
                    } else {
                        sq[0] = __fadd2_rn(sq[0], q);
                        if (BACK) pg[0] = __fadd2_rn(pg[0], r);
                    }
                }
            }
            float inv_q = 1.f, inv_k = 1.f, cq = 0.f, ck = 0.f;
            bool failed = !ok;
            if constexpr (NORM) {
                float s0 = warp_sum(sq[0].x + sq[0].y), p0 = BACK ? warp_sum(pg[0].x + pg[0].y) : 0.f, s1 = 0.f, p1 = 0.f;
                if (mixed) {
                    s1 = warp_sum(sq[1].x + sq[1].y);
                    if (BACK) p1 = warp_sum(pg[1].x + pg[1].y);
                    failed = __any_sync(0xffffffffu, failed);
                } else {
                    // slots of this token: [x^2 | w g x][kSlots]; a job's warps only meet their own
                    float *slot = red + par * 2 * kSlots;
                    if (lane == 0) {
                        slot[gw] = s0;
                        if (BACK) slot[kSlots + gw] = p0;
                    }
                    failed = group_sync_or(failed, group, a.warps);
                    s0 = s1 = p0 = p1 = 0.f;
                    const int w0 = wk ? a.warps0 : 0, w1 = wk ? a.warps : a.warps0;
                    for (int w = w0; w < w1; ++w) s0 += slot[w];
                    if (BACK)
                        for (int w = w0; w < w1; ++w) p0 += slot[kSlots + w];
                    if (wk) {
                        s1 = s0;
                        p1 = p0;
                    }
                }
                inv_q = rsqrtf(s0 / dq + a.eps);
                inv_k = rsqrtf(s1 / dk + a.eps);
                if constexpr (BACK) {
                    cq = inv_q * inv_q * (p0 / dq);
                    ck = inv_k * inv_k * (p1 / dk);
                }
            } else {
                failed = __any_sync(0xffffffffu, failed);
            }
            if (failed) break;
            uint8_t *yq = a.job[0].y + n * a.job[0].ldy;
            uint8_t *yk = a.job[1].y + n * a.job[1].ldy - a.job[1].row_off;
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                const bool k = mixed ? (is_k >> i) & 1u : wk;
                const float inv = k ? inv_k : inv_q;
                if constexpr (BACK) {
                    const float2 nc = both(-(k ? ck : cq)), inv2 = both(inv);
                    float2 w[H];
                    weights(off_a[i] >= 0 ? off_a[i] : 0, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        da[i][p] = __ffma2_rn(ga[i][p], __fmul2_rn(va[i][p], inv2), da[i][p]);
                        va[i][p] = __fmul2_rn(inv2, __ffma2_rn(va[i][p], nc, __fmul2_rn(w[p], ga[i][p])));
                    }
                    weights(off_b[i] >= 0 ? off_b[i] : 0, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        db[i][p] = __ffma2_rn(gb[i][p], __fmul2_rn(vb[i][p], inv2), db[i][p]);
                        vb[i][p] = __fmul2_rn(inv2, __ffma2_rn(vb[i][p], nc, __fmul2_rn(w[p], gb[i][p])));
                    }
                } else if (tab[i] >= 0) {
                    turn<H, HALF, NORM>(va[i], vb[i], tab_s + tab[i], run, sin_off, inv);
                } else if (NORM) {
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        va[i][p] = __fmul2_rn(va[i][p], both(inv));
                        vb[i][p] = __fmul2_rn(vb[i][p], both(inv));
                    }
                }
                uint8_t *y = k ? yk : yq;
                if (off_a[i] >= 0) st_stream_batched(y + off_a[i], pack2<TA, H>(va[i]));
                if (off_b[i] >= 0) st_stream_batched(y + off_b[i], pack2<TA, H>(vb[i]));
            }
            __syncwarp();  // the warp has read the stage and its table
            if (lane == 0) mbar_arrive(empty + 8u * stage);
            if (++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
            }
            par ^= 1;
        }
    }

    if constexpr (BACK) {
        // one row of partial sums per block: the groups' sums meet in the ring, added in group order
        const int dq = a.job[0].d, d = dq + (a.njobs > 1 ? a.job[1].d : 0);
        float *out = a.part + (int64_t)blockIdx.x * d;
        float *mine = a.groups > 1 ? reinterpret_cast<float *>(rings) + (size_t)group * d : out;
        __syncthreads();  // every group has read its last stage
        if (gw < a.warps) {
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                if (off_a[i] < 0) continue;
                const bool k = (is_k >> i) & 1u;
                const int col = k ? dq : 0, ro = k ? a.job[1].row_off : 0;
                float2 *pa = reinterpret_cast<float2 *>(mine + col + (off_a[i] - ro) / 16 * E);
#pragma unroll
                for (int p = 0; p < H; ++p) pa[p] = da[i][p];
                if (off_b[i] >= 0) {
                    float2 *pb = reinterpret_cast<float2 *>(mine + col + (off_b[i] - ro) / 16 * E);
#pragma unroll
                    for (int p = 0; p < H; ++p) pb[p] = db[i][p];
                }
            }
        }
        if (a.groups > 1) {
            __syncthreads();
            const float *all = reinterpret_cast<const float *>(rings);
            for (int c = threadIdx.x; c < d; c += blockDim.x) {
                float s = all[c];
                for (int gi = 1; gi < a.groups; ++gi) s += all[(size_t)gi * d + c];
                out[c] = s;
            }
        }
    }
}

// ---------------------------------------------------------------- host side

struct Plan {
    bool fits;
    int upt, warps, warps0, groups, threads;
    bool wide;
};

constexpr int kMaxCtas = 4;  // blocks per SM at most (the partial gradients' rows are sized by it)

// Whether the unit kernel takes the call, and its geometry: a rule on the
// rows' widths, types and alignment, never on the number of tokens.
template <typename TA, typename TW, int MODE>
Plan plan(const Args &a, Params &p) {
    constexpr int E = Chunk<TA>::E;
    Plan r{};
    p.x_bytes = 0;
    for (int i = 0; i < a.njobs; ++i) {
        const Job &j = a.job[i];
        Rows &J = p.job[i];
        const int D = a.r ? a.D : j.d;
        if (D % E != 0 || a.r % (2 * E) != 0 || !aligned(j.x, 16) || !aligned(j.y, 16) || j.ldx % 16 || j.ldy % 16)
            return r;
        if (MODE == kNormBack && (!aligned(j.g, 16) || j.ldg % 16)) return r;
        if (MODE != kRotate && !aligned(j.w, 4)) return r;
        if ((int64_t)j.d * (int64_t)sizeof(TA) > kSmemLimit) return r;
        J.x = j.x;
        J.g = j.g;
        J.y = j.y;
        J.w = j.w;
        J.ldx = j.ldx;
        J.ldg = j.ldg;
        J.ldy = j.ldy;
        J.d = j.d;
        J.row_bytes = j.d * (int)sizeof(TA);
        J.row_off = p.x_bytes;
        p.x_bytes += J.row_bytes;
        J.head_chunks = D / E;
        J.tail_chunks = (D - a.r) / E;
        J.tail_units = (J.tail_chunks + 1) / 2;
        J.units_per_head = a.r / (2 * E) + J.tail_units;
        J.nunits = j.d / D * J.units_per_head;
    }
    if (a.njobs == 1) p.job[1] = Rows{};
    p.stage_bytes = p.x_bytes * (MODE == kNormBack ? 2 : 1);
    p.rot_units = a.r / (2 * E);
    const int u0 = p.job[0].nunits, u1 = a.njobs > 1 ? p.job[1].nunits : 0;
    auto warps_of = [](int units, int upt) { return (units + 32 * upt - 1) / (32 * upt); };
    // two units of 16 bf16 elements or four of 8 fp32 a thread; half of that where one warp is
    // enough for both tensors, twice that for rows too wide otherwise
    constexpr int kUsual = sizeof(TA) == 4 ? 4 : 2;
    const int most = MODE == kNormBack ? kUsual : 4;
    for (r.upt = u0 + u1 <= 16 * kUsual ? kUsual / 2 : kUsual; r.upt <= most; r.upt *= 2) {
        if (u0 + u1 <= 32 * r.upt) {  // one warp for both tensors
            r.warps0 = r.warps = 1;
        } else {
            r.warps0 = warps_of(u0, r.upt);
            r.warps = r.warps0 + warps_of(u1, r.upt);
        }
        if (r.warps <= kMaxWarps) break;
    }
    if (r.upt > most) return r;
    r.wide = r.warps > 10;
    r.groups = r.warps == 1 ? 4 : r.warps == 2 ? 3 : r.warps <= 4 ? 2 : 1;
    r.threads = r.groups * (r.warps + 1) * 32;
    r.fits = true;
    return r;
}

template <typename TA, typename TW, int MODE, int UPT, bool HALF, bool WIDE>
qkn_status launch_kernel(Params &p, const Plan &r, int *grid, cudaStream_t s, bool *taken) {
    const auto kernel = rotary_unit_kernel<TA, TW, MODE, UPT, HALF, WIDE>;
    static std::atomic<int> registers[64];  // per device: registers per thread, 0 until asked
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    int regs = known ? registers[dev].load(std::memory_order_acquire) : 0;
    if (regs == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(rotary_unit_kernel)");
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, kernel);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(rotary_unit_kernel)");
        regs = fa.numRegs;
        if (known) registers[dev].store(regs, std::memory_order_release);
    }
    // as many blocks per SM as the registers hold (16384 per quarter of an SM, whole warps), with
    // at least two stages each
    int ctas = 16384 / ((regs + 7) / 8 * 8 * 32) * 4 / (r.threads / 32), smem = 0;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    if (ctas < 1) ctas = 1;
    *taken = false;
    for (; ctas >= 1 && !*taken; --ctas) {
        const int budget = ctas == 1 ? kSmemLimit : 228 * 1024 / ctas - 1024;  // 1 KiB per block is the system's
        for (p.stages = 8; p.stages >= 1; --p.stages) {
            smem = p.w_bytes + r.groups * (p.stages * p.stage_bytes + group_fixed(p.r, p.stages));
            if (smem <= budget) break;
        }
        if (p.stages >= 2 || (ctas == 1 && p.stages == 1)) {
            *taken = true;
            break;
        }
    }
    if (!*taken) return QKN_OK;
    const int64_t need = (p.T + r.groups - 1) / r.groups, cap = (int64_t)ctas * sm_count();
    *grid = (int)(need < cap ? need : cap);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)*grid, 1, 1);
    cfg.blockDim = dim3((unsigned)r.threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess) return cuda_fail(e, "rotary_unit_kernel launch");
    return check_launch("rotary_unit_kernel launch");
}

template <typename TA, typename TW, int MODE, int UPT, bool WIDE>
qkn_status launch_layout(Params &p, const Plan &r, int layout, int *grid, cudaStream_t s, bool *taken) {
    return layout == QKN_ROTARY_HALF ? launch_kernel<TA, TW, MODE, UPT, true, WIDE>(p, r, grid, s, taken)
                                     : launch_kernel<TA, TW, MODE, UPT, false, WIDE>(p, r, grid, s, taken);
}

// Launches the unit kernel when it takes the call (*taken); *grid is its number of blocks.
template <typename TA, typename TW, int MODE>
qkn_status launch(const Args &a, bool *taken, int *grid, cudaStream_t s) {
    Params p{};
    const Plan r = plan<TA, TW, MODE>(a, p);
    *taken = r.fits;
    if (!r.fits) return QKN_OK;
    p.njobs = a.njobs;
    p.T = a.T;
    p.r = a.r;
    p.pos = a.pos;
    p.pos64 = a.pos64;
    p.freq = a.freq;
    p.mscale = a.mscale;
    p.sign = a.sign;
    p.eps = a.eps;
    p.part = a.part;
    p.warps = r.warps;
    p.warps0 = r.warps0;
    p.groups = r.groups;
    p.wait_ns = kWaitTimeoutNs;
    p.w_bytes = MODE == kRotate ? 0 : ((p.job[0].d + p.job[1].d) * (int)sizeof(TW) + 15) / 16 * 16;
    constexpr int kUsual = sizeof(TA) == 4 ? 4 : 2;
    if (r.upt < kUsual) return launch_layout<TA, TW, MODE, kUsual / 2, false>(p, r, a.layout, grid, s, taken);
    if (r.upt == kUsual)
        return r.wide ? launch_layout<TA, TW, MODE, kUsual, true>(p, r, a.layout, grid, s, taken)
                      : launch_layout<TA, TW, MODE, kUsual, false>(p, r, a.layout, grid, s, taken);
    if constexpr (MODE != kNormBack && kUsual < 4)
        return launch_layout<TA, TW, MODE, 4, true>(p, r, a.layout, grid, s, taken);
    return fail(QKN_ERR_UNSUPPORTED, "rotary_unit_kernel: no variant for these rows");
}

}  // namespace unit
}  // namespace rot

// Reads and clears the unit kernel's device error word (current device).
qkn_status read_rotary_error(int *flag) {
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_rotary_error, sizeof(int));
    if (e != cudaSuccess) return cuda_fail(e, "reading the rotary kernel's device error word");
    if (*flag) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_rotary_error, &zero, sizeof zero);
    }
    return QKN_OK;
}

}  // namespace qkn
