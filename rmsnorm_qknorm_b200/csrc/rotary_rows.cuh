// Unit kernel of the rotary entry points: rows of 16- or 8-byte chunks,
// persistent, fed by bulk copies.
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
// chunks, chunk j and chunk j + r / 2E of a head (E elements per chunk, 16
// bytes of them, or 8 where the rotated part of a bf16 head is a multiple of
// 16 but not of 32 bytes).  In the half layout the two chunks hold the two
// sides of E pairs;
// in the interleaved layout each holds E / 2 whole pairs.  Either way a unit
// needs the cos and sin of two runs of E / 2 frequencies, which the table
// keeps at positions j and j + r / 2E (filled in the order the layout asks
// for), so neighbouring threads read neighbouring 16-byte words.  Chunks
// behind the rotated part form units of their own, copied (or only
// normalised).  Rows so narrow that one warp has lanes to spare go several
// tokens to a stage, each with its share of the warp's lanes (and its table).
// Fixed columns keep the weights' gradients in registers over all tokens; the
// weights are read from a copy in shared memory.
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
    int stages, stage_bytes, x_bytes;  // x_bytes: the rows of one token
    int tokens, lanes;       // tokens per stage (a power of two), lanes per token
    int table;               // floats of a token's table: cos, sin and, where units are flipped, -sin
    int flip;                // units with this bit in their number take their chunks in the other order (0: none)
    int w_bytes, w_bf16;     // the block's fp32 copy of the weights, in front of the rings; their type in memory
    uint64_t wait_ns;
};

constexpr int kMaxWarps = 15;  // consumer warps per group
constexpr int kSlots = 16;     // sums per tensor and token

inline __host__ __device__ int table_bytes(int floats) { return (floats * 4 + 15) / 16 * 16; }  // of a stage
// per group: tables, 2 tokens x 2 tensors x (sum x^2, sum w g x) x kSlots sums, full and empty barriers
inline __host__ __device__ int group_fixed(int floats, int stages) {
    return stages * table_bytes(floats) + 8 * kSlots * 4 + stages * 16;
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

// A chunk in shared memory as E / 2 = H pairs of fp32 (16 bytes, or 8: four bf16).
template <typename TA, int H> __device__ __forceinline__ void lds_chunk(uint32_t addr, float2 (&f)[H]) {
    if constexpr (sizeof(TA) == 4) {
        const uint4 v = lds128(addr);
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    } else if constexpr (H == 2) {
        uint2 v;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
        f[0] = make_float2(bf16lo(v.x), bf16hi(v.x));
        f[1] = make_float2(bf16lo(v.y), bf16hi(v.y));
    } else {
        const uint4 v = lds128(addr);
        f[0] = make_float2(bf16lo(v.x), bf16hi(v.x));
        f[1] = make_float2(bf16lo(v.y), bf16hi(v.y));
        f[2] = make_float2(bf16lo(v.z), bf16hi(v.z));
        f[3] = make_float2(bf16lo(v.w), bf16hi(v.w));
    }
}
template <typename TA, int H> __device__ __forceinline__ void store_chunk(uint8_t *p, const float2 (&f)[H]) {
    if constexpr (sizeof(TA) == 4)
        st_stream_batched(p, make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                                        __float_as_uint(f[1].y)));
    else if constexpr (H == 2)
        asm("st.global.cs.v2.u32 [%0], {%1, %2};"
            ::"l"(p), "r"(pack_bf16x2(f[0].x, f[0].y)), "r"(pack_bf16x2(f[1].x, f[1].y)) : "memory");
    else
        st_stream_batched(p, make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                        pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y)));
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

// cos and sin of a unit's two frequency runs.
template <int H> struct Turns {
    float2 c[H], s[H];
    __device__ __forceinline__ void load(uint32_t cos_addr, uint32_t run, uint32_t sin_off) {
        float2 t[H / 2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            lds_run<H>(cos_addr + (q ? run : 0u), t);
#pragma unroll
            for (int p = 0; p < H / 2; ++p) c[q * (H / 2) + p] = t[p];
            lds_run<H>(cos_addr + sin_off + (q ? run : 0u), t);
#pragma unroll
            for (int p = 0; p < H / 2; ++p) s[q * (H / 2) + p] = t[p];
        }
    }
};

// The two chunks of a unit, turned and (SCALE) multiplied by inv.
template <int H, bool HALF, bool SCALE>
__device__ __forceinline__ void turn(float2 (&a)[H], float2 (&b)[H], const Turns<H> &t, float inv) {
    if constexpr (HALF) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float2 x = a[i], y = b[i];
            const float2 xc = __fmul2_rn(x, t.c[i]), ys = __fmul2_rn(y, t.s[i]), yc = __fmul2_rn(y, t.c[i]);
            if constexpr (SCALE) {
                a[i] = __ffma2_rn(ys, both(-inv), __fmul2_rn(xc, both(inv)));
                b[i] = __fmul2_rn(__ffma2_rn(x, t.s[i], yc), both(inv));
            } else {
                a[i] = __ffma2_rn(ys, both(-1.f), xc);
                b[i] = __ffma2_rn(x, t.s[i], yc);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2 * H; ++i) {  // chunk a's pairs take the first run, chunk b's the second
            const int f = i;
            const float ce = (f & 1) ? t.c[f >> 1].y : t.c[f >> 1].x, se = (f & 1) ? t.s[f >> 1].y : t.s[f >> 1].x;
            const float2 v = i < H ? a[i % H] : b[i % H];
            float2 r = make_float2(v.x * ce - v.y * se, v.y * ce + v.x * se);
            if constexpr (SCALE) r = __fmul2_rn(r, both(inv));
            if (i < H) a[i % H] = r;
            else b[i % H] = r;
        }
    }
}

// The weights of a unit's chunk from shared memory, as pairs.  They are kept as
// fp32, the first four of every chunk in one array and, for chunks of eight,
// the others `upper` bytes behind: neighbouring threads read neighbouring
// words.  The chunks lie in the row's order, or (ORDERED) in the units', all
// first chunks before all second ones.
template <int H>
__device__ __forceinline__ void lds_weights(uint32_t addr, uint32_t upper, float2 (&f)[H]) {
    const uint4 a = lds128(addr);
    f[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    f[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    if constexpr (H == 4) {
        const uint4 b = lds128(addr + upper);
        f[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
        f[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
    }
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The sum of a over the warp on lanes 0 .. 15, of b on lanes 16 .. 31: each half hands the other
// what it does not keep, then both reduce at once.
__device__ __forceinline__ float warp_sum_of_two(float a, float b, int lane) {
    const bool upper = lane & 16;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
    for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The sum over the lanes of a token.
__device__ __forceinline__ float token_sum(float v, int lanes) {
    for (int off = lanes >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Threads of a block: 20 warps leave a thread 96 registers, 16 warps 128 (the
// gradients, and the variant with twice the units).
template <int MODE, int UPT, int E> constexpr int max_threads() { return MODE == kNormBack || UPT * E > 16 ? 512 : 640; }

// How the warps of a group divide the rows.
enum Shape {
    SPLIT,  // q and k have warps of their own
    MIXED,  // warps serve both tensors (with the norm, one warp does)
    MULTI   // one warp serves both tensors of several tokens at a time
};

// ORDERED: for heads in which units next to one another meet in shared memory's banks (see ordered_of).
template <typename TA, int E, int MODE, int UPT, bool HALF, int SHAPE, bool ORDERED>
__global__ void __launch_bounds__(max_threads<MODE, UPT, E>(), 1) rotary_unit_kernel(const Params a) {
    constexpr bool BOTH = SHAPE != SPLIT, BATCH = SHAPE == MULTI;
    constexpr int H = E / 2, CB = E * (int)sizeof(TA);  // bytes of a chunk
    constexpr bool NORM = MODE != kRotate, BACK = MODE == kNormBack;
    extern __shared__ __align__(128) uint8_t smem[];
    const int gthreads = (a.warps + 1) * 32;
    const int group = threadIdx.x / gthreads, gt = threadIdx.x - group * gthreads;  // thread within its group
    const int lane = threadIdx.x & 31, gw = gt >> 5;
    uint8_t *rings = smem + a.w_bytes;
    uint8_t *fix_p = rings + (size_t)a.groups * a.stages * a.stage_bytes + (size_t)group * group_fixed(a.table * a.tokens, a.stages);
    const uint32_t ring = smem_u32(rings + (size_t)group * a.stages * a.stage_bytes);
    const int tbytes = table_bytes(a.table * a.tokens);
    float *red = reinterpret_cast<float *>(fix_p + (size_t)a.stages * tbytes);
    const uint32_t full = smem_u32(red + 8 * kSlots), empty = full + 8u * a.stages;
    // Tokens are taken `tokens` at a time: batch n holds tokens n * tokens ...
    const int per = BATCH ? a.tokens : 1;
    const int64_t batches = BATCH ? (a.T + per - 1) / per : a.T;
    const int64_t step = (int64_t)gridDim.x * a.groups;
    const int64_t first_batch = (int64_t)group * gridDim.x + blockIdx.x;  // few tokens spread over the SMs first
    const int g_off = a.x_bytes * per;  // of the gradients in a stage

    // copies of a batch's rows into a stage (the producer warp)
    auto fill = [&](int64_t n, int stage) {
        const uint32_t bar = full + 8u * stage, dst = ring + (uint32_t)(stage * a.stage_bytes);
        if constexpr (!BATCH) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, (uint32_t)a.stage_bytes);
                bulk_g2s(dst, a.job[0].x + n * a.job[0].ldx, a.job[0].row_bytes, bar);
                if (BACK) bulk_g2s(dst + a.x_bytes, a.job[0].g + n * a.job[0].ldg, a.job[0].row_bytes, bar);
                if (a.njobs > 1) {
                    bulk_g2s(dst + a.job[1].row_off, a.job[1].x + n * a.job[1].ldx, a.job[1].row_bytes, bar);
                    if (BACK)
                        bulk_g2s(dst + a.x_bytes + a.job[1].row_off, a.job[1].g + n * a.job[1].ldg, a.job[1].row_bytes, bar);
                }
            }
        } else {
            const int64_t t0 = n * per;
            const int rows = a.T - t0 < per ? (int)(a.T - t0) : per;
            if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(rows * a.x_bytes * (BACK ? 2 : 1)));
            __syncwarp();
            for (int i = lane; i < rows * a.njobs; i += 32) {
                const int t = a.njobs > 1 ? i >> 1 : i;
                const Rows J = pick(a, a.njobs > 1 ? i & 1 : 0);
                const uint32_t to = dst + (uint32_t)(t * a.x_bytes + J.row_off);
                bulk_g2s(to, J.x + (t0 + t) * J.ldx, J.row_bytes, bar);
                if (BACK) bulk_g2s(to + g_off, J.g + (t0 + t) * J.ldg, J.row_bytes, bar);
            }
        }
    };
    uint32_t issued = 0;  // stages filled (the producer warp)
    if (gw == a.warps) {
        if (lane == 0) {
            for (int s = 0; s < a.stages; ++s) {
                mbar_init(full + 8u * s, 2);         // the producer's two arrivals and the copies' bytes
                mbar_init(empty + 8u * s, a.warps);  // one per consumer warp
            }
            mbar_init_fence();
        }
        __syncwarp();
        // the previous kernel on the stream has finished before any global memory is touched
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int64_t n = first_batch;
        for (int s = 0; s < a.stages && n < batches; ++s, n += step) {
            fill(n, s);
            issued |= 1u << s;
        }
    }
    for (int i = gt; i < 8 * kSlots; i += gthreads) red[i] = 0.f;
    // places of the weights' copy: the row's chunks or the units, and one of zeros.  What a thread has no
    // chunk for it reads there, its rows' elements and its weights: 0 times another weight would be
    // NaN where that weight is not finite
    const int units0 = a.job[0].nunits, chunks0 = a.job[0].row_bytes / CB;
    const int places = (ORDERED ? units0 + a.job[1].nunits : a.x_bytes / CB) + 1;
    const uint32_t zero_at = NORM ? (uint32_t)(places - 1) * 16u : 0u;
    auto flipped = [&](int u) { return ORDERED && (u & a.flip) != 0; };
    if (!NORM && threadIdx.x < 4) reinterpret_cast<float *>(smem)[threadIdx.x] = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if constexpr (NORM) {
        float4 *w = reinterpret_cast<float4 *>(smem);
        for (int i = threadIdx.x; i < (ORDERED ? 2 * places : places); i += blockDim.x) {
            const int side = ORDERED && i >= places ? 1 : 0, place = i - side * places;
            const bool k = place >= (ORDERED ? units0 : chunks0), last = place == places - 1;
            int at = last ? -1 : place - (k ? (ORDERED ? units0 : chunks0) : 0);  // the chunk of the row, -1: zeros
            const Rows J = pick(a, k ? 1 : 0);
            float f[E];
            if (ORDERED && !last) {
                const int u = at, h = u / J.units_per_head, j = u - h * J.units_per_head;
                const int t = j - a.rot_units, second = t < 0 ? a.rot_units : J.tail_units;  // from first chunk to second
                const bool pair = t < 0 || t + J.tail_units < J.tail_chunks;
                at = h * J.head_chunks + (t < 0 ? j : j + a.rot_units) + (pair && (side ^ (flipped(u) ? 1 : 0)) ? second : 0);
                if (side && !pair) at = -1;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = 0.f;
            if (at >= 0) {
                if (a.w_bf16) load_weights_batched<__nv_bfloat16, E>(static_cast<const __nv_bfloat16 *>(J.w) + at * E, f);
                else load_weights_batched<float, E>(static_cast<const float *>(J.w) + at * E, f);
            }
#pragma unroll
            for (int q = 0; q < E / 4; ++q)
                w[(side * (E / 4) + q) * places + place] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
        }
    }
    __syncthreads();

    float2 da[UPT][H], db[UPT][H];  // gradients of the weights, over this group's tokens
    int off_a[UPT], off_b[UPT], tab[UPT];  // stage offsets of a unit's chunks (-1: none), table offset (-1: not turned)
    uint32_t is_k = 0, flips = 0;  // bit i: unit i is of the keys, has its chunks in the other order

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
        auto entry = [&](float *t, int64_t pt, double turns) {
            float c, s;
            cos_sin(pt, turns, a.mscale, a.sign, c, s);
            t[0] = c;
            t[nf] = s;
            if (ORDERED && HALF && a.flip) t[2 * nf] = -s;
        };
        int stage = 0;
        uint32_t phase = 0;
        bool first = true;  // the first round of stages is filled already
        int64_t p = pos_at(first_batch * per + (BATCH ? lane % per : 0));  // lane t holds token t's position
        for (int64_t n = first_batch; n < batches; n += step) {
            const uint32_t bar = full + 8u * stage;
            if (!first) {
                const bool ok = mbar_wait_fast(empty + 8u * stage, phase ^ 1u, &g_rotary_error, a.wait_ns);
                if (__any_sync(0xffffffffu, !ok)) break;
                fill(n, stage);
            }
            const int64_t next = pos_at((n + step) * per + (BATCH ? lane % per : 0));
            float *t = reinterpret_cast<float *>(fix_p + (size_t)stage * tbytes);
            // one token after the other where its pairs fill the warp, all at once where they do not
            if (BATCH && nf < 32) {
                for (int i0 = 0; i0 < per * nf; i0 += 32) {
                    const int i = i0 + lane, tok = min(i / nf, per - 1), f = i - i / nf * nf;
                    const int64_t pt = __shfl_sync(0xffffffffu, p, tok);
                    if (i < per * nf) entry(t + tok * a.table + place(f), pt, __ldg(a.freq + f) * kInvTwoPi);
                }
            } else {
                for (int tok = 0; tok < per; ++tok, t += a.table) {
                    const int64_t pt = BATCH ? __shfl_sync(0xffffffffu, p, tok) : p;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (lane + 32 * i < nf) entry(t + at[i], pt, turns[i]);
                    for (int f = lane + 64; f < nf; f += 32) entry(t + place(f), pt, __ldg(a.freq + f) * kInvTwoPi);
                }
            }
            p = next;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
            if (++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
                first = false;
            }
        }
        // no copy may still be writing when the block exits: the last phase filled on every stage
        // (on the normal path the consumers have waited for them all already).  Stages behind
        // `stage` were last filled in the round before, or, in the first round, in this one
        if (lane == 0)
            for (int s = 0; s < a.stages; ++s)
                if (issued & (1u << s))
                    mbar_wait(full + 8u * s, s < stage || first ? phase : phase ^ 1u, &g_rotary_error, a.wait_ns);
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- consumer warps
        const bool wk = !BOTH && gw >= a.warps0;  // a warp of the keys
        int slot[UPT];  // of the unit's weights
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            int which = wk ? 1 : 0;
            const int jw = wk ? a.warps - a.warps0 : a.warps0;
            int u = BATCH ? lane % a.lanes + i * a.lanes : gt - (wk ? a.warps0 * 32 : 0) + i * jw * 32;
            if (BOTH && u >= a.job[0].nunits) {
                u -= a.job[0].nunits;
                which = 1;
            }
            off_a[i] = off_b[i] = tab[i] = -1;
            slot[i] = ORDERED ? places - 1 : 0;
            if (which) is_k |= 1u << i;
            if (u >= (which ? a.job[1].nunits : a.job[0].nunits)) continue;
            const Rows J = pick(a, which);
            const int h = u / J.units_per_head, j = u - h * J.units_per_head;
            const int first = h * J.head_chunks;
            if (j < a.rot_units) {
                off_a[i] = J.row_off + (first + j) * CB;
                off_b[i] = off_a[i] + a.rot_units * CB;
                tab[i] = j * H * 4;
            } else {
                const int t = j - a.rot_units;
                off_a[i] = J.row_off + (first + 2 * a.rot_units + t) * CB;
                if (t + J.tail_units < J.tail_chunks) off_b[i] = off_a[i] + J.tail_units * CB;
            }
            if constexpr (ORDERED) slot[i] = u + (which ? units0 : 0);
            if (flipped(u) && off_b[i] >= 0) {
                const int t = off_a[i];
                off_a[i] = off_b[i];
                off_b[i] = t;
                flips |= 1u << i;
            }
        }
        if constexpr (BACK) {
#pragma unroll
            for (int i = 0; i < UPT; ++i)
#pragma unroll
                for (int p = 0; p < H; ++p) da[i][p] = db[i][p] = make_float2(0.f, 0.f);
        }
        const uint32_t sin_off = (uint32_t)a.r * 2u, run = (uint32_t)a.rot_units * H * 4u;  // bytes
        const uint32_t tables = smem_u32(fix_p), w_s = smem_u32(smem), upper = (uint32_t)places * 16u;
        // the turns of unit i: flipped, the half layout takes the negative sine, the interleaved one its runs the other way
        auto load_turns = [&](Turns<H> &cs, uint32_t tab_s, int i) {
            const bool f = ORDERED && ((flips >> i) & 1u);
            if constexpr (HALF) cs.load(tab_s + tab[i], run, f ? 2 * sin_off : sin_off);
            else cs.load(tab_s + tab[i] + (f ? run : 0u), f ? 0u - run : run, sin_off);
        };
        // a chunk that is not there reads zeros (behind the weights) and stores nothing
        const uint32_t zeros = w_s + zero_at;
        auto weights_at = [&](int off) { return off < 0 ? zeros : w_s + (uint32_t)off * (16 / CB); };
        auto weights_a = [&](int i) { return ORDERED ? w_s + (uint32_t)slot[i] * 16u : weights_at(off_a[i]); };
        auto weights_b = [&](int i) { return ORDERED ? w_s + (uint32_t)slot[i] * 16u + upper * (uint32_t)(E / 4) : weights_at(off_b[i]); };
        // a thread's units lie at the same place of their heads when a head's units divide the
        // warps' stride (powers of two do): cos and sin are then read once per token (not for the
        // gradients, which would spill the registers that keeping them takes)
        bool same = !BACK;
#pragma unroll
        for (int i = 1; i < UPT; ++i) same = same && (off_a[i] < 0 || (tab[i] == tab[0] && ((flips >> i) & 1u) == (flips & 1u)));
        if (!BACK) same = __all_sync(0xffffffffu, same);
        const float d_q = (float)a.job[0].d, d_k = (float)a.job[1].d;
        // rows of the results, moved by the chunk's place in a stage
        const int sub = BATCH ? lane / a.lanes : 0;  // this lane's token of a batch
        int64_t token = first_batch * per + sub;
        uint8_t *yq = (wk ? a.job[1].y - a.job[1].row_off : a.job[0].y) + token * (wk ? a.job[1].ldy : a.job[0].ldy);
        uint8_t *yk = BOTH ? a.job[1].y - a.job[1].row_off + token * a.job[1].ldy : nullptr;
        const int64_t yq_step = step * per * (wk ? a.job[1].ldy : a.job[0].ldy), yk_step = step * per * a.job[1].ldy;
        const int my_warps = wk ? a.warps - a.warps0 : a.warps0, my_warp = wk ? gw - a.warps0 : gw;

        int stage = 0, par = 0;
        uint32_t phase = 0;
        // batches of this group (fewer than 2^31)
        for (int left = first_batch < batches ? (int)((batches - first_batch - 1) / step) + 1 : 0; left > 0; --left) {
            const bool ok = mbar_wait_fast(full + 8u * stage, phase, &g_rotary_error, a.wait_ns);
            const uint32_t src = ring + (uint32_t)(stage * a.stage_bytes + (BATCH ? sub * a.x_bytes : 0));
            const uint32_t tab_s = tables + (uint32_t)(stage * tbytes + (BATCH ? sub * a.table * 4 : 0));
            const bool live = !BATCH || token < a.T;  // the last batch may have fewer tokens
            float2 va[UPT][H], vb[UPT][H];  // rotary: x; with the norm: x w; gradients: g, dy turned back
            float2 sq[2] = {both(0.f), both(0.f)}, pg[2] = {both(0.f), both(0.f)};  // sums of x^2 and of w g x
            Turns<H> cs;
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                const bool has_a = live && off_a[i] >= 0, has_b = live && off_b[i] >= 0;
                const uint32_t pa = has_a ? src + off_a[i] : zeros, pb = has_b ? src + off_b[i] : zeros;
                const uint32_t qa = weights_a(i), qb = weights_b(i);
                const int m = BOTH ? (is_k >> i) & 1u : 0;
                if constexpr (MODE == kRotate) {
                    lds_chunk<TA, H>(pa, va[i]);
                    lds_chunk<TA, H>(pb, vb[i]);
                } else if constexpr (MODE == kNorm) {
                    float2 q = both(0.f), w[H];
                    lds_chunk<TA, H>(pa, va[i]);
                    lds_weights<H>(qa, upper, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) q = __ffma2_rn(va[i][p], va[i][p], q);
#pragma unroll
                    for (int p = 0; p < H; ++p) va[i][p] = __fmul2_rn(va[i][p], w[p]);
                    lds_chunk<TA, H>(pb, vb[i]);
                    lds_weights<H>(qb, upper, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) q = __ffma2_rn(vb[i][p], vb[i][p], q);
#pragma unroll
                    for (int p = 0; p < H; ++p) vb[i][p] = __fmul2_rn(vb[i][p], w[p]);
                    if (m) sq[1] = __fadd2_rn(sq[1], q);
                    else sq[0] = __fadd2_rn(sq[0], q);
                } else {
                    lds_chunk<TA, H>(has_a ? pa + g_off : zeros, va[i]);
                    lds_chunk<TA, H>(has_b ? pb + g_off : zeros, vb[i]);
                    if (tab[i] >= 0) {
                        load_turns(cs, tab_s, i);
                        turn<H, HALF, false>(va[i], vb[i], cs, 1.f);
                    }
                    float2 q = both(0.f), r = both(0.f), w[H], x[H];
                    lds_chunk<TA, H>(pa, x);
                    lds_weights<H>(qa, upper, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        q = __ffma2_rn(x[p], x[p], q);
                        r = __ffma2_rn(__fmul2_rn(x[p], va[i][p]), w[p], r);
                    }
                    lds_chunk<TA, H>(pb, x);
                    lds_weights<H>(qb, upper, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        q = __ffma2_rn(x[p], x[p], q);
                        r = __ffma2_rn(__fmul2_rn(x[p], vb[i][p]), w[p], r);
                    }
                    if (m) {
                        sq[1] = __fadd2_rn(sq[1], q);
                        pg[1] = __fadd2_rn(pg[1], r);
                    } else {
                        sq[0] = __fadd2_rn(sq[0], q);
                        pg[0] = __fadd2_rn(pg[0], r);
                    }
                }
            }
            float inv_q = 1.f, inv_k = 1.f, cq = 0.f, ck = 0.f;
            bool failed = !ok;
            if constexpr (NORM) {
                float s, t = 0.f;
                if constexpr (BOTH) {
                    const int lanes = BATCH ? a.lanes : 32;
                    s = token_sum(sq[0].x + sq[0].y, lanes);
                    if (BACK) t = token_sum(pg[0].x + pg[0].y, lanes);
                    inv_k = rsqrtf(token_sum(sq[1].x + sq[1].y, lanes) / d_k + a.eps);
                    if (BACK) ck = inv_k * inv_k * (token_sum(pg[1].x + pg[1].y, lanes) / d_k);
                    failed = __any_sync(0xffffffffu, failed);
                } else {
                    // the sums of this token: [q | k][x^2 | w g x][kSlots], slots without a warp hold zero
                    float *slot = red + (par * 4 + (wk ? 2 : 0)) * kSlots;
                    if constexpr (BACK) {
                        // both sums in one pass: the lower lanes end with the first, the upper with the second
                        const float u = warp_sum_of_two(sq[0].x + sq[0].y, pg[0].x + pg[0].y, lane);
                        if ((lane & 15) == 0) slot[(lane ? kSlots : 0) + my_warp] = u;
                    } else {
                        s = warp_sum(sq[0].x + sq[0].y);
                        if (lane == 0) slot[my_warp] = s;
                    }
                    failed = group_sync_or(failed, group, a.warps);
                    s = t = 0.f;
                    for (int w = 0; w < my_warps; w += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(slot + w);
                        s = (((s + v.x) + v.y) + v.z) + v.w;
                        if constexpr (BACK) {
                            const float4 u = *reinterpret_cast<const float4 *>(slot + kSlots + w);
                            t = (((t + u.x) + u.y) + u.z) + u.w;
                        }
                    }
                }
                const float d = wk ? d_k : d_q;
                inv_q = rsqrtf(s / d + a.eps);
                if (BACK) cq = inv_q * inv_q * (t / d);
                if (BATCH && !live) inv_q = inv_k = cq = ck = 0.f;  // no row: nothing for the weights' sums
            } else {
                failed = __any_sync(0xffffffffu, failed);
            }
            if (failed) break;
            if (!BACK && same && tab[0] >= 0) load_turns(cs, tab_s, 0);
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                const bool has_a = live && off_a[i] >= 0, has_b = live && off_b[i] >= 0;
                const bool m = BOTH && ((is_k >> i) & 1u);
                const float inv = m ? inv_k : inv_q;
                uint8_t *y = m ? yk : yq;
                if constexpr (BACK) {
                    const float2 nc = both(-(m ? ck : cq)), inv2 = both(inv);
                    float2 w[H], x[H];
                    lds_chunk<TA, H>(has_a ? src + off_a[i] : zeros, x);
                    lds_weights<H>(weights_a(i), upper, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        da[i][p] = __ffma2_rn(va[i][p], __fmul2_rn(x[p], inv2), da[i][p]);
                        va[i][p] = __fmul2_rn(inv2, __ffma2_rn(x[p], nc, __fmul2_rn(w[p], va[i][p])));
                    }
                    if (has_a) store_chunk<TA, H>(y + off_a[i], va[i]);
                    lds_chunk<TA, H>(has_b ? src + off_b[i] : zeros, x);
                    lds_weights<H>(weights_b(i), upper, w);
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        db[i][p] = __ffma2_rn(vb[i][p], __fmul2_rn(x[p], inv2), db[i][p]);
                        vb[i][p] = __fmul2_rn(inv2, __ffma2_rn(x[p], nc, __fmul2_rn(w[p], vb[i][p])));
                    }
                    if (has_b) store_chunk<TA, H>(y + off_b[i], vb[i]);
                } else {
                    if (tab[i] >= 0) {
                        if (!same) load_turns(cs, tab_s, i);
                        turn<H, HALF, NORM>(va[i], vb[i], cs, inv);
                    } else if (NORM) {
#pragma unroll
                        for (int p = 0; p < H; ++p) {
                            va[i][p] = __fmul2_rn(va[i][p], both(inv));
                            vb[i][p] = __fmul2_rn(vb[i][p], both(inv));
                        }
                    }
                    if (has_a) store_chunk<TA, H>(y + off_a[i], va[i]);
                    if (has_b) store_chunk<TA, H>(y + off_b[i], vb[i]);
                }
            }
            yq += yq_step;
            if (BOTH) yk += yk_step;
            if (BATCH) token += step * per;
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
        if (BATCH && gw < a.warps)  // the sums of a batch's tokens meet in the lanes of the first
            for (int off = a.lanes; off < 32; off <<= 1)
#pragma unroll
                for (int i = 0; i < UPT; ++i)
#pragma unroll
                    for (int p = 0; p < H; ++p) {
                        da[i][p].x += __shfl_xor_sync(0xffffffffu, da[i][p].x, off);
                        da[i][p].y += __shfl_xor_sync(0xffffffffu, da[i][p].y, off);
                        db[i][p].x += __shfl_xor_sync(0xffffffffu, db[i][p].x, off);
                        db[i][p].y += __shfl_xor_sync(0xffffffffu, db[i][p].y, off);
                    }
        if (gw < a.warps && (!BATCH || lane < a.lanes)) {
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                if (off_a[i] < 0) continue;
                const bool k = (is_k >> i) & 1u;
                const int col = k ? dq : 0, ro = k ? a.job[1].row_off : 0;
                float2 *pa = reinterpret_cast<float2 *>(mine + col + (off_a[i] - ro) / CB * E);
#pragma unroll
                for (int p = 0; p < H; ++p) pa[p] = da[i][p];
                if (off_b[i] >= 0) {
                    float2 *pb = reinterpret_cast<float2 *>(mine + col + (off_b[i] - ro) / CB * E);
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
    int upt, warps, warps0, groups, threads, tokens;
    bool mixed, ordered;
};

// Whether the unit kernel takes the call, and its geometry: a rule on the
// rows' widths, types and alignment, never on the number of tokens.
template <typename TA, int E, int MODE>
Plan plan(const Args &a, Params &p, size_t w_size) {
    Plan r{};
    p.x_bytes = 0;
    for (int i = 0; i < a.njobs; ++i) {
        const Job &j = a.job[i];
        Rows &J = p.job[i];
        const int D = a.r ? a.D : j.d;
        if (D % E != 0 || a.r % (2 * E) != 0 || !aligned(j.x, 16) || !aligned(j.y, 16) || j.ldx % 16 || j.ldy % 16)
            return r;
        if (MODE == kNormBack && (!aligned(j.g, 16) || j.ldg % 16)) return r;
        if (MODE != kRotate && !aligned(j.w, E * w_size < 16 ? E * w_size : 16)) return r;
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
        if (J.row_bytes % 16 != 0) return r;
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
    // Two units of 16 bf16 elements or four of 8 fp32 a thread, twice that in bf16 forward calls for
    // rows too wide otherwise; what 15 warps then do not hold (15360 elements of q and k together, or
    // twice that) the element-wise kernel serves.  (Half of it leaves fewer groups to an SM, and it is the groups that hide one
    // another's barriers: 16384 x (5120 + 1024) bf16, gradients 145 against 118 us, rotary alone 93
    // against 67.)  Warps serve both tensors where nothing is summed over a row, or where one warp
    // is enough.
    constexpr int kUsual = 16 / E;
    const int most = MODE == kNormBack ? kUsual : 4;
    r.upt = kUsual;
    r.mixed = MODE == kRotate || u0 + u1 <= 32 * kUsual;
    for (;; r.upt *= 2) {
        if (r.upt > most) return r;
        r.warps0 = r.mixed ? warps_of(u0 + u1, r.upt) : warps_of(u0, r.upt);
        r.warps = r.mixed ? r.warps0 : r.warps0 + warps_of(u1, r.upt);
        if (r.warps <= kMaxWarps) break;
    }
    // several tokens to a stage while one warp has the lanes for them
    r.tokens = 1;
    while (r.mixed && r.warps == 1 && r.tokens < 8 && (u0 + u1) * r.tokens * 2 <= 32 * r.upt) r.tokens *= 2;
    p.stage_bytes *= r.tokens;
    // groups side by side in a block (one block per SM, so that they share the weights' copy)
    r.groups = (MODE == kNormBack || r.upt * E > 16 ? 16 : 20) / (r.warps + 1);
    r.threads = r.groups * (r.warps + 1) * 32;
    r.fits = true;
    return r;
}

template <typename TA, int E, int MODE, int UPT, bool HALF, int SHAPE, bool ORDERED>
qkn_status launch_kernel(Params &p, const Plan &r, int *grid, cudaStream_t s, bool *taken) {
    const auto kernel = rotary_unit_kernel<TA, E, MODE, UPT, HALF, SHAPE, ORDERED>;
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (!known || !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(rotary_unit_kernel)");
        if (known) attr_set[dev].store(true, std::memory_order_release);
    }
    int smem = 0;
    for (p.stages = 8; p.stages >= 1; --p.stages) {
        smem = p.w_bytes + p.groups * (p.stages * p.stage_bytes + group_fixed(p.table * p.tokens, p.stages));
        if (smem <= kSmemLimit) break;
    }
    *taken = p.stages >= 1;
    if (!*taken) return QKN_OK;
    const int64_t batches = (p.T + p.tokens - 1) / p.tokens;
    *grid = (int)(batches < sm_count() ? batches : sm_count());
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

template <typename TA, int E, int MODE, int UPT, int SHAPE, bool ORDERED>
qkn_status launch_ordered(Params &p, const Plan &r, int layout, int *grid, cudaStream_t s, bool *taken) {
    return layout == QKN_ROTARY_HALF ? launch_kernel<TA, E, MODE, UPT, true, SHAPE, ORDERED>(p, r, grid, s, taken)
                                     : launch_kernel<TA, E, MODE, UPT, false, SHAPE, ORDERED>(p, r, grid, s, taken);
}
template <typename TA, int E, int MODE, int UPT, int SHAPE>
qkn_status launch_layout(Params &p, const Plan &r, int layout, int *grid, cudaStream_t s, bool *taken) {
    if constexpr (MODE != kRotate)
        if (r.ordered) return launch_ordered<TA, E, MODE, UPT, SHAPE, true>(p, r, layout, grid, s, taken);
    return launch_ordered<TA, E, MODE, UPT, SHAPE, false>(p, r, layout, grid, s, taken);
}

// Whether units next to one another meet in shared memory's banks; sets p.flip.
//
// The threads that are served at once (eight with 16 bytes each, sixteen with 8) read without
// conflict where their chunks differ mod their number.  With units in a head that are not a
// multiple of it (heads of 64, 80 or 96 bf16, half of 128 turned) the first chunks of all units do
// not: then the weights lie in the order of the units, and where a power of two of units leaves the
// first chunks in half of the banks, every other four (eight) units take their second chunk first.
// 32768 x (4096 + 1024) bf16, norm and gradients: heads of 64 137 -> 114 and 241 -> 193 us, of 96
// (3840 + 960) 142 -> 125 and 237 -> 206; heads of 128 lose (108 -> 109, 188 -> 194).  Rotary alone, which reads
// a chunk once, runs at the copy's rate without.
template <int CB>
bool ordered_of(Params &p) {
    constexpr int L = 128 / CB;
    const Rows &J = p.job[0];
    p.flip = 0;
    if (J.nunits <= L) return false;
    int seen[2] = {0, 0};
    for (int u = 0, h = 0, j = 0; u < L; ++u) {
        const bool turned = j < p.rot_units;
        const int a = h * J.head_chunks + (turned ? j : j + p.rot_units), b = a + (turned ? p.rot_units : J.tail_units);
        seen[0] |= 1 << a % L;
        seen[1] |= 1 << ((u & L / 2) ? b : a) % L;
        if (++j == J.units_per_head) j = 0, ++h;
    }
    const int plain = __builtin_popcount(seen[0]);
    // (units in no power of two: the pattern changes from head to head)
    if ((J.units_per_head & (J.units_per_head - 1)) == 0 && __builtin_popcount(seen[1]) > plain) p.flip = L / 2;
    return plain < L;
}

// Launches the unit kernel when it takes the call (*taken); *grid is its number of blocks.
template <typename TA, typename TW, int E, int MODE>
qkn_status launch_chunks(const Args &a, bool *taken, int *grid, cudaStream_t s) {
    Params p{};
    Plan r = plan<TA, E, MODE>(a, p, sizeof(TW));
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
    p.tokens = r.tokens;
    p.lanes = 32 / r.tokens;
    p.wait_ns = kWaitTimeoutNs;
    p.w_bf16 = sizeof(TW) == 2;
    r.ordered = MODE != kRotate && ordered_of<E * (int)sizeof(TA)>(p);
    p.table = a.r + (p.flip && a.layout == QKN_ROTARY_HALF ? a.r / 2 : 0);
    // the weights and a place of zeros
    p.w_bytes = MODE == kRotate ? 16 : r.ordered ? (p.job[0].nunits + p.job[1].nunits + 1) * 2 * E * 4
                                                 : (p.job[0].d + p.job[1].d + E) * 4;
    constexpr int kUsual = 16 / E;
    if (r.tokens > 1) return launch_layout<TA, E, MODE, kUsual, MULTI>(p, r, a.layout, grid, s, taken);
    if constexpr (MODE == kRotate) {
        if (r.upt == kUsual) return launch_layout<TA, E, MODE, kUsual, MIXED>(p, r, a.layout, grid, s, taken);
        if constexpr (kUsual < 4) return launch_layout<TA, E, MODE, 4, MIXED>(p, r, a.layout, grid, s, taken);
    } else {
        if (r.mixed) return launch_layout<TA, E, MODE, kUsual, MIXED>(p, r, a.layout, grid, s, taken);
        if (r.upt == kUsual) return launch_layout<TA, E, MODE, kUsual, SPLIT>(p, r, a.layout, grid, s, taken);
        if constexpr (MODE == kNorm && kUsual < 4) return launch_layout<TA, E, MODE, 4, SPLIT>(p, r, a.layout, grid, s, taken);
    }
    return fail(QKN_ERR_UNSUPPORTED, "rotary_unit_kernel: no variant for these rows");
}

// Chunks of 16 bytes, or of 8 where only those divide the heads and their rotated part.
template <typename TA, typename TW, int MODE>
qkn_status launch(const Args &a, bool *taken, int *grid, cudaStream_t s) {
    const qkn_status st = launch_chunks<TA, TW, Chunk<TA>::E, MODE>(a, taken, grid, s);
    if constexpr (sizeof(TA) == 2)
        if (st == QKN_OK && !*taken) return launch_chunks<TA, TW, 4, MODE>(a, taken, grid, s);
    return st;
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
