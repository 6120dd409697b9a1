// Unit kernel of the rotary entry points: rows of 16-byte chunks, persistent,
// fed by bulk copies.
//
// Included by rotary.cu only (one translation unit: its device error word,
// Args and helpers).
//
// The work is all HBM: every row is read once and written once (gradients:
// x and dy read, dx written).  A token's rows (q and k together) are handled
// by a group of G warps; a block holds NG groups that never wait for one
// another.  Each group owns a ring of stages in shared memory, one token per
// stage, filled by 1-D bulk copies that run while earlier tokens are
// computed.
//
// A thread owns the same columns of every token: UPT "units" of two 16-byte
// chunks, chunk j and chunk j + r / 2E of a head (E elements per chunk).  In
// the half layout the two chunks hold the two sides of E pairs; in the
// interleaved layout each holds E / 2 whole pairs.  Either way a unit needs
// the cos and sin of two runs of E / 2 frequencies, which the group's table
// keeps at positions j and j + r / 2E (filled in the order the layout asks
// for), so the arithmetic below is the same for both and neighbouring threads
// read neighbouring 16-byte words.  Chunks behind the rotated part form units
// of their own, copied (or only normalised).  Fixed columns keep the weights,
// and the weights' gradients, in registers over all tokens.
//
// One barrier per token: before it, threads read their chunks, add up squares
// and park the warp's sums, and fill the table of the NEXT token; after it
// the stage is free (every thread holds its chunks in registers) and is
// refilled, the row's factor is formed and the results are stored.  Sums are
// double-buffered and tables triple-buffered by token, which one barrier per
// token makes safe.
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
    int warps, groups;       // warps per group, groups per block
    int stages, stage_bytes, x_bytes;
    uint64_t wait_ns;
};

inline __host__ __device__ int table_bytes(int r) { return 3 * r * 4; }          // cos and sin of 3 tokens
inline __host__ __device__ int red_bytes(int warps) { return 2 * warps * 16; }   // 2 x 4 sums per warp
inline __host__ __device__ int group_fixed(int r, int warps, int stages) {
    return (table_bytes(r) + 15) / 16 * 16 + red_bytes(warps) + (stages + 1) / 2 * 16;
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

// Barrier of a group, true on every thread when any of them failed.
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

// H = E / 2 consecutive floats of the table.
template <int H>
__device__ __forceinline__ void lds_run(uint32_t addr, float (&f)[H]) {
    if constexpr (H == 4)
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(addr));
    else
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f[0]), "=f"(f[1]) : "r"(addr));
}

// The two chunks of a unit, turned.
template <int E, bool HALF>
__device__ __forceinline__ void turn(float (&a)[E], float (&b)[E], uint32_t cos_addr, uint32_t run, uint32_t sin_off) {
    constexpr int H = E / 2;
    float c0[H], s0[H], c1[H], s1[H];
    lds_run<H>(cos_addr, c0);
    lds_run<H>(cos_addr + run, c1);
    lds_run<H>(cos_addr + sin_off, s0);
    lds_run<H>(cos_addr + sin_off + run, s1);
    if constexpr (HALF) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float c = e < H ? c0[e % H] : c1[e % H], s = e < H ? s0[e % H] : s1[e % H];
            const float x = a[e], y = b[e];
            a[e] = x * c - y * s;
            b[e] = y * c + x * s;
        }
    } else {
#pragma unroll
        for (int e = 0; e < H; ++e) {
            const float x = a[2 * e], y = a[2 * e + 1], z = b[2 * e], w = b[2 * e + 1];
            a[2 * e] = x * c0[e] - y * s0[e];
            a[2 * e + 1] = y * c0[e] + x * s0[e];
            b[2 * e] = z * c1[e] - w * s1[e];
            b[2 * e + 1] = w * c1[e] + z * s1[e];
        }
    }
}

// The weights of a chunk, as they are stored.
template <typename TW, int E> struct RawWeights {
    static constexpr int N = E * (int)sizeof(TW) / 4;
    uint32_t v[N];
    __device__ __forceinline__ void load(const void *w, int element) {
        const uint32_t *p = reinterpret_cast<const uint32_t *>(static_cast<const TW *>(w) + element);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __ldg(p + i);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0u;
    }
    __device__ __forceinline__ float get(int e) const {
        if constexpr (sizeof(TW) == 4) return __uint_as_float(v[e]);
        else return (e & 1) ? bf16hi(v[e >> 1]) : bf16lo(v[e >> 1]);
    }
};

template <typename TA, typename TW, int MODE, int UPT, bool HALF>
__global__ void __launch_bounds__(kMaxThreads, (MODE == kNormBack || UPT == 4) ? 1 : 2)
rotary_unit_kernel(const Params a) {
    constexpr int E = Chunk<TA>::E, H = E / 2;
    constexpr bool NORM = MODE != kRotate, BACK = MODE == kNormBack;
    extern __shared__ __align__(128) uint8_t smem[];
    const int threads = a.warps * 32;
    const int group = threadIdx.x / threads, gt = threadIdx.x - group * threads;  // thread within its group
    const int lane = threadIdx.x & 31, gw = gt >> 5;
    const int fixed = group_fixed(a.r, a.warps, a.stages);
    uint8_t *ring_p = smem + (size_t)group * a.stages * a.stage_bytes;
    uint8_t *fix_p = smem + (size_t)a.groups * a.stages * a.stage_bytes + (size_t)group * fixed;
    const uint32_t ring = smem_u32(ring_p);
    float *table = reinterpret_cast<float *>(fix_p);
    float4 *red = reinterpret_cast<float4 *>(fix_p + (table_bytes(a.r) + 15) / 16 * 16);
    const uint32_t bars = smem_u32(red + 2 * a.warps);
    const uint32_t table_s = smem_u32(table);
    const uint32_t sin_off = (uint32_t)a.r * 2u, run = (uint32_t)a.rot_units * H * 4u;  // bytes

    if (gt == 0) {
        for (int s = 0; s < a.stages; ++s) mbar_init(bars + 8u * s, 1);
        mbar_init_fence();
    }

    // this thread's units
    int off_a[UPT], off_b[UPT], tab[UPT];  // stage offsets of the chunks (-1: none), table offset (-1: not turned)
    uint32_t is_k = 0;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
        int u = gt + i * threads;
        off_a[i] = off_b[i] = tab[i] = -1;
        const int which = u >= a.job[0].nunits ? 1 : 0;
        if (which) {
            u -= a.job[0].nunits;
            is_k |= 1u << i;
        }
        if (which >= a.njobs || u >= (which ? a.job[1].nunits : a.job[0].nunits)) continue;
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

    // the previous kernel on the stream has finished before any memory is touched
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t step = (int64_t)gridDim.x * a.groups;
    const int64_t first_token = (int64_t)blockIdx.x * a.groups + group;
    __syncthreads();  // barriers initialised

    auto issue = [&](int64_t n, int stage) {
        const uint32_t bar = bars + 8u * stage, dst = ring + (uint32_t)(stage * a.stage_bytes);
        mbar_arrive_expect_tx(bar, (uint32_t)a.stage_bytes);
        bulk_g2s(dst, a.job[0].x + n * a.job[0].ldx, a.job[0].row_bytes, bar);
        if (BACK) bulk_g2s(dst + a.x_bytes, a.job[0].g + n * a.job[0].ldg, a.job[0].row_bytes, bar);
        if (a.njobs > 1) {
            bulk_g2s(dst + a.job[1].row_off, a.job[1].x + n * a.job[1].ldx, a.job[1].row_bytes, bar);
            if (BACK)
                bulk_g2s(dst + a.x_bytes + a.job[1].row_off, a.job[1].g + n * a.job[1].ldg, a.job[1].row_bytes, bar);
        }
    };
    int64_t issued = 0;  // stages filled so far (thread 0 of the group)
    if (gt == 0)
        for (int64_t n = first_token; issued < a.stages && n < a.T; n += step) issue(n, (int)issued), ++issued;

    RawWeights<TW, E> wa[UPT], wb[UPT];
    if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const bool k = (is_k >> i) & 1u;
            const void *w = k ? a.job[1].w : a.job[0].w;
            const int ro = k ? a.job[1].row_off : 0;
            if (off_a[i] >= 0) wa[i].load(w, (off_a[i] - ro) / 16 * E);
            else wa[i].clear();
            if (off_b[i] >= 0) wb[i].load(w, (off_b[i] - ro) / 16 * E);
            else wb[i].clear();
        }
    }
    float da[UPT][E], db[UPT][E];  // gradients of the weights, over this group's tokens
    if constexpr (BACK) {
#pragma unroll
        for (int i = 0; i < UPT; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) da[i][e] = db[i][e] = 0.f;
    }

    // cos and sin of a token: frequency f sits in run f / H, at the run's place in the layout's order
    const int nf = a.r >> 1;
    auto place = [&](int f) {
        const int q = f / H;
        return (HALF ? (q & 1) * a.rot_units + (q >> 1) : q) * H + f % H;
    };
    const double turns0 = gt < nf ? __ldg(a.freq + gt) * kInvTwoPi : 0.0;
    const int place0 = place(gt);
    auto fill = [&](int64_t p, int buf) {
        float *t = table + buf * a.r;
        if (gt < nf) cos_sin(p, turns0, a.mscale, a.sign, t[place0], t[nf + place0]);
        for (int f = gt + threads; f < nf; f += threads)
            cos_sin(p, __ldg(a.freq + f) * kInvTwoPi, a.mscale, a.sign, t[place(f)], t[nf + place(f)]);
    };
    auto pos_at = [&](int64_t n) -> int64_t {
        if (a.r == 0 || n >= a.T) return 0;
        return a.pos64 ? __ldg(static_cast<const long long *>(a.pos) + n) : (int64_t)__ldg(static_cast<const int *>(a.pos) + n);
    };
    int64_t next_pos = pos_at(first_token + step);
    if (first_token < a.T) fill(pos_at(first_token), 0);
    if (BACK || !NORM) group_sync_or(false, group, a.warps);  // the first table is read before the first token's barrier

    int stage = 0, buf = 0, par = 0;
    uint32_t phase = 0;
    int64_t it = 0, n = first_token;
    for (; n < a.T; n += step, ++it) {
        const bool ok = mbar_wait_fast(bars + 8u * stage, phase, &g_rotary_error, a.wait_ns);
        const uint32_t src = ring + (uint32_t)(stage * a.stage_bytes);
        uint4 xa[UPT], xb[UPT];
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            xa[i] = off_a[i] >= 0 ? lds128(src + off_a[i]) : make_uint4(0u, 0u, 0u, 0u);
            xb[i] = off_b[i] >= 0 ? lds128(src + off_b[i]) : make_uint4(0u, 0u, 0u, 0u);
        }
        float ga[UPT][E], gb[UPT][E];  // gradients turned back
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);  // sums of x^2 (q, k), of w g x (q, k)
        const uint32_t tab_s = table_s + (uint32_t)(buf * a.r) * 4u;
        if constexpr (NORM) {
#pragma unroll
            for (int i = 0; i < UPT; ++i) {
                float fa[E], fb[E];
                Chunk<TA>::unpack(xa[i], fa);
                Chunk<TA>::unpack(xb[i], fb);
                float sq = 0.f, pg = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) sq = fmaf(fa[e], fa[e], sq);
#pragma unroll
                for (int e = 0; e < E; ++e) sq = fmaf(fb[e], fb[e], sq);
                if constexpr (BACK) {
                    Chunk<TA>::unpack(off_a[i] >= 0 ? lds128(src + a.x_bytes + off_a[i]) : make_uint4(0u, 0u, 0u, 0u), ga[i]);
                    Chunk<TA>::unpack(off_b[i] >= 0 ? lds128(src + a.x_bytes + off_b[i]) : make_uint4(0u, 0u, 0u, 0u), gb[i]);
                    if (tab[i] >= 0) turn<E, HALF>(ga[i], gb[i], tab_s + tab[i], run, sin_off);
#pragma unroll
                    for (int e = 0; e < E; ++e) pg = fmaf(fa[e] * ga[i][e], wa[i].get(e), pg);
#pragma unroll
                    for (int e = 0; e < E; ++e) pg = fmaf(fb[e] * gb[i][e], wb[i].get(e), pg);
                }
                const bool k = (is_k >> i) & 1u;
                acc.x += k ? 0.f : sq;
                acc.y += k ? sq : 0.f;
                acc.z += k ? 0.f : pg;
                acc.w += k ? pg : 0.f;
            }
            for (int off = 16; off > 0; off >>= 1) {
                acc.x += __shfl_xor_sync(0xffffffffu, acc.x, off);
                acc.y += __shfl_xor_sync(0xffffffffu, acc.y, off);
                if constexpr (BACK) {
                    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, off);
                    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, off);
                }
            }
            if (a.warps > 1 && lane == 0) red[par * a.warps + gw] = acc;
        }
        const int next_buf = buf == 2 ? 0 : buf + 1;
        if (a.r != 0 && n + step < a.T) {
            fill(next_pos, next_buf);
            next_pos = pos_at(n + 2 * step);
        }
        if (group_sync_or(!ok, group, a.warps)) break;
        if (gt == 0 && n + (int64_t)a.stages * step < a.T) {
            issue(n + (int64_t)a.stages * step, stage);
            ++issued;
        }
        float inv_q = 1.f, inv_k = 1.f, cq = 0.f, ck = 0.f;
        if constexpr (NORM) {
            if (a.warps > 1) {
                acc = red[par * a.warps];
                for (int w = 1; w < a.warps; ++w) {
                    const float4 v = red[par * a.warps + w];
                    acc.x += v.x;
                    acc.y += v.y;
                    if constexpr (BACK) {
                        acc.z += v.z;
                        acc.w += v.w;
                    }
                }
            }
            inv_q = rsqrtf(acc.x / (float)a.job[0].d + a.eps);
            inv_k = a.njobs > 1 ? rsqrtf(acc.y / (float)a.job[1].d + a.eps) : 0.f;
            if constexpr (BACK) {
                cq = inv_q * inv_q * (acc.z / (float)a.job[0].d);
                ck = a.njobs > 1 ? inv_k * inv_k * (acc.w / (float)a.job[1].d) : 0.f;
            }
        }
        uint8_t *yq = a.job[0].y + n * a.job[0].ldy;
        uint8_t *yk = a.job[1].y + n * a.job[1].ldy - a.job[1].row_off;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            if (off_a[i] < 0) continue;
            const bool k = (is_k >> i) & 1u;
            uint8_t *y = k ? yk : yq;
            float fa[E], fb[E];
            Chunk<TA>::unpack_again(xa[i], fa);
            Chunk<TA>::unpack_again(xb[i], fb);
            if constexpr (BACK) {
                const float inv = k ? inv_k : inv_q, c = k ? ck : cq;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    da[i][e] = fmaf(ga[i][e], fa[e] * inv, da[i][e]);
                    db[i][e] = fmaf(gb[i][e], fb[e] * inv, db[i][e]);
                    fa[e] = inv * (wa[i].get(e) * ga[i][e] - fa[e] * c);
                    fb[e] = inv * (wb[i].get(e) * gb[i][e] - fb[e] * c);
                }
            } else {
                if constexpr (NORM) {
                    const float inv = k ? inv_k : inv_q;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        fa[e] = (fa[e] * inv) * wa[i].get(e);
                        fb[e] = (fb[e] * inv) * wb[i].get(e);
                    }
                }
                if (tab[i] >= 0) turn<E, HALF>(fa, fb, tab_s + tab[i], run, sin_off);
            }
            st_stream_batched(y + off_a[i], Chunk<TA>::pack(fa));
            if (off_b[i] >= 0) st_stream_batched(y + off_b[i], Chunk<TA>::pack(fb));
        }
        if (++stage == a.stages) {
            stage = 0;
            phase ^= 1u;
        }
        buf = next_buf;
        par ^= 1;
    }
    // after a wait that gave up: no copy may still be writing when the block exits
    if (gt == 0 && n < a.T)
        for (int64_t i = it; i < issued; ++i)
            mbar_wait(bars + 8u * (uint32_t)(i % a.stages), (uint32_t)(i / a.stages) & 1u, &g_rotary_error, a.wait_ns);

    if constexpr (BACK) {
        // one row of partial sums per block: the groups' sums meet in the ring, added in group order
        const int dq = a.job[0].d, d = dq + (a.njobs > 1 ? a.job[1].d : 0);
        float *out = a.part + (int64_t)blockIdx.x * d;
        float *mine = a.groups > 1 ? reinterpret_cast<float *>(smem) + (size_t)group * d : out;
        __syncthreads();  // every group has read its last stage
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            if (off_a[i] < 0) continue;
            const bool k = (is_k >> i) & 1u;
            const int col = k ? dq : 0, ro = k ? a.job[1].row_off : 0;
            float *pa = mine + col + (off_a[i] - ro) / 16 * E;
#pragma unroll
            for (int e = 0; e < E; ++e) pa[e] = da[i][e];
            if (off_b[i] >= 0) {
                float *pb = mine + col + (off_b[i] - ro) / 16 * E;
#pragma unroll
                for (int e = 0; e < E; ++e) pb[e] = db[i][e];
            }
        }
        if (a.groups > 1) {
            __syncthreads();
            const float *all = reinterpret_cast<const float *>(smem);
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
    int upt, warps, groups, ctas, stages, stage_bytes, x_bytes, smem;
};

constexpr int kMaxCtas = 4;  // blocks per SM at most (the partial gradients' rows are sized by it)

// Whether the unit kernel takes the call, and its geometry: a rule on the
// rows' widths, types and alignment, never on the number of tokens.
template <typename TA, typename TW, int MODE>
Plan plan(const Args &a, Params &p) {
    constexpr int E = Chunk<TA>::E;
    Plan r{};
    p.x_bytes = 0;
    int units = 0;
    for (int i = 0; i < a.njobs; ++i) {
        const Job &j = a.job[i];
        Rows &J = p.job[i];
        const int D = a.r ? a.D : j.d;
        if (D % E != 0 || a.r % (2 * E) != 0 || !aligned(j.x, 16) || !aligned(j.y, 16) || j.ldx % 16 || j.ldy % 16)
            return r;
        if (MODE == kNormBack && (!aligned(j.g, 16) || j.ldg % 16)) return r;
        if (MODE != kRotate && !aligned(j.w, 4)) return r;
        J.x = j.x;
        J.g = j.g;
        J.y = j.y;
        J.w = j.w;
        J.ldx = j.ldx;
        J.ldg = j.ldg;
        J.ldy = j.ldy;
        J.d = j.d;
        if ((int64_t)j.d * (int64_t)sizeof(TA) > kSmemLimit) return r;
        J.row_bytes = j.d * (int)sizeof(TA);
        J.row_off = p.x_bytes;
        p.x_bytes += J.row_bytes;
        J.head_chunks = D / E;
        J.tail_chunks = (D - a.r) / E;
        J.tail_units = (J.tail_chunks + 1) / 2;
        J.units_per_head = a.r / (2 * E) + J.tail_units;
        J.nunits = j.d / D * J.units_per_head;
        units += J.nunits;
    }
    if (a.njobs == 1) p.job[1] = Rows{};
    p.stage_bytes = p.x_bytes * (MODE == kNormBack ? 2 : 1);
    p.rot_units = a.r / (2 * E);
    r.upt = units <= 32 ? 1 : 2;
    if (MODE != kNormBack && units > 32 * 2 * 16) r.upt = 4;
    r.warps = (units + 32 * r.upt - 1) / (32 * r.upt);
    if (r.warps > kMaxThreads / 32) return r;
    r.groups = r.warps == 1 ? 8 : r.warps == 2 ? 4 : r.warps <= 4 ? 2 : 1;
    const int threads = r.warps * r.groups * 32;
    const int most = MODE == kNormBack || r.upt == 4 ? 512 : 768;
    for (r.ctas = most / threads < 1 ? 1 : most / threads > kMaxCtas ? kMaxCtas : most / threads; r.ctas >= 1; --r.ctas) {
        const int budget = kSmemLimit / r.ctas - 1024;  // the system keeps 1 KiB per block
        for (r.stages = 8; r.stages >= 1; --r.stages) {
            r.smem = r.groups * (r.stages * p.stage_bytes + group_fixed(a.r, r.warps, r.stages));
            if (r.smem <= budget) break;
        }
        if (r.stages >= 2 || (r.ctas == 1 && r.stages >= 1)) {
            r.fits = true;
            return r;
        }
    }
    return r;
}

template <typename TA, typename TW, int MODE, int UPT, bool HALF>
qkn_status launch_kernel(const Params &p, int grid, int threads, int smem, cudaStream_t s) {
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    cudaGetDevice(&dev);
    const bool known = dev >= 0 && dev < 64;
    if (!known || !attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(rotary_unit_kernel<TA, TW, MODE, UPT, HALF>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(rotary_unit_kernel)");
        if (known) attr_set[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rotary_unit_kernel<TA, TW, MODE, UPT, HALF>, p);
    if (e != cudaSuccess) return cuda_fail(e, "rotary_unit_kernel launch");
    return check_launch("rotary_unit_kernel launch");
}

template <typename TA, typename TW, int MODE, int UPT>
qkn_status launch_layout(const Params &p, int layout, int grid, int threads, int smem, cudaStream_t s) {
    return layout == QKN_ROTARY_HALF ? launch_kernel<TA, TW, MODE, UPT, true>(p, grid, threads, smem, s)
                                     : launch_kernel<TA, TW, MODE, UPT, false>(p, grid, threads, smem, s);
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
    p.groups = r.groups;
    p.stages = r.stages;
    p.wait_ns = kWaitTimeoutNs;
    const int64_t need = (a.T + r.groups - 1) / r.groups, cap = (int64_t)r.ctas * sm_count();
    *grid = (int)(need < cap ? need : cap);
    const int threads = r.warps * r.groups * 32;
    if (r.upt == 1) return launch_layout<TA, TW, MODE, 1>(p, a.layout, *grid, threads, r.smem, s);
    if (r.upt == 2) return launch_layout<TA, TW, MODE, 2>(p, a.layout, *grid, threads, r.smem, s);
    if constexpr (MODE != kNormBack) return launch_layout<TA, TW, MODE, 4>(p, a.layout, *grid, threads, r.smem, s);
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
