// Shared host/device helpers of libqknorm: error reporting, alignment checks,
// bf16 <-> fp32 conversion of 16-byte chunks, and streaming memory accesses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qknorm.h"

namespace qkn {

// Thread-local message behind qkn_last_error(); returns `st` for chaining.
qkn_status fail(qkn_status st, const char *fmt, ...);

// Maps a CUDA runtime error to QKN_ERR_CUDA with the runtime's message.
qkn_status cuda_fail(cudaError_t e, const char *what);

// Checks the launch(es) just issued; QKN_OK when the runtime reports none.
qkn_status check_launch(const char *what);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Rows of a call's operand or result: `rows` of `bytes`, `pitch` bytes apart.
struct Span {
    const void *p;
    int64_t rows, bytes, pitch;
};

// sum over 0 <= i < n of floor((a i + b) / m), in a number of steps logarithmic in a and m: whole
// parts of a / m and b / m add up directly, what is left counts the lattice points under a line, with
// the axes exchanged.
inline unsigned __int128 floor_sum(unsigned __int128 n, unsigned __int128 m, unsigned __int128 a, unsigned __int128 b) {
    unsigned __int128 sum = 0;
    while (true) {
        sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
        a %= m;
        const unsigned __int128 top = a * n + b % m;
        if (top < m) return sum;
        n = top / m;
        b = top % m;
        const unsigned __int128 t = a;
        a = m;
        m = t;
    }
}

// Whether any row of a shares a byte with a row of b.  Columns of one wider buffer do not, although
// their address ranges cross.  Never a walk over the rows, of which a call may have 2^31.
inline bool rows_overlap(const Span &a, const Span &b) {
    using wide = __int128;  // pitches are the caller's: rows * pitch may pass 64 bits
    if (a.p == nullptr || b.p == nullptr || a.rows < 1 || b.rows < 1 || a.bytes < 1 || b.bytes < 1) return false;
    if (a.rows > b.rows) return rows_overlap(b, a);
    const wide b0 = (wide)reinterpret_cast<uintptr_t>(b.p) - (wide)reinterpret_cast<uintptr_t>(a.p);  // from a's start
    if (b0 + (wide)(b.rows - 1) * b.pitch + b.bytes <= 0 || (wide)(a.rows - 1) * a.pitch + a.bytes <= b0) return false;
    if (a.rows > 1 && a.pitch == b.pitch) {
        const wide at = (b0 % a.pitch + a.pitch) % a.pitch;  // where b's rows begin in a's
        return at < a.bytes || at + b.bytes > a.pitch;
    }
    // a's rows between b's first byte and its last one.  One of them that meets b's rows continued in
    // both directions meets b itself: the row before b's first one, or behind its last one, is met
    // only together with that one.  Row i meets as many rows as there are j with
    // i pa - bytes(b) < b0 + j pb < i pa + bytes(a).
    const wide pa = a.rows > 1 ? a.pitch : 1, pb = b.rows > 1 ? b.pitch : 1;
    const wide first = a.rows == 1 || b0 < a.bytes ? 0 : (b0 - a.bytes) / pa + 1;
    const wide end = a.rows == 1 ? 1 : (b0 + (b.rows - 1) * pb + b.bytes - 1) / pa + 1;  // behind the last one
    const wide n = (end < a.rows ? end : a.rows) - first;
    if (n < 1) return false;
    const wide at = first * pa - b0, low = at - b.bytes, high = at + a.bytes - 1;
    const wide up = low < 0 ? (-low / pb + 1) * pb : 0;  // whole rows, so that nothing is negative
    return floor_sum(n, pb, pa, high + up) != floor_sum(n, pb, pa, low + up);
}

// The same rows: a result that replaces its operand in place.
inline bool same_rows(const Span &a, const Span &b) {
    return a.p == b.p && a.rows == b.rows && a.bytes == b.bytes && (a.rows <= 1 || a.pitch == b.pitch);
}

// A vector or a workspace of `bytes`.
inline Span flat(const void *p, int64_t bytes) { return {p, 1, bytes, bytes}; }

inline size_t dtype_size(qkn_dtype t) { return t == QKN_F32 ? 4 : 2; }

inline bool valid_dtype(int t) { return t == QKN_F32 || t == QKN_BF16; }

// n_seg within [1, QKN_MAX_SEG], else QKN_ERR_SHAPE with a message.
inline qkn_status check_seg(int n_seg) {
    if (n_seg < 1 || n_seg > QKN_MAX_SEG) return fail(QKN_ERR_SHAPE, "n_seg=%d outside [1, %d]", n_seg, QKN_MAX_SEG);
    return QKN_OK;
}

// Number of SMs of the current device (cached per device).
int sm_count();

// Reads the norm kernels' device error word into *flag and clears it.
qkn_status read_norm_error(int *flag);

// ---------------------------------------------------------------- device side

// Streaming 16-byte load: data read once, evict-first in L1 and L2.
__device__ __forceinline__ uint4 ld_stream(const void *p) {
    return __ldcs(reinterpret_cast<const uint4 *>(p));
}

// Streaming 16-byte store.  Volatile asm keeps stores in program order with
// the other volatile accesses below, which bounds register pressure.
__device__ __forceinline__ void st_stream(void *p, uint4 v) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w) : "memory");
}

// Cached read-only 16- and 8-byte loads kept in program order (see st_stream).
__device__ __forceinline__ uint4 ld_ro_v4(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ld_ro_v2(const void *p) {
    uint2 r;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// bf16 bit pattern (low / high half of a 32-bit word) -> fp32, exact.
__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 -> packed bf16x2 with round-to-nearest-even (lo in the low half).
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&h);
}

// A 16-byte chunk of activations of type T as fp32 values.
template <typename T> struct Chunk;

template <> struct Chunk<float> {
    static constexpr int E = 4;
    __device__ __forceinline__ static void unpack(const uint4 &v, float (&f)[E]) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static void unpack_again(const uint4 &v, float (&f)[E]) { unpack(v, f); }
    __device__ __forceinline__ static uint4 pack(const float (&f)[E]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                          __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <> struct Chunk<__nv_bfloat16> {
    static constexpr int E = 8;
    __device__ __forceinline__ static void unpack(const uint4 &v, float (&f)[E]) {
        f[0] = bf16lo(v.x); f[1] = bf16hi(v.x); f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
        f[4] = bf16lo(v.z); f[5] = bf16hi(v.z); f[6] = bf16lo(v.w); f[7] = bf16hi(v.w);
    }
    // Same values as unpack(), formed with byte permutes: a second unpack of a
    // chunk is then recomputed rather than kept live from the first one.
    __device__ __forceinline__ static void unpack_again(const uint4 &v, float (&f)[E]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(__byte_perm(w[i], 0u, 0x1044u));
            f[2 * i + 1] = __uint_as_float(__byte_perm(w[i], 0u, 0x3244u));
        }
    }
    __device__ __forceinline__ static uint4 pack(const float (&f)[E]) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
};

// Loads E consecutive weights of type TW (read-only path, cached) as fp32.
template <typename TW, int E>
__device__ __forceinline__ void load_weights(const TW *w, float (&f)[E]);

template <>
__device__ __forceinline__ void load_weights<float, 4>(const float *w, float (&f)[4]) {
    Chunk<float>::unpack(ld_ro_v4(w), f);
}
template <>
__device__ __forceinline__ void load_weights<float, 8>(const float *w, float (&f)[8]) {
    uint4 a = ld_ro_v4(w), b = ld_ro_v4(w + 4);
    f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
}
template <>
__device__ __forceinline__ void load_weights<__nv_bfloat16, 8>(const __nv_bfloat16 *w, float (&f)[8]) {
    Chunk<__nv_bfloat16>::unpack(ld_ro_v4(w), f);
}
template <>
__device__ __forceinline__ void load_weights<__nv_bfloat16, 4>(const __nv_bfloat16 *w, float (&f)[4]) {
    uint2 a = ld_ro_v2(w);
    f[0] = bf16lo(a.x); f[1] = bf16hi(a.x); f[2] = bf16lo(a.y); f[3] = bf16hi(a.y);
}

// Same values as load_weights, through plain read-only-path intrinsics that
// the compiler may batch and hoist (for kernels with registers to spare).
template <typename TW, int E>
__device__ __forceinline__ void load_weights_batched(const TW *w, float (&f)[E]) {
    if constexpr (sizeof(TW) * E == 16) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(w));
        if constexpr (E == 8) {
            Chunk<__nv_bfloat16>::unpack(a, f);
        } else {
            Chunk<float>::unpack(a, f);
        }
    } else if constexpr (sizeof(TW) * E == 32) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(w));
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(w) + 1);
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2 *>(w));
        f[0] = bf16lo(a.x); f[1] = bf16hi(a.x); f[2] = bf16lo(a.y); f[3] = bf16hi(a.y);
    }
}

// Streaming 16-byte store through the intrinsic (freely schedulable).
__device__ __forceinline__ void st_stream_batched(void *p, uint4 v) {
    __stcs(reinterpret_cast<uint4 *>(p), v);
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

}  // namespace qkn
