// Device helpers of the Int8 kernels (gfx950): eq. (1) of section 3.1 with one constant per row, and
// the sums over a workgroup that the row kernels share.
#pragma once

#include "common.h"

namespace nf4k {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void unpack8_bf16(const u32x4 &v, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ u32x4 pack8_bf16(const float f[8]) {
    return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// ---- sums and maxima over a wave: four DPP shifts within rows of 16, two broadcasts across rows;
// the result sits in lane 63 and is read back as a scalar ----
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp0(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ float wave_sum(float x) {
    x += __uint_as_float(dpp0<0x111, 0xF>(__float_as_uint(x)));
    x += __uint_as_float(dpp0<0x112, 0xF>(__float_as_uint(x)));
    x += __uint_as_float(dpp0<0x114, 0xF>(__float_as_uint(x)));
    x += __uint_as_float(dpp0<0x118, 0xF>(__float_as_uint(x)));
    x += __uint_as_float(dpp0<0x142, 0xA>(__float_as_uint(x)));
    x += __uint_as_float(dpp0<0x143, 0xC>(__float_as_uint(x)));
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), 63));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max(x, dpp0<0x111, 0xF>(x));
    x = max(x, dpp0<0x112, 0xF>(x));
    x = max(x, dpp0<0x114, 0xF>(x));
    x = max(x, dpp0<0x118, 0xF>(x));
    x = max(x, dpp0<0x142, 0xA>(x));
    x = max(x, dpp0<0x143, 0xC>(x));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// ---- eq. (1) for one row ----
// The row's constant from max |x|, held as float bits with the sign cleared (an integer maximum
// orders them, with infinities and NaN above every finite value).
struct RowCode {
    float scale;         // what is stored: fp32(a / 127), or NaN for a row that is not finite
    float step, inv;     // the quotient's divisor (a normal number) and about its reciprocal
    float half, below;   // step / 2 and the float below it
    float mul;           // 2^64 where the constant is so small that 1 / scale would overflow, else 1
    int mode;            // ROW_ZERO .. ROW_PLAIN
};
// ROW_ZERO: no usable constant, the codes are 0.  ROW_TINY: x and the constant times 2^64 first (exact),
// the quotient clamped (a denormal constant may be far from a / 127).  ROW_TIES: a quotient may be a
// half-integer.  ROW_PLAIN: none can be, see below.
enum { ROW_ZERO, ROW_TINY, ROW_TIES, ROW_PLAIN };
template <bool F32>
__device__ __forceinline__ RowCode row_code(uint32_t amax_bits) {
    RowCode c;
    const bool finite = amax_bits < 0x7F800000u;
    c.scale = finite ? __uint_as_float(amax_bits) / 127.0f : __uint_as_float(0x7FC00000u);
    const bool tiny = c.scale < 0x1p-100f;
    c.mul = tiny ? 0x1p64f : 1.0f;
    c.step = c.scale * c.mul;
    c.inv = 1.0f / c.step;
    c.half = 0.5f * c.step;
    c.below = __uint_as_float(__float_as_uint(c.half) - 1u);
    // x = (k + 1/2) scale exactly: 2 x is an odd number times scale, so it has at least scale's
    // significant bits.  A bf16 x has 8: no ties unless scale has at most 8 too.
    const bool ties = F32 || (__float_as_uint(c.scale) & 0xFFFFu) == 0u;
    c.mode = !finite || c.scale == 0.0f ? ROW_ZERO : (tiny ? ROW_TINY : (ties ? ROW_TIES : ROW_PLAIN));
    return c;
}
// Nearest integer to the real quotient x / step, ties to even, as a float whose low byte is the code
// (the integer plus 1.5 * 2^23).  r from the rounded quotient is at most one off, and only next to a
// border; e = x - r step has no rounding: for |x| >= step both terms are multiples of step's last
// place and e is below step; for |x| < step r is 0, or +-1 with x within a factor of two of step.  So
// comparing |e| with step / 2 decides the border exactly (for an odd r, a tie goes on to the even
// neighbour: |e| is compared with the float below).
// About 7 VALU operations per element; with a division or the conversions of a plain form (37 in all)
// the VALU and not HBM bounded the rows' quantization (4096 x 4096 bf16: 15.7 us).
template <int MODE>
__device__ __forceinline__ uint32_t code_bits(float x, const RowCode &c) {
    const float big = 12582912.0f;
    if (MODE == ROW_TINY) x *= c.mul;
    float u = __builtin_fmaf(x, c.inv, big);
    if (MODE == ROW_TINY) u = __builtin_fminf(__builtin_fmaxf(u, big - 127.0f), big + 127.0f);
    const float e = __builtin_fmaf(big - u, c.step, x);
    const float h = MODE != ROW_PLAIN && (__float_as_uint(u) & 1u) ? c.below : c.half;
    const float v = u + __builtin_copysignf(1.0f, e);
    u = __builtin_fabsf(e) > h ? v : u;
    if (MODE == ROW_TINY) u = __builtin_fminf(__builtin_fmaxf(u, big - 127.0f), big + 127.0f);
    return __float_as_uint(u);
}
template <int MODE>
__device__ __forceinline__ uint2 codes8(const float x[8], const RowCode &c) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = MODE == ROW_ZERO ? 0u : code_bits<MODE>(x[i], c);
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        o[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0C0C0400u), 0x05040100u);
    return uint2{o[0], o[1]};
}
// f(the mode as a constant) once, by the row's (uniform) mode
template <int MODE>
struct IntConst {
    static constexpr int value = MODE;
};
template <class F>
__device__ __forceinline__ void by_mode(const RowCode &c, F f) {
    const int mode = __builtin_amdgcn_readfirstlane(c.mode);
    if (mode == ROW_PLAIN) f(IntConst<ROW_PLAIN>());
    else if (mode == ROW_TIES) f(IntConst<ROW_TIES>());
    else if (mode == ROW_TINY) f(IntConst<ROW_TINY>());
    else f(IntConst<ROW_ZERO>());
}

// ---- rows to codes ----
// eight elements of a row as they lie in memory
template <bool F32>
struct Raw8 {
    u32x4 v[F32 ? 2 : 1];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = u32x4{0u, 0u, 0u, 0u};
    }
    // elements e .. e + 7 of x (e a multiple of 8); STREAM: past the caches
    template <bool STREAM = false>
    __device__ __forceinline__ void load(const void *x, int64_t e) {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(x) + e * (F32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = STREAM ? __builtin_nontemporal_load(p + i) : p[i];
    }
    __device__ __forceinline__ void floats(float f[8]) const {
        if (F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[(F32 ? 1 : 0) * (i >> 2)][i & 3]);
        } else {
            unpack8_bf16(v[0], f);
        }
    }
};
// Running maximum of |x| as bits: float32 words, or pairs of bf16 halves (one packed maximum per pair).
template <bool F32>
struct Amax {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    uint32_t m = 0;
    __device__ __forceinline__ void add(const Raw8<F32> &r) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (F32) m = max(m, r.v[i][k] & 0x7FFFFFFFu);
                else m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                               __builtin_bit_cast(u16x2, r.v[i][k] & 0x7FFF7FFFu)));
            }
    }
    // as float bits
    __device__ __forceinline__ uint32_t bits() const { return F32 ? m : max(m & 0xFFFF0000u, m << 16); }
};

// One row per TPR threads (64: a wave of its own, else the whole workgroup), held in registers as V
// pieces per thread, so that it is read once: cols <= 8 V TPR.
template <bool F32, int TPR, int V>
__device__ __forceinline__ void int8_row_regs(const void *__restrict__ x, int64_t row, int64_t cols,
                                              int8_t *__restrict__ codes, float *__restrict__ scales) {
    const int t = TPR == 64 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
    Raw8<F32> r[V];
    Amax<F32> am;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * TPR + t) * 8;
        r[v].zero();
        if (c < cols) r[v].load(x, row * cols + c);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) am.add(r[v]);
    uint32_t m = wave_max(am.bits());
    if (TPR > 64) {
        __shared__ uint32_t red[TPR / 64];
        if ((t & 63) == 0) red[t >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) m = max(m, red[w]);
    }
    const RowCode rc = row_code<F32>(m);
    if (t == 0) scales[row] = rc.scale;
    by_mode(rc, [&](auto mode) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * TPR + t) * 8;
            float f[8];
            r[v].floats(f);
            const uint2 o = codes8<decltype(mode)::value>(f, rc);
            if (c < cols) *reinterpret_cast<uint2 *>(codes + row * cols + c) = o;
        }
    });
}

// Longer rows: one workgroup of 256 threads, the row read twice.  The rows in flight are larger than the L2s
// (five workgroups a CU with 88 KB each, in float32 at 22016 columns), so the second read comes from the
// memory-side cache at best: 8192 x 22016 241 us in float32 and 143 in bf16, 3.7 TB/s of the bytes counted
// once (5.6 up to 16384 columns).
template <bool F32>
__device__ __forceinline__ void int8_row_loop(const void *__restrict__ x, int64_t row, int64_t cols,
                                              int8_t *__restrict__ codes, float *__restrict__ scales) {
    __shared__ uint32_t red[4];
    const int tid = threadIdx.x;
    Amax<F32> am;
    for (int64_t c = tid * 8; c < cols; c += 256 * 8) {
        Raw8<F32> r;
        r.load(x, row * cols + c);
        am.add(r);
    }
    uint32_t m = wave_max(am.bits());
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    const RowCode rc = row_code<F32>(m);
    if (tid == 0) scales[row] = rc.scale;
    by_mode(rc, [&](auto mode) {
        for (int64_t c = tid * 8; c < cols; c += 256 * 8) {
            Raw8<F32> r;
            float f[8];
            r.load(x, row * cols + c);
            r.floats(f);
            *reinterpret_cast<uint2 *>(codes + row * cols + c) = codes8<decltype(mode)::value>(f, rc);
        }
    });
}

// Workgroup `blk` of the rows' quantization (256 threads): four rows up to 2048 columns, else one.  The
// branch is uniform; a row of up to 16384 columns is read once.
template <bool F32>
__device__ __forceinline__ void int8_rows_block(const void *__restrict__ x, int64_t blk, int64_t rows, int64_t cols,
                                                int8_t *__restrict__ codes, float *__restrict__ scales) {
    if (cols <= 2048) {
        const int64_t row = blk * 4 + (threadIdx.x >> 6);
        if (row >= rows) return;
        if (cols <= 512) int8_row_regs<F32, 64, 1>(x, row, cols, codes, scales);
        else if (cols <= 1024) int8_row_regs<F32, 64, 2>(x, row, cols, codes, scales);
        else int8_row_regs<F32, 64, 4>(x, row, cols, codes, scales);
    } else if (cols <= 4096) {
        int8_row_regs<F32, 256, 2>(x, blk, cols, codes, scales);
    } else if (cols <= 8192) {
        int8_row_regs<F32, 256, 4>(x, blk, cols, codes, scales);
    } else if (cols <= 16384) {
        int8_row_regs<F32, 256, 8>(x, blk, cols, codes, scales);
    } else {
        int8_row_loop<F32>(x, blk, cols, codes, scales);
    }
}
inline int64_t int8_rows_blocks(int64_t rows, int64_t cols) { return cols <= 2048 ? (rows + 3) / 4 : rows; }

}  // namespace nf4k
