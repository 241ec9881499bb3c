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
    float scale;     // what is stored: fp32(a / 127), or NaN for a row that is not finite
    float step;      // scale times mul: the quotient's divisor, a normal number
    float inv;       // about 1 / step
    float mul;       // 2^64 where the constant is so small that 1 / scale would overflow, else 1
};
__device__ __forceinline__ RowCode row_code(uint32_t amax_bits) {
    RowCode c;
    const bool finite = amax_bits < 0x7F800000u;
    c.scale = finite ? __uint_as_float(amax_bits) / 127.0f : __uint_as_float(0x7FC00000u);
    c.mul = c.scale < 0x1p-100f ? 0x1p64f : 1.0f;
    c.step = c.scale * c.mul;
    c.inv = (finite && c.scale > 0.0f) ? 1.0f / c.step : 0.0f;
    return c;
}
// Nearest integer to the real quotient x / step, ties to even.  r = rint(fp32 quotient) is at most
// one off next to a border, and e = x - r step has no rounding: for |x| >= step both terms are
// multiples of step's last place and e is below step; for |x| < step r is 0, or +-1 with x within a
// factor of two of step.  So comparing e with step / 2 decides the border exactly.
__device__ __forceinline__ float code_f32(float x, const RowCode &c) {
    const float xs = x * c.mul;
    float r = __builtin_rintf(xs * c.inv);
    const float e = __builtin_fmaf(-r, c.step, xs);
    const float d = __builtin_fabsf(e) - 0.5f * c.step;     // sign exact: both are floats
    const bool odd = ((int32_t)r & 1) != 0;
    const bool off = d > 0.0f || (d == 0.0f && odd);
    r += off ? __builtin_copysignf(1.0f, e) : 0.0f;
    r = __builtin_fminf(__builtin_fmaxf(r, -127.0f), 127.0f);
    return r;
}
// Eight codes as bytes.  Rows without a usable constant (inv = 0) store zeros.
__device__ __forceinline__ uint2 codes8(const float x[8], const RowCode &c) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = c.inv != 0.0f ? code_f32(x[i], c) : 0.0f;
        b[i] = (uint32_t)(int32_t)r & 0xFFu;
    }
    return uint2{b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24), b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24)};
}

template <bool F32>
__device__ __forceinline__ void load8(const void *x, int64_t i8, float f[8]) {
    if (F32) {
        typedef float f32v4 __attribute__((ext_vector_type(4)));
        const f32v4 a = reinterpret_cast<const f32v4 *>(x)[2 * i8], b = reinterpret_cast<const f32v4 *>(x)[2 * i8 + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    } else {
        unpack8_bf16(reinterpret_cast<const u32x4 *>(x)[i8], f);
    }
}

// One row per workgroup of 256 threads, the row read twice.
template <bool F32>
__device__ __forceinline__ void int8_row(const void *__restrict__ x, int64_t row, int64_t cols, int8_t *__restrict__ codes,
                                         float *__restrict__ scales) {
    __shared__ uint32_t red[4];
    const int64_t c8 = cols >> 3;
    const int tid = threadIdx.x;
    uint32_t m = 0;
    for (int64_t i = tid; i < c8; i += 256) {
        float f[8];
        load8<F32>(x, row * c8 + i, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(f[k]) & 0x7FFFFFFFu);
    }
    m = wave_max(m);
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    m = max(max(red[0], red[1]), max(red[2], red[3]));
    const RowCode rc = row_code(m);
    if (tid == 0) scales[row] = rc.scale;
    for (int64_t i = tid; i < c8; i += 256) {
        float f[8];
        load8<F32>(x, row * c8 + i, f);
        reinterpret_cast<uint2 *>(codes)[row * c8 + i] = codes8(f, rc);
    }
}

}  // namespace nf4k
