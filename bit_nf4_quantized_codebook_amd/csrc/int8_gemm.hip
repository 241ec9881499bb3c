// Int8 product of the Int8 QLoRA linear forward (gfx950):
//   Y[m, n] = xs[m] ws[n] sum_k Xq[m, k] Wq[n, k] + (sT L2)[m, n]
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net), section 3.1
// eq. (1) (8-bit integers), section 3.5 eq. (5), section 4 eq. (3).
//
// Block tile 64 x 64, reduction step 64, four waves of 32 x 32 with v_mfma_i32_32x32x32_i8.

#include "common.h"
#include "dqtile.h"
#include "int8.h"
#include "launch.h"

namespace nf4k {

namespace {

constexpr int BT = 64;
constexpr int PITCH = BT + 16;     // bytes of a padded LDS row

__global__ __launch_bounds__(256) void int8_gemm_kernel(Int8Product g) {
    __shared__ __align__(16) uint8_t As[BT * PITCH];
    __shared__ __align__(16) uint8_t Bs[BT * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hh = lane >> 5;
    const int64_t m0 = (int64_t)blockIdx.y * BT, n0 = (int64_t)blockIdx.x * BT;
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.Xq + m0 * g.K, (g.M - m0) * g.K);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.Wq + n0 * g.K, (g.N - n0) * g.K);
    const int row = tid >> 2, q = tid & 3;
    i32x16 acc = {};
    for (int64_t k0 = 0; k0 < g.K; k0 += BT) {
        const uint32_t off = (uint32_t)(row * g.K + k0 + 16 * q);
        const u32x4 a = bload16(rA, off), b = bload16(rB, off);
        __syncthreads();
        *reinterpret_cast<u32x4 *>(As + row * PITCH + 16 * q) = a;
        *reinterpret_cast<u32x4 *>(Bs + row * PITCH + 16 * q) = b;
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const i32x4 fa = *reinterpret_cast<const i32x4 *>(As + (wm * 32 + r32) * PITCH + s * 32 + hh * 16);
            const i32x4 fb = *reinterpret_cast<const i32x4 *>(Bs + (wn * 32 + r32) * PITCH + s * 32 + hh * 16);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa, fb, acc, 0, 0, 0);
        }
    }
    const int64_t n = n0 + wn * 32 + r32;
    if (n >= g.N) return;
    const float ws = g.ws[n];
#pragma unroll
    for (int v = 0; v < 16; ++v) {
        const int64_t m = m0 + wm * 32 + (v >> 2) * 8 + hh * 4 + (v & 3);
        if (m >= g.M) continue;
        float y = ((float)acc[v] * g.xs[m]) * ws;
        float l = 0.0f;
        for (int j = 0; j < g.r; ++j)
            l = __builtin_fmaf(bf16_to_f32(g.sT[m * g.r + j]), bf16_to_f32(g.L2[(int64_t)j * g.N + n]), l);
        g.Y[m * g.N + n] = (uint16_t)f32_to_bf16(y + l);
    }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8Product &p, hipStream_t stream) {
    timing_before(stream, 0);
    hipLaunchKernelGGL(int8_gemm_kernel, dim3((unsigned)((p.N + BT - 1) / BT), (unsigned)((p.M + BT - 1) / BT)), dim3(256), 0,
                       stream, p);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace nf4k
