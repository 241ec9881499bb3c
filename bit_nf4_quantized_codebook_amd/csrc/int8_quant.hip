// Row-wise 8-bit integer quantization and the bf16 expansion of an Int8 weight (gfx950).
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net),
// section 3.1 eq. (1) (absmax Int8, here one constant per row) and eq. (2).
//
// Bound by HBM: float32 rows 40 us at 11008 x 4096 (225 MB, 5.6 TB/s), bf16 rows 7.0 us at 777 x 8192 (19 MB;
// 9.4 us with 37 VALU operations per element, int8.h).

#include "common.h"
#include "int8.h"
#include "launch.h"
#include "reduce.h"
#include "transpose.h"

namespace nf4k {

namespace {

template <bool F32>
__global__ __launch_bounds__(256) void int8_rows_kernel(const void *__restrict__ x, int64_t rows, int64_t cols,
                                                        int8_t *__restrict__ codes, float *__restrict__ scales) {
    int8_rows_block<F32>(x, blockIdx.x, rows, cols, codes, scales);
}

// The short jobs first, so that they run alongside the rows instead of trailing them.
struct PrepArgs {
    const uint16_t *X;
    int64_t M, K;
    int8_t *Xq;
    float *xs;
    RedProb red;
    const uint16_t *L2;
    uint16_t *L2T;
    int32_t r;
    int64_t N;
    uint32_t ntr, nred;
};
__global__ __launch_bounds__(256) void int8_prep_kernel(PrepArgs g) {
    if (blockIdx.x < g.ntr) {
        transpose_block(g.L2, g.L2T, g.r, g.N, blockIdx.x);
        return;
    }
    if (blockIdx.x < g.ntr + g.nred) {
        reduce_partials_block(g.red, blockIdx.x - g.ntr, g.nred);
        return;
    }
    int8_rows_block<false>(g.X, blockIdx.x - g.ntr - g.nred, g.M, g.K, g.Xq, g.xs);
}

__device__ __forceinline__ float sext8(uint32_t w, int i) { return (float)((int32_t)(w << (24 - 8 * i)) >> 24); }

// out[n, k] = bf16(scales[n] * codes[n, k]), 8 elements per thread and step
__global__ __launch_bounds__(256) void int8_expand_rows_kernel(const int8_t *__restrict__ codes,
                                                               const float *__restrict__ scales, int64_t rows,
                                                               int64_t cols, uint16_t *__restrict__ out) {
    const int64_t c8 = cols >> 3, n8 = rows * c8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
        const uint2 v = reinterpret_cast<const uint2 *>(codes)[i];
        const float s = scales[i / c8];
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f[k] = s * sext8(v.x, k);
            f[4 + k] = s * sext8(v.y, k);
        }
        reinterpret_cast<u32x4 *>(out)[i] = pack8_bf16(f);
    }
}

// out[k, n] = bf16(scales[n] * codes[n, k]), one tile of 128 weight rows by 128 columns per workgroup,
// turned through LDS.  Thread t takes rows 2 p and 2 p + 1 (p = t / 4) of the tile and 32 columns from
// 32 q (q = t % 4); it writes the bf16 pairs (row 2p, row 2p + 1) of each column into an LDS tile
// [128 columns][64 pairs], and 16 lanes write each column's 128 rows out, 16 bytes each.  In the tile the
// 16-byte group of four pairs is XOR-ed with 4 q, so that a wave's 16 pairs by 4 column ranges land on 64
// banks.  N % 8 == 0 and K % 64 == 0: pairs, groups of 8 rows and ranges of 32 columns are whole.
// Bound by HBM: 1 byte read and 2 written per weight.
struct ExpandTArgs {
    const int8_t *codes;
    const float *scales;
    int64_t N, K;
    uint16_t *out;
    RedProb red;             // nred workgroups more, the first of the launch: a pending reduction
    uint32_t nred;
};
constexpr int ET = 128;
__global__ __launch_bounds__(256) void int8_expand_transposed_kernel(ExpandTArgs g) {
    __shared__ __align__(16) uint32_t tile[ET * (ET / 2)];
    if (blockIdx.x < g.nred) {
        reduce_partials_block(g.red, blockIdx.x, g.nred);
        return;
    }
    const int64_t tb = blockIdx.x - g.nred, ntn = (g.N + ET - 1) / ET;
    const int64_t n0 = (tb % ntn) * ET, k0 = (tb / ntn) * ET;
    const int t = threadIdx.x;
    {
        const int p = t >> 2, q = t & 3;
        const int64_t n = n0 + 2 * p, k = k0 + 32 * q;
        if (n < g.N && k < g.K) {
            const u32x4 *pa = reinterpret_cast<const u32x4 *>(g.codes + n * g.K + k);
            const u32x4 *pb = reinterpret_cast<const u32x4 *>(g.codes + (n + 1) * g.K + k);
            const u32x4 a[2] = {pa[0], pa[1]}, b[2] = {pb[0], pb[1]};
            const float sa = g.scales[n], sb = g.scales[n + 1];
            uint32_t *col = tile + (((p >> 2) ^ (4 * q)) * 4 + (p & 3));
#pragma unroll
            for (int i = 0; i < 32; ++i)
                col[(32 * q + i) * (ET / 2)] = pack_bf16x2(sa * sext8(a[i >> 4][(i >> 2) & 3], i & 3),
                                                           sb * sext8(b[i >> 4][(i >> 2) & 3], i & 3));
        }
    }
    __syncthreads();
    const int c = t & 15, r16 = t >> 4;
    const int64_t n = n0 + 8 * c;
#pragma unroll
    for (int it = 0; it < ET / 16; ++it) {
        const int kk = r16 + 16 * it;
        if (k0 + kk < g.K && n < g.N)
            *reinterpret_cast<u32x4 *>(g.out + (k0 + kk) * g.N + n) =
                *reinterpret_cast<const u32x4 *>(tile + kk * (ET / 2) + ((c ^ (4 * (kk >> 5))) * 4));
    }
}

}  // namespace

hipError_t launch_int8_rows(const void *x, bool f32, int64_t rows, int64_t cols, int8_t *codes, float *scales,
                            hipStream_t stream) {
    for (int64_t r0 = 0; r0 < rows; r0 += kMaxRowGrid) {
        const int64_t n = rows - r0 < kMaxRowGrid ? rows - r0 : kMaxRowGrid;
        const char *xr = reinterpret_cast<const char *>(x) + r0 * cols * (f32 ? 4 : 2);
        const dim3 grid((unsigned)int8_rows_blocks(n, cols));
        if (f32)
            hipLaunchKernelGGL(int8_rows_kernel<true>, grid, dim3(256), 0, stream, xr, n, cols, codes + r0 * cols, scales + r0);
        else
            hipLaunchKernelGGL(int8_rows_kernel<false>, grid, dim3(256), 0, stream, xr, n, cols, codes + r0 * cols, scales + r0);
    }
    return hipGetLastError();
}

hipError_t launch_int8_prep(const Int8Prep &p, hipStream_t stream) {
    PrepArgs a{};
    a.X = p.X; a.M = p.M; a.K = p.K; a.Xq = p.Xq; a.xs = p.xs;
    a.L2 = p.L2; a.L2T = p.L2T; a.r = p.r; a.N = p.N;
    if (p.L2) a.ntr = transpose_blocks(p.r, p.N);
    if (p.Tred) a.red = red_prob(*p.Tred, a.nred);
    // X stays below 2 GiB with at least 64 columns: fewer than 2^24 rows, 2^30 threads
    const int64_t grid = (int64_t)a.ntr + a.nred + (p.X ? int8_rows_blocks(p.M, p.K) : 0);
    if (grid == 0) return hipSuccess;
    if (grid >= (int64_t)1 << 24) return hipErrorInvalidValue;
    hipLaunchKernelGGL(int8_prep_kernel, dim3((unsigned)grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_int8_expand(const Int8View &w, bool transposed, uint16_t *out, const Reduction *red, hipStream_t stream) {
    if (!transposed) {
        if (red) return hipErrorInvalidValue;
        int64_t grid = ((w.rows * w.cols >> 3) + 255) / 256;
        if (grid > 256 * 64) grid = 256 * 64;
        hipLaunchKernelGGL(int8_expand_rows_kernel, dim3((unsigned)grid), dim3(256), 0, stream, w.codes, w.scales,
                           w.rows, w.cols, out);
    } else {
        ExpandTArgs a{};
        a.codes = w.codes; a.scales = w.scales; a.N = w.rows; a.K = w.cols; a.out = out;
        if (red) a.red = red_prob(*red, a.nred);
        const int64_t tiles = ((w.rows + ET - 1) / ET) * ((w.cols + ET - 1) / ET);
        hipLaunchKernelGGL(int8_expand_transposed_kernel, dim3((unsigned)tiles + a.nred), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace nf4k
