// Transpose of a small bf16 matrix (an adapter's L2 [r, N] -> [N, r], so that the product's adapter
// step loads it with the reduction index contiguous), carried as extra workgroups by launches that
// run before the product.
#pragma once

#include "common.h"

namespace nf4k {

// One 64 x 64 tile of in [r, n] -> out [n, r] per workgroup of 256 threads.  Thread t loads two
// 16-byte pieces of row t / 4 of the tile (columns 16 (t % 4) ..), and stores two 16-byte pieces of
// output row t / 4; r and n are multiples of 8, so no piece straddles an edge.
__device__ __forceinline__ void transpose_block(const uint16_t *in, uint16_t *out, int32_t r, int64_t n_all, int64_t blk) {
    __shared__ uint16_t tt[64][64 + 8];
    const int64_t ncb = (n_all + 63) / 64;
    const int64_t j0 = (blk / ncb) * 64, n0 = (blk % ncb) * 64;
    const int t = threadIdx.x, row = t >> 2, c0 = (t & 3) * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t j = j0 + row, n = n0 + c0 + 8 * h;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (j < r && n < n_all) v = *reinterpret_cast<const u32x4 *>(in + j * n_all + n);
        *reinterpret_cast<u32x4 *>(&tt[row][c0 + 8 * h]) = v;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t n = n0 + row, j = j0 + c0 + 8 * h;
        if (n < n_all && j < r) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = (uint32_t)tt[c0 + 8 * h + 2 * k][row] | ((uint32_t)tt[c0 + 8 * h + 2 * k + 1][row] << 16);
            *reinterpret_cast<u32x4 *>(out + n * r + j) = u32x4{w[0], w[1], w[2], w[3]};
        }
    }
}
inline uint32_t transpose_blocks(int32_t r, int64_t n) { return (uint32_t)(((r + 63) / 64) * ((n + 63) / 64)); }

}  // namespace nf4k
