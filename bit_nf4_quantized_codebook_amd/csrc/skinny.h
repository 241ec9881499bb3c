// The streaming product of an activation with a rank-r partner, as one workgroup's share of it: used by
// its own launch and, for few tokens, alongside the activation's quantization to 8-bit integers.
#pragma once

#include "common.h"
#include "dqtile.h"

namespace nf4k {

constexpr int ST = 64;          // block tile (both output dims) and reduction step
constexpr int NSTAGE = 4;       // reduction steps in flight per block tile (skinny_nt)
// skinny_tn: two steps per tile and half the LDS, so four workgroups share a CU and fill each
// other's load waits (dL2 + dL1: 16.6 against 18.9 us at 4096 tokens; skinny_nt gained nothing)
constexpr int NSTAGE_TN = 2;
constexpr int ROWB = (ST + 8) * 2;   // padded LDS row, bytes (144: conflict-free 16-byte reads)


// 16-byte fragment of row `row` (the M/N index), reduction elements 16 s + 8 hh .. +7 of a tile
// stored [row][reduction]
__device__ __forceinline__ bf16x8 frag_rows(const uint8_t *t, int row, int s, int hh) {
    return *reinterpret_cast<const bf16x8 *>(t + row * ROWB + (s * 16 + hh * 8) * 2);
}
// same fragment from a tile stored [reduction][col]: two transposing reads
__device__ __forceinline__ bf16x8 frag_tr(const uint8_t *t, int col0, int s, int lane) {
    const int i16 = lane & 15, hh = lane >> 5, half = (lane >> 4) & 1;
    const int rowb = s * 16 + hh * 8 + (i16 >> 2);
    const uint8_t *base = t + (col0 + half * 16 + 4 * (i16 & 3)) * 2;
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(base + rowb * ROWB));
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(base + (rowb + 4) * ROWB));
    const v8i16 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
}

// Each thread moves 2 x 16 bytes of each 64 x 64 operand tile per step: tile row = tid/8 (+32),
// 16-byte chunk = tid%8.
struct TileLoad {
    u32x4 v[2];
};

// P[ks][m][j] = sum_{k in chunk ks} A[m][k] * B(k, j)
//   B_ROWS_K = true : B given as Bk [Kred, R] (row k), tile stored [k][j] -> transposing reads
//   B_ROWS_K = false: B given as Bt [R, Kred] (row j), tile stored [j][k] -> row reads
// Workgroup (256 threads) (bx, by, bz): rows 64 bx .., columns 64 by .., reduction chunk bz.
template <bool B_ROWS_K>
__device__ __forceinline__ void skinny_nt_block(const uint16_t *__restrict__ A, const uint16_t *__restrict__ B,
                                                float *__restrict__ P, int64_t M, int32_t R, int64_t Kred,
                                                int64_t kchunk, uint32_t bx, uint32_t by, uint32_t bz) {
    __shared__ __align__(16) uint8_t As[NSTAGE][ST * ROWB];
    __shared__ __align__(16) uint8_t Bs[NSTAGE][ST * ROWB];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hh = lane >> 5;
    const int64_t m0 = (int64_t)bx * ST;
    const int j0 = by * ST;
    const int64_t kbeg = (int64_t)bz * kchunk;
    const int64_t kend = (kbeg + kchunk < Kred) ? kbeg + kchunk : Kred;
    const int nsteps = kend > kbeg ? (int)((kend - kbeg + ST - 1) / ST) : 0;

    const __amdgpu_buffer_rsrc_t rA = make_rsrc(A + m0 * Kred, (M - m0) * Kred * 2);
    const __amdgpu_buffer_rsrc_t rB = B_ROWS_K ? make_rsrc(B, Kred * (int64_t)R * 2)
                                               : make_rsrc(B + (int64_t)j0 * Kred, ((int64_t)R - j0) * Kred * 2);
    const int trow = tid >> 3, tch = tid & 7;

    auto load = [&](int step, TileLoad &a, TileLoad &b) {
        const int64_t k0 = kbeg + (int64_t)step * ST;
        const bool live = step < nsteps;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = trow + 32 * h;
            // A: row m0+row, columns k0 + 8 tch; columns past the chunk end read zeros
            const int64_t ka = k0 + tch * 8;
            a.v[h] = bload16(rA, (live && ka < kend) ? (uint32_t)((row * Kred + ka) * 2) : 0xFFFFFFF0u);
            if (B_ROWS_K) {
                // B tile row = k0 + row, columns j0 + 8 tch (j < R)
                const int64_t kb = k0 + row;
                const bool ok = live && kb < kend && j0 + tch * 8 < R;
                b.v[h] = bload16(rB, ok ? (uint32_t)((kb * R + j0 + tch * 8) * 2) : 0xFFFFFFF0u);
            } else {
                // B tile row = j0 + row, columns k0 + 8 tch
                b.v[h] = bload16(rB, (live && ka < kend) ? (uint32_t)((row * Kred + ka) * 2) : 0xFFFFFFF0u);
            }
        }
    };
    auto store = [&](int slot, const TileLoad &a, const TileLoad &b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = trow + 32 * h;
            *reinterpret_cast<u32x4 *>(&As[slot][row * ROWB + tch * 16]) = a.v[h];
            *reinterpret_cast<u32x4 *>(&Bs[slot][row * ROWB + tch * 16]) = b.v[h];
        }
    };

    f32x16 acc = {};
    TileLoad la[NSTAGE], lb[NSTAGE];
    for (int g0 = 0; g0 < nsteps; g0 += NSTAGE) {
#pragma unroll
        for (int u = 0; u < NSTAGE; ++u) load(g0 + u, la[u], lb[u]);
#pragma unroll
        for (int u = 0; u < NSTAGE; ++u) store(u, la[u], lb[u]);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NSTAGE; ++u) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const bf16x8 fa = frag_rows(As[u], wm * 32 + r32, s, hh);
                const bf16x8 fb = B_ROWS_K ? frag_tr(Bs[u], wn * 32, s, lane)
                                           : frag_rows(Bs[u], wn * 32 + r32, s, hh);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
            }
        }
        __syncthreads();
    }
    const int col = j0 + wn * 32 + r32;
    if (col < R) {
        float *Pk = P + (int64_t)bz * M * R;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int64_t row = m0 + wm * 32 + (v >> 2) * 8 + hh * 4 + (v & 3);
            if (row < M) Pk[row * R + col] = acc[v];
        }
    }
}

}  // namespace nf4k
