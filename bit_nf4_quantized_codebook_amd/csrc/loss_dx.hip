// dX's product of the loss over the vocabulary (gfx950):  D[t, n] = sum_v P[t, v] W[v, n]  over a piece
// of the vocabulary, P as loss_logits.hip wrote it.
//
// The reduction runs over W's rows, so W's tile is staged as it lies in memory (64 rows of 256 columns) and
// its fragments come from transposing LDS reads (ds_read_b64_tr_b16: each 16-lane group turns 4 rows x 16
// columns).  A row of the stage is 512 bytes; its 64-byte granules are XOR-swizzled by row % 4, so the
// four rows that half a wave reads at once lie in different banks.  P's blocks are copied as they are.
//
// The MFMAs take W's columns as the first operand and the tokens as the second: a lane holds four
// consecutive columns of a token.
//
// Few tiles (the live rows are counted on the device): a tile's reduction is split over several
// workgroups; all write float32 partials, which loss_fold_kernel sums in a fixed order.

#include "common.h"
#include "dqtile.h"
#include "loss.h"
#include "loss_tile.h"

namespace nf4k {

namespace {

__global__ __launch_bounds__(256, 1) void loss_dx_kernel(LossDxArgs g) {
    __shared__ __align__(16) uint8_t As0[LBLOCK * 2];
    __shared__ __align__(16) uint8_t As1[LBLOCK * 2];
    __shared__ __align__(16) uint8_t Bs0[LBLOCK * 2];
    __shared__ __align__(16) uint8_t Bs1[LBLOCK * 2];

    const int count = __builtin_amdgcn_readfirstlane(g.count[0]);
    const int ntm = (count + LT - 1) / LT, ntn = (int)((g.K + LT - 1) / LT);
    const int tiles = ntm * ntn;
    const LossSplit sp = loss_split(tiles, g.steps);
    if ((int)blockIdx.x >= tiles * sp.ks) return;
    const int split = (int)blockIdx.x / tiles;
    int tm, tn;
    tile_coords_grouped<4>(ntm, ntn, (int)blockIdx.x - split * tiles, tm, tn);
    const int64_t n0 = (int64_t)tn * LT;
    const int kb = split * sp.per, steps = min(g.steps - kb, sp.per);

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;      // along dX's columns, along the tokens
    const int r32 = lane & 31, hh = lane >> 5;

    // W from this workgroup's first row; rows past V read zeros
    const int64_t v0 = g.v0 + (int64_t)kb * LSTEP;
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + v0 * g.K, (g.V - v0) * g.K * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.P + ((int64_t)tm * g.steps + kb) * LBLOCK, (int64_t)steps * LBLOCK * 2);

    // W: instruction q of wave w writes stage rows 2u, 2u + 1 (u = 8w + q); lane l takes row 2u + l/32 and
    // physical 16-byte chunk l%32, whose granule (l%32)/4 holds logical granule ((l%32)/4) ^ (row%4)
    uint32_t aoff[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = 2 * (8 * wave + q) + (lane >> 5);
        const int col = ((((lane & 31) >> 2) ^ (row & 3)) * 4 + (lane & 3)) * 8;
        aoff[q] = n0 + col < g.K ? (uint32_t)((row * g.K + n0 + col) * 2) : 0x80000000u;
    }
    const uint32_t row4_off = (uint32_t)(4 * g.K * 2);
    const uint32_t step_off = (uint32_t)(LSTEP * g.K * 2);
    const uint32_t boff = (uint32_t)(wave * 8192 + lane * 16);
    auto load = [&](int step, uint8_t *A, uint8_t *B, int q0, int q1) {
        lds_u8 *da = (lds_u8 *)A + wave * 8192, *db = (lds_u8 *)B + wave * 8192;
        const bool live = step < steps;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < q0 || q >= q1) continue;
            // rows 2q and 2q + 1 of the wave's 16: q and q + 2 share row % 4
            const uint32_t v = aoff[q & 1] + (uint32_t)(q >> 1) * row4_off + (uint32_t)step * step_off;
            const uint32_t x = boff + (uint32_t)q * 1024u + (uint32_t)step * (uint32_t)(LBLOCK * 2);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(da + q * 1024), 16, live && aoff[q & 1] != 0x80000000u ? v : 0x80000000u, 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(db + q * 1024), 16, live ? x : 0x80000000u, 0, 0, 0);
        }
    };
    // W's fragment of sub-step s, columns wm*128 + 32 i ..: 16-lane group (hh, half) reads rows
    // 16 s + 8 hh + i16/4 (+ 4), columns 16 half + 4 (i16 % 4) .. +3; lane i16 ends with column 16 half + i16
    const int i16 = lane & 15, half = (lane >> 4) & 1, rq = i16 >> 2;
    uint32_t aread[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        aread[i] = (uint32_t)((8 * hh + rq) * 512 + ((wm * 4 + (i ^ rq)) * 64) + half * 32 + (i16 & 3) * 8);
    uint32_t bread[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) bread[s] = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
    auto read = [&](const uint8_t *A, const uint8_t *B, int s, LossFrags &f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *p = A + aread[i] + s * 16 * 512;
            const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)p);
            const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(p + 4 * 512));
            f.a[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const bf16x8 *>(B + bread[s] + (wn * 128 + 32 * j) * 128);
    };
    f32x16 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    loss_loop<12>(steps, As0, Bs0, As1, Bs1, acc, load, read);

    // lane (r32, hh) of tile (i, j) holds token wn*128 + 32 j + r32 and columns wm*128 + 32 i + 8 (v/4) + 4 hh + v%4
    float *out = g.part + ((int64_t)split * tiles + (int64_t)tm * ntn + tn) * (LT * LT);
    const int lane_e = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float *p = out + (wn * 128 + 32 * j + (lane_e & 31)) * LT + wm * 128 + 4 * (lane_e >> 5);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
                *reinterpret_cast<f32x4 *>(p + 32 * i + 8 * v4) =
                    f32x4{acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2], acc[i][j][4 * v4 + 3]};
    }
}

}  // namespace

hipError_t launch_loss_dx(const LossDxArgs &a, hipStream_t stream) {
    const int64_t tiles = (int64_t)(a.Mp / LT) * ((a.K + LT - 1) / LT);
    const int64_t grid = tiles > 256 ? tiles : 256;
    hipLaunchKernelGGL(loss_dx_kernel, dim3((uint32_t)grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nf4k
