// Logits of the output head with the softmax's statistics in the epilogue (gfx950):
//   l[t, v] = log2(e) sum_k X[row t, k] W[v, k];   per token and tile of 256 vocabulary rows:
//   c (an integer), sum over v != label of 2^(l - c), and (for the gradient) p = bf16(2^(l - c)).
// The logits themselves are never written.
//
// The MFMAs take W's rows as the first operand and the tokens as the second, so a lane holds 64
// vocabulary rows of each of its four tokens: the maximum and the sum are taken in registers, with one
// exchange between the wave's halves and one through LDS between the two waves along the vocabulary.
//
// p's layout is the dX product's LDS image: for each 256 tokens and 64 vocabulary rows a block of 32 KB,
// 128 bytes a token, its 16-byte chunks XOR-swizzled by (token / 2) % 8, so that product loads a
// step as one contiguous run.  The label's own p is left out (0): its coefficient in dX is
// -(1 - p_label), which a rounded p_label near 1 would lose; the sum leaves it out for the same reason.
//
// p is rounded to bf16 because it is an operand of the next product; the sum takes the unrounded values.

#include <type_traits>

#include "common.h"
#include "dqtile.h"
#include "loss.h"
#include "loss_tile.h"

namespace nf4k {

namespace {

// A row's reference is kept while no logit exceeds it by more than this (log2 units): p stays far from bf16's and
// float32's limits (2^127).  The first is 0, which lies within this of the largest logit of nearly every tile there
// is (33 in natural units), and where it does not, the tile takes its own maximum and is rescaled afterwards.
constexpr float kSlack = 48.0f;

template <bool GRAD>
__global__ __launch_bounds__(256, 1) void loss_logits_kernel(LogitsArgs g) {
    // one LDS object per stage: a fragment read of one stage provably never aliases the
    // direct-to-LDS loads in flight into the other
    __shared__ __align__(16) uint8_t As0[LBLOCK * 2];
    __shared__ __align__(16) uint8_t As1[LBLOCK * 2];
    __shared__ __align__(16) uint8_t Bs0[LBLOCK * 2];
    __shared__ __align__(16) uint8_t Bs1[LBLOCK * 2];
    __shared__ float red[2][2][LT];

    const int count = __builtin_amdgcn_readfirstlane(g.r.count[0]);
    const int ntm = (count + LT - 1) / LT;
    if ((int64_t)blockIdx.x >= (int64_t)ntm * g.ntile) return;
    int tm, tn;
    tile_coords_grouped<4>(ntm, g.ntile, (int)blockIdx.x, tm, tn);
    tn += g.tile0;
    const int m0 = tm * LT;
    const int64_t n0 = (int64_t)tn * LT;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;      // along the vocabulary, along the tokens
    const int r32 = lane & 31, hh = lane >> 5;

    // rows of W past V read zeros; the whole of X is one descriptor, its rows gathered
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + n0 * g.K, (g.V - n0) * g.K * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.X, 0x7FFFFFF0LL);

    // instruction q of wave w writes stage rows 8u .. 8u+7 (u = 8w + q); lane l takes row 8u + l/8 and
    // physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8)
    uint32_t voff[2], xoff[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int row = 8 * (8 * wave + q) + (lane >> 3);
        const uint32_t col = (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
        if (q < 2) voff[q] = (uint32_t)(64 * wave + (lane >> 3)) * (uint32_t)(g.K * 2) + col;
        xoff[q] = m0 + row < count ? (uint32_t)g.r.row[m0 + row] * (uint32_t)(g.K * 2) + col : 0x80000000u;
    }
    const uint32_t row8_off = (uint32_t)(8 * g.K * 2);
    const int steps = (int)(g.K / LSTEP);
    auto load = [&](int step, uint8_t *A, uint8_t *B, int q0, int q1) {
        lds_u8 *da = (lds_u8 *)A + wave * 8192, *db = (lds_u8 *)B + wave * 8192;
        const uint32_t at = (uint32_t)step * (LSTEP * 2);
        const uint32_t dead = step < steps ? 0u : 0x80000000u;      // past every descriptor's end
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < q0 || q >= q1) continue;
            const uint32_t v = voff[q & 1] + (uint32_t)q * row8_off + at, x = xoff[q] + at;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(da + q * 1024), 16, v | dead, 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(db + q * 1024), 16, x | dead, 0, 0, 0);
        }
    };
    uint32_t lds_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) lds_off[s] = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
    auto read = [&](const uint8_t *A, const uint8_t *B, int s, LossFrags &f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f.a[i] = *reinterpret_cast<const bf16x8 *>(A + lds_off[s] + (wm * 128 + 32 * i) * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const bf16x8 *>(B + lds_off[s] + (wn * 128 + 32 * j) * 128);
    };
    f32x16 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    loss_loop<8>(steps, As0, Bs0, As1, Bs1, acc, load, read);

    // ---- epilogue.  Lane (r32, hh) of tile (i, j) holds token wn*128 + 32 j + r32 and vocabulary rows
    // wm*128 + 32 i + 8 (v/4) + 4 hh + v%4 ----
    const int lane_e = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    const int c32 = lane_e & 31, he = lane_e >> 5;
    const float NEG = -__builtin_inff();
    // rows of this wave's half that are in the vocabulary (the others hold zeros)
    const int left = (int)min(g.V - n0 - wm * 128, (int64_t)128);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float z = NEG;
        int end = left - 4 * he;
        asm("" : "+v"(end));      // its own for each j: 64 compare masks kept for all four would spill
        if (left == 128) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v) z = fmaxf(z, acc[i][j][v]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    z = fmaxf(z, 32 * i + 8 * (v >> 2) + (v & 3) < end ? acc[i][j][v] : NEG);
        }
        z = fmaxf(z, __shfl_xor(z, 32));
        if (he == 0) red[0][wm][wn * 128 + 32 * j + c32] = z;
    }
    __syncthreads();
    // a token's reference: the one it has, or 0, unless this tile lies too far from it
    auto reference = [&](int tl) {
        const float top = fmaxf(red[0][0][tl], red[0][1][tl]) * kLog2e;
        const float ref = g.ref ? (m0 + tl < count ? g.ref[m0 + tl] : 0.0f) : 0.0f;
        return top <= ref + kSlack && (g.ref || top >= -kSlack) ? ref : ceilf(top);
    };
    const __amdgpu_buffer_rsrc_t rP = make_rsrc(
        GRAD ? g.P + ((int64_t)tm * g.psteps + (int64_t)(tn - g.table0) * 4 + wm * 2) * LBLOCK : nullptr, GRAD ? LBLOCK * 4 : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __builtin_amdgcn_sched_barrier(0);
        const int row = wn * 128 + 32 * j + c32, t = m0 + row;
        const float c = reference(row);
        const int64_t lab64 = t < count ? (int64_t)g.r.label[t] - n0 - wm * 128 : -1;
        const int lab = lab64 >= 0 && lab64 < 128 ? (int)lab64 - 4 * he : -8;
        const uint32_t off = (uint32_t)(row * 128 + ((he ^ ((row >> 1) & 7)) * 16));
        float s = 0.0f, zl = 0.0f;
        int end = left - 4 * he;
        asm("" : "+v"(end));
        // MASK: a label or the vocabulary's end lies in this wave's rows (few have one)
        auto part = [&](auto mask) {
            constexpr bool MASK = decltype(mask)::value;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v4 = 0; v4 < 4; v4 += 2) {
                    uint32_t p[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        float e[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int v = 4 * v4 + 2 * h + u, at = 32 * i + 8 * (v >> 2) + (v & 3);
                            const float l = acc[i][j][v];
                            e[u] = __builtin_amdgcn_exp2f(__builtin_fmaf(l, kLog2e, -c));
                            if (MASK) {
                                zl = at == lab ? l : zl;
                                asm volatile("" : "+v"(zl));      // taken here: 64 masks kept for later would spill
                                e[u] = at == lab || at >= end ? 0.0f : e[u];
                            }
                            s += e[u];
                        }
                        p[h] = pack_bf16x2(e[0], e[1]);
                    }
                    if (GRAD) {
                        // a chunk of 8 vocabulary rows lies half in each half of the wave: after the exchange lanes
                        // 0-31 hold chunk v4, lanes 32-63 chunk v4 + 1
                        const auto x = __builtin_amdgcn_permlane32_swap(p[0], p[2], false, false);
                        const auto y = __builtin_amdgcn_permlane32_swap(p[1], p[3], false, false);
                        __builtin_amdgcn_raw_buffer_store_b128(u32x4{x[0], y[0], x[1], y[1]}, rP, off ^ ((4 * (i & 1) + v4) * 16),
                                                               (i >> 1) * (int)(LBLOCK * 2), 0);
                    }
                }
        };
        if (left < 128 || __builtin_amdgcn_ballot_w64(lab > -8)) {
            part(std::true_type{});
            const int in = lab & ~4;      // whose half holds it: lab = 8 k + 0..3 there
            if (lab >= 0 && in == lab) g.r.zl[t] = zl * kLog2e;
        } else {
            part(std::false_type{});
        }
        s += __shfl_xor(s, 32);
        if (he == 0) red[1][wm][row] = s;
    }
    __syncthreads();
    if (m0 + tid < count) {
        const int64_t o = (int64_t)(tn - g.table0) * g.Mp + m0 + tid;
        g.tref[o] = reference(tid);
        g.tsum[o] = red[1][0][tid] + red[1][1][tid];
    }
}

}  // namespace

hipError_t launch_loss_logits(const LogitsArgs &a, hipStream_t stream) {
    const int64_t grid = (int64_t)(a.Mp / LT) * a.ntile;
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    if (a.P) hipLaunchKernelGGL(loss_logits_kernel<true>, dim3((uint32_t)grid), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(loss_logits_kernel<false>, dim3((uint32_t)grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nf4k
