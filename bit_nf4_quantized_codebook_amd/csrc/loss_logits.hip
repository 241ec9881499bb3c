// Logits of the output head with the softmax's statistics in the epilogue (gfx950):
//   l[t, v] = log2(e) sum_k X[row t, k] W[v, k];   per token and tile of 256 vocabulary rows:
//   c (an integer), sum over v != label of 2^(l - c), and (for the gradient) p = bf16(2^(l - c)).
// The logits themselves are never written.
//
// The MFMAs take W's rows as the first operand and the tokens as the second, so a lane holds four consecutive vocabulary
// rows of a token at a time.  After the last step each wave turns its values through its own part of LDS, 32 tokens at a
// time, into a token's vocabulary rows side by side: a lane then has eight of them, a whole chunk of p.
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

// A row's reference is kept while no logit exceeds it by more than about this (log2 units): p stays far from bf16's
// and float32's limits (2^127).  The first is 0, which lies within this of the largest logit of nearly every tile there
// is (33 in natural units); the sums tell where it does not, and such a tile is done once more against its own maxima
// and rescaled afterwards.  (The maximum first and then the sums, as two passes over the accumulators for every tile,
// was slower.)
constexpr int kSlack = 48;

struct LossStages {
    uint8_t *As0, *Bs0, *As1, *Bs1;
    float *refs;              // [LT]
    int *labs;                // [LT] labels, counted from the tile's first vocabulary row; -1: not in the tile
    float (*sums)[LT];        // [2] by the waves along the vocabulary
    float (*tops)[LT];
};

// the sum or maximum over groups of N lanes (8 or 16), in all of them
template <int N, class Op>
__device__ __forceinline__ float over_lanes(float x, Op op) {
    auto dpp = [](float v, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    x = op(x, dpp(x, std::integral_constant<int, 0xB1>{}));       // lane ^ 1
    x = op(x, dpp(x, std::integral_constant<int, 0x4E>{}));       // lane ^ 2
    x = op(x, dpp(x, std::integral_constant<int, 0x141>{}));      // mirrored within 8
    if (N == 16) x = op(x, dpp(x, std::integral_constant<int, 0x140>{}));      // mirrored within 16
    return x;
}

// One tile: 64 IA vocabulary rows from n0, tokens from m0; entry: its row of the tables; P's blocks from step p0
template <bool GRAD, int IA>
__device__ __forceinline__ void logits_tile(const LogitsArgs &g, const LossStages &st, int count, int tm, int64_t n0, int entry, int p0) {
    const int m0 = tm * LT;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;      // along the vocabulary, along the tokens
    const int r32 = lane & 31, hh = lane >> 5;
    constexpr int WV = 32 * IA;                   // vocabulary rows of a wave
    constexpr int QA = 2 * IA;                    // a wave's loads of W a step

    {
        const int t = m0 + tid;
        const int64_t lab = t < count ? (int64_t)g.r.label[t] - n0 : -1;
        st.labs[tid] = lab >= 0 && lab < 64 * IA ? (int)lab : -1;
        st.refs[tid] = g.ref && t < count ? g.ref[t] : 0.0f;
    }
    // rows of W past V read zeros; the whole of X is one descriptor, its rows gathered
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + n0 * g.K, (g.V - n0) * g.K * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.X, 0x7FFFFFF0LL);

    // instruction q of wave w writes stage rows 8u .. 8u+7 (u = 8w + q; W: QA w + q); lane l takes row 8u + l/8 and
    // physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8)
    uint32_t voff[2], xoff[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int row = 8 * (8 * wave + q) + (lane >> 3);
        const uint32_t col = (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 16);
        if (q < 2) voff[q] = (uint32_t)(8 * QA * wave + (lane >> 3)) * (uint32_t)(g.K * 2) + col;
        xoff[q] = m0 + row < count ? (uint32_t)g.r.row[m0 + row] * (uint32_t)(g.K * 2) + col : 0x80000000u;
    }
    const uint32_t row8_off = (uint32_t)(8 * g.K * 2);
    const int steps = (int)(g.K / LSTEP);
    auto load = [&](int step, uint8_t *A, uint8_t *B, int part) {
        lds_u8 *da = (lds_u8 *)A + wave * (QA * 1024), *db = (lds_u8 *)B + wave * 8192;
        const uint32_t at = (uint32_t)step * (LSTEP * 2);
        const uint32_t dead = step < steps ? 0u : 0x80000000u;      // past every descriptor's end
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if ((q >> 2) != part) continue;
            if (IA == 4 || (q & 1) == 0) {
                const int qa = IA == 4 ? q : q >> 1;
                const uint32_t v = voff[qa & 1] + (uint32_t)qa * row8_off + at;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(da + qa * 1024), 16, v | dead, 0, 0, 0);
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(db + q * 1024), 16, (xoff[q] + at) | dead, 0, 0, 0);
        }
    };
    uint32_t lds_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) lds_off[s] = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
    auto read = [&](const uint8_t *A, const uint8_t *B, int s, LossFrags<IA> &f) {
#pragma unroll
        for (int i = 0; i < IA; ++i) f.a[i] = *reinterpret_cast<const bf16x8 *>(A + lds_off[s] + (wm * WV + 32 * i) * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const bf16x8 *>(B + lds_off[s] + (wn * 128 + 32 * j) * 128);
    };
    f32x16 acc[IA][4];
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    loss_loop<IA, 4 + IA, 4 + IA>(steps, st.As0, st.Bs0, st.As1, st.Bs1, acc, load, read);

    // ---- epilogue.  Lane (r32, hh) of tile (i, j) holds token wn*128 + 32 j + r32 and vocabulary rows
    // wm*WV + 32 i + 8 (v/4) + 4 hh + v%4.  turn(j) lays token group j out as rows of WV floats, whose 16-byte pieces are
    // permuted by the token so that neither the writes nor the reads of two neighbouring pieces meet in a bank. ----
    const int lane_e = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    uint8_t *lds = wave == 0 ? st.As0 : (wave == 1 ? st.As1 : (wave == 2 ? st.Bs0 : st.Bs1));
    constexpr int PIECES = WV / 4;                // a row's pieces of four vocabulary rows
    auto piece = [](int p, int token) { return ((p ^ (p / (PIECES / 2))) ^ (token & (PIECES - 1))) * 16; };
    auto order = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    auto turn = [&](auto jc) {
        constexpr int j = decltype(jc)::value;
        const int c32 = lane_e & 31, he = lane_e >> 5;
        order();
#pragma unroll
        for (int i = 0; i < IA; ++i)
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
                *reinterpret_cast<f32x4 *>(lds + c32 * (WV * 4) + piece(8 * i + 2 * v4 + he, c32)) =
                    f32x4{acc[i][j][4 * v4], acc[i][j][4 * v4 + 1], acc[i][j][4 * v4 + 2], acc[i][j][4 * v4 + 3]};
        order();
    };
    // a lane's eight vocabulary rows: chunk q of token TI it + tt of the group
    constexpr int NQ = WV / 8, TI = 64 / NQ;
    const int q = lane_e & (NQ - 1), tt = lane_e / NQ;
    auto eight = [&](int token, float (&x)[8]) {
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(lds + token * (WV * 4) + piece(2 * q, token));
        const f32x4 hi = *reinterpret_cast<const f32x4 *>(lds + token * (WV * 4) + piece(2 * q + 1, token));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[k] = lo[k];
            x[4 + k] = hi[k];
        }
    };
    // this lane's vocabulary rows from here on are past V (they hold zeros)
    const int64_t left = g.V - n0 - wm * WV;
    const int end = (int)min(max(left - 8 * q, (int64_t)0), (int64_t)8);
    const bool ragged = left < WV;
    const __amdgpu_buffer_rsrc_t rP = make_rsrc(
        GRAD ? g.P + ((int64_t)tm * g.psteps + p0 + wm * (IA / 2)) * LBLOCK : nullptr, GRAD ? LBLOCK * IA : 0);
    auto group = [&](auto jc) {
        turn(jc);
        // B iterations' reads at a time: a wave is alone on its SIMD, nothing else hides their latency
        constexpr int B = 4;
#pragma unroll 1
        for (int it = 0; it < 32 / TI; it += B) {
            float x[B][8], c[B], s[B];
            int lab[B];
            const int tl0 = wn * 128 + 32 * decltype(jc)::value + TI * it + tt;
            bool any = ragged;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                eight(TI * (it + b) + tt, x[b]);
                c[b] = st.refs[tl0 + TI * b];
                lab[b] = st.labs[tl0 + TI * b];
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                // the label's place among this lane's eight, or anything else
                lab[b] = lab[b] < 0 ? -1 : lab[b] - wm * WV - 8 * q;
                any |= (uint32_t)lab[b] < 8u;
            }
            // few batches hold a label
            const bool masked = __builtin_amdgcn_ballot_w64(any) != 0;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float zl = 0.0f;
                s[b] = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float z = x[b][k];
                    x[b][k] = __builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -c[b]));
                    if (masked) {
                        zl = lab[b] == k ? z : zl;
                        x[b][k] = lab[b] == k || k >= end ? 0.0f : x[b][k];
                    }
                    s[b] += x[b][k];
                }
                if (masked && (uint32_t)lab[b] < 8u) g.r.zl[m0 + tl0 + TI * b] = zl * kLog2e;
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                s[b] = over_lanes<NQ>(s[b], [](float a, float b) { return a + b; });
                const int row = tl0 + TI * b;
                if (q == 0) st.sums[wm][row] = s[b];
                if (GRAD) {
                    const float *e = x[b];
                    __builtin_amdgcn_raw_buffer_store_b128(
                        u32x4{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7])}, rP,
                        (uint32_t)((q >> 3) * (int)(LBLOCK * 2) + row * 128 + (((q & 7) ^ ((row >> 1) & 7)) * 16)), 0, 0);
                }
            }
        }
    };
    auto groups = [&]() {
        group(std::integral_constant<int, 0>{});
        group(std::integral_constant<int, 1>{});
        group(std::integral_constant<int, 2>{});
        group(std::integral_constant<int, 3>{});
        __syncthreads();
    };
    groups();
    float sum = st.sums[0][tid] + st.sums[1][tid];
    // Is every token's sum where it should be?  Above 2^kSlack a logit lies too far above the reference; below
    // 2^-kSlack all lie too far below it, or there are none but the label (a reference of an earlier piece may lie
    // above all of this tile); NaN fails too.
    const bool ok = m0 + tid >= count || (sum <= __builtin_ldexpf(1.0f, kSlack) && (g.ref || sum >= __builtin_ldexpf(1.0f, -kSlack)));
    if (!__syncthreads_and(ok)) {
        // the tile once more, those tokens against their own largest logit
        auto top = [&](auto jc) {
            turn(jc);
            for (int it = 0; it < 32 / TI; ++it) {
                const int token = TI * it + tt;
                float x[8], z = -__builtin_inff();
                eight(token, x);
#pragma unroll
                for (int k = 0; k < 8; ++k) z = fmaxf(z, k < end ? x[k] : -__builtin_inff());
                z = over_lanes<NQ>(z, [](float a, float b) { return fmaxf(a, b); });
                if (q == 0) st.tops[wm][wn * 128 + 32 * decltype(jc)::value + token] = z;
            }
        };
        top(std::integral_constant<int, 0>{});
        top(std::integral_constant<int, 1>{});
        top(std::integral_constant<int, 2>{});
        top(std::integral_constant<int, 3>{});
        __syncthreads();
        // (no logit at all, past the vocabulary's end, or NaN only: the reference stays)
        const float most = fmaxf(st.tops[0][tid], st.tops[1][tid]);
        if (!ok && most > -__builtin_inff()) st.refs[tid] = ceilf(most * kLog2e);
        __syncthreads();
        groups();
        sum = st.sums[0][tid] + st.sums[1][tid];
    }
    if (m0 + tid < count) {
        const int64_t o = (int64_t)entry * g.Mp + m0 + tid;
        g.tref[o] = st.refs[tid];
        g.tsum[o] = sum;
    }
}

template <bool GRAD>
__global__ __launch_bounds__(256, 1) void loss_logits_kernel(LogitsArgs g) {
    // one LDS object per stage: a fragment read of one stage provably never aliases the
    // direct-to-LDS loads in flight into the other
    __shared__ __align__(16) uint8_t As0[LBLOCK * 2];
    __shared__ __align__(16) uint8_t As1[LBLOCK * 2];
    __shared__ __align__(16) uint8_t Bs0[LBLOCK * 2];
    __shared__ __align__(16) uint8_t Bs1[LBLOCK * 2];
    __shared__ float refs[LT], sums[2][LT], tops[2][LT];
    __shared__ int labs[LT];
    const LossStages st{As0, Bs0, As1, Bs1, refs, labs, sums, tops};

    const int count = __builtin_amdgcn_readfirstlane(g.r.count[0]);
    const LossTiles tiles((count + LT - 1) / LT, g.ntile);
    const int all = tiles.ntm * tiles.ntn, bid = (int)blockIdx.x;
    int tm, tn;
    if (bid < tiles.whole) {
        // each XCD (bid % 8) takes a contiguous run of tiles
        const int q = tiles.whole / 8;
        tiles.place(bid < 8 * q ? (bid % 8) * q + bid / 8 : bid, tm, tn);
        logits_tile<GRAD, 4>(g, st, count, tm, (int64_t)(g.tile0 + tn) * LT, tn, 4 * tn);
    } else if (bid < 2 * all - tiles.whole) {
        const int h = (bid - tiles.whole) / (all - tiles.whole);
        tiles.place(bid - h * (all - tiles.whole), tm, tn);
        logits_tile<GRAD, 2>(g, st, count, tm, (int64_t)(g.tile0 + tn) * LT + 128 * h, tn + h * g.ntile, 4 * tn + 2 * h);
    }
}

}  // namespace

hipError_t launch_loss_logits(const LogitsArgs &a, hipStream_t stream) {
    // the live rows may have any number of tiles up to Mp's; 128 more workgroups for tiles that are cut
    const int64_t grid = (int64_t)(a.Mp / LT) * a.ntile + 128;
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidValue;
    if (a.P) hipLaunchKernelGGL(loss_logits_kernel<true>, dim3((uint32_t)grid), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(loss_logits_kernel<false>, dim3((uint32_t)grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nf4k
