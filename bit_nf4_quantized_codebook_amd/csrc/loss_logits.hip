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
// p is rounded to bf16 because it is an operand of the next product.  The loss takes the sum of the unrounded values, dX
// that of the rounded ones: the weights that its rows of W enter with then add up to 1, and what all rows have in common
// cancels against the label's row as it does in the formula.  (Divided by the unrounded sum, p's rounding errors met that
// common part: with one four times the rows' own and a largest p of 0.5 a token's dX was off by up to 6.5e-3 of itself,
// now 1.95e-3, of which its own rounding is 1.8e-3.  The second sum costs 1 us of 117 at 129 x 32000 x 4096 with 39
// labelled and 5 of 1650 at 4096.)
//
// 256 x 256 tiles: both operands of a step are then 64 KB for 2048 cycles of MFMAs, two stages fill the LDS.  Bound by
// the MFMAs at the clock that their power allows: a step of 64 takes 1.57 us (1.37 PFLOP/s over the chip), a tile's
// epilogue 8.  4096 x 32000 x 4096 with p: 860 us of kernel, 1.25 PFLOP/s; 2048 x 32000 x 8192 without: 805 us, 1.33.
// A library product of the same operands, which writes the logits, reaches 1.34.

#include "common.h"
#include "dqtile.h"
#include "loss.h"
#include "loss_tile.h"

namespace nf4k {

namespace {

struct LossStages {
    uint8_t *S0, *S1;
    float *refs;              // [LT]
    int *labs;                // [LT] labels, counted from the tile's first vocabulary row; -1: not in the tile
    float (*sums)[LT];        // [2] by the waves along the vocabulary
    float (*psums)[LT];       // the same of p
    float (*tops)[LT];
};

struct LossPlace {
    int tm;                   // tile of rows
    int64_t n0;               // first vocabulary row
    int entry, p0;            // row of the tables; first step of P's blocks
};

// A workgroup's tiles of 64 IA vocabulary rows, one after the other: place(i), i < n.  The next tile's first step is
// loaded (into S1) before this one's epilogue, which works in S0.
template <bool GRAD, int IA, class Place>
__device__ __forceinline__ void logits_tiles(const LogitsArgs &g, const LossStages &st, int count, int n, Place place) {
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;      // along the vocabulary, along the tokens
    const int r32 = lane & 31, hh = lane >> 5;
    constexpr int WV = 32 * IA;                   // vocabulary rows of a wave
    constexpr int QA = 2 * IA;                    // a wave's loads of W a step

    // Instruction q of wave w writes stage rows 8u .. 8u+7 (u = 8w + q; W: QA w + q); lane l takes row 8u + l/8 and
    // physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8).  Rows of W past V read zeros; the whole of X is
    // one descriptor, its rows gathered.  A row out of range is so by its lane offset alone, so the step goes into the
    // scalar offset and a load costs no VALU; steps past the last load the last one again (never used, and in range).
    const int l8 = lane >> 3;
    auto chunk = [&](int q) { return (uint32_t)(((lane & 7) ^ ((4 * q + (l8 >> 1)) & 7)) * 16); };
    __amdgpu_buffer_rsrc_t rA;
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.X, 0x7FFFFFF0LL);
    uint32_t voff[QA], xoff[8];
    int rows[8];
#pragma unroll
    for (int q = 0; q < QA; ++q) voff[q] = (uint32_t)(8 * (QA * wave + q) + l8) * (uint32_t)(g.K * 2) + chunk(q);
    const int steps = (int)(g.K / LSTEP);
    // what a tile needs of its rows: their tokens, and this thread's label and reference
    int label;
    float ref;
    auto fetch = [&](const LossPlace &p) {
        const int m0 = p.tm * LT;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int row = m0 + 8 * (8 * wave + q) + l8;
            rows[q] = row < count ? g.r.row[row] : -1;
        }
        label = m0 + tid < count ? g.r.label[m0 + tid] : -1;
        ref = g.ref && m0 + tid < count ? g.ref[m0 + tid] : 0.0f;
    };
    auto load = [&](int step, uint8_t *stage, int part) {
        lds_u8 *da = (lds_u8 *)stage + wave * (QA * 1024), *db = (lds_u8 *)(stage + LOPB) + wave * 8192;
        const int at = min(step, steps - 1) * (LSTEP * 2);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if ((q >> 2) != part) continue;
            if (IA == 4 || (q & 1) == 0) {
                const int qa = IA == 4 ? q : q >> 1;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(da + qa * 1024), 16, voff[qa], at, 0, 0);
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(db + q * 1024), 16, xoff[q], at, 0, 0);
        }
    };
    auto first_loads = [&](const LossPlace &p) {
        rA = make_rsrc(g.W + p.n0 * g.K, (g.V - p.n0) * g.K * 2);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            xoff[q] = rows[q] >= 0 ? (uint32_t)rows[q] * (uint32_t)(g.K * 2) + chunk(q) : 0x80000000u;
        load(0, st.S1, 0);
        load(0, st.S1, 1);
    };
    uint32_t lds_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) lds_off[s] = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
    auto read = [&](const uint8_t *A, int s, LossFrags<IA> &f) {
        const uint8_t *B = A + LOPB;
#pragma unroll
        for (int i = 0; i < IA; ++i) f.a[i] = *reinterpret_cast<const bf16x8 *>(A + lds_off[s] + (wm * WV + 32 * i) * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const bf16x8 *>(B + lds_off[s] + (wn * 128 + 32 * j) * 128);
    };
    if (n <= 0) return;
    LossPlace cur = place(0);
    fetch(cur);
    first_loads(cur);
#pragma unroll 1
    for (int index = 0;; ++index) {
        const int m0 = cur.tm * LT;
        const int64_t n0 = cur.n0;
        {
            const int64_t lab = (int64_t)label - n0;
            st.labs[tid] = label >= 0 && lab >= 0 && lab < 64 * IA ? (int)lab : -1;
            st.refs[tid] = ref;
        }
        const bool more = index + 1 < n;
        const LossPlace next = more ? place(index + 1) : cur;
        fetch(next);
        f32x16 acc[IA][4];
#pragma unroll
        for (int i = 0; i < IA; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        // between the first step's loads and here lie p's stores, whose end nothing waits for
        constexpr int STORES = GRAD ? 32 * WV / 128 : 0;
        loss_loop<IA, 4 + IA, 4 + IA, STORES>(steps, index > 0, st.S1, st.S0, acc, load, read);
        if (more) first_loads(next);

        // ---- epilogue.  Lane (r32, hh) of tile (i, j) holds token wn*128 + 32 j + r32 and vocabulary rows
        // wm*WV + 32 i + 8 (v/4) + 4 hh + v%4.  turn(j) lays token group j out as rows of WV floats, whose 16-byte pieces are
        // permuted by the token so that neither the writes nor the reads of two neighbouring pieces meet in a bank. ----
        const int lane_e = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        uint8_t *lds = st.S0 + wave * 16384;          // 32 tokens of WV floats
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
            GRAD ? g.P + ((int64_t)cur.tm * g.psteps + cur.p0 + wm * (IA / 2)) * LBLOCK : nullptr, GRAD ? LBLOCK * IA : 0);
        auto group = [&](auto jc, auto far) {
            turn(jc);
            // B iterations' reads at a time: a wave is alone on its SIMD, nothing else hides their latency
            constexpr int B = 4;
#pragma unroll 1
            for (int it = 0; it < 32 / TI; it += B) {
                float x[B][8], c[B], s[B], sp[B];
                u32x4 p[B];
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
                // few batches hold a label; the empty statement keeps this a branch (as selects for every element it doubled
                // the epilogue's time)
                if (__builtin_amdgcn_ballot_w64(any)) {
                    asm volatile("");
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        float zl = 0.0f;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            zl = lab[b] == k ? x[b][k] : zl;
                            x[b][k] = lab[b] == k || k >= end ? -__builtin_inff() : x[b][k];
                        }
                        if ((uint32_t)lab[b] < 8u) g.r.zl[m0 + tl0 + TI * b] = zl * kLog2e;
                    }
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[b][k] = __builtin_amdgcn_exp2f(loss_above(x[b][k], c[b], decltype(far)::value));
                    const float *e = x[b];
                    s[b] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
                    if (GRAD) {
                        p[b] = u32x4{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7])};
                        sp[b] = add_bf16x2(add_bf16x2(0.0f, p[b][0]), p[b][1]) + add_bf16x2(add_bf16x2(0.0f, p[b][2]), p[b][3]);
                    }
                }
                const auto plus = [](float a, float b) { return a + b; };
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    s[b] = over_lanes<NQ>(s[b], plus);
                    if (GRAD) sp[b] = over_lanes<NQ>(sp[b], plus);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int row = tl0 + TI * b;
                    st.sums[wm][row] = s[b];      // the same from all of a token's lanes
                    if (GRAD) {      // nontemporal: 1647 us for the whole call at 4096 x 32000 x 4096, 1659 without
                        st.psums[wm][row] = sp[b];
                        __builtin_amdgcn_raw_buffer_store_b128(
                            p[b], rP, (uint32_t)((q >> 3) * (int)(LBLOCK * 2) + row * 128 + (((q & 7) ^ ((row >> 1) & 7)) * 16)), 0, 2);
                    }
                }
            }
        };
        auto groups = [&](auto far) {
            group(std::integral_constant<int, 0>{}, far);
            group(std::integral_constant<int, 1>{}, far);
            group(std::integral_constant<int, 2>{}, far);
            group(std::integral_constant<int, 3>{}, far);
            __syncthreads();
        };
        groups(std::false_type{});
        float sum = st.sums[0][tid] + st.sums[1][tid];
        // Is every token's sum where it should be?  Above 2^kLossSlack a logit lies too far above the reference; below
        // 2^-kLossSlack all lie too far below it, or there are none but the label (a reference of an earlier piece may lie
        // above all of this tile, but needs the other pass from kLossFar on); NaN fails too.
        const bool ok = m0 + tid >= count || (sum <= __builtin_ldexpf(1.0f, kLossSlack) &&
                                              (g.ref ? fabsf(st.refs[tid]) < kLossFar : sum >= __builtin_ldexpf(1.0f, -kLossSlack)));
        if (!__syncthreads_and(ok)) {
            // the tile once more, those tokens against their largest logit but the label's (which may lie so far above the others
            // that float32 would hold nothing of them beside it)
            auto top = [&](auto jc) {
                turn(jc);
                for (int it = 0; it < 32 / TI; ++it) {
                    const int token = TI * it + tt;
                    float x[8], z = -__builtin_inff();
                    eight(token, x);
                    const int at = st.labs[wn * 128 + 32 * decltype(jc)::value + token], lab = at < 0 ? -1 : at - wm * WV - 8 * q;
#pragma unroll
                    for (int k = 0; k < 8; ++k) z = fmaxf(z, k < end && k != lab ? x[k] : -__builtin_inff());
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
            groups(std::true_type{});
            sum = st.sums[0][tid] + st.sums[1][tid];
        }
        if (m0 + tid < count) {
            const int64_t o = (int64_t)cur.entry * g.Mp + m0 + tid;
            g.tref[o] = st.refs[tid];
            g.tsum[o] = sum;
            if (GRAD) g.tp[o] = st.psums[0][tid] + st.psums[1][tid];
        }
        if (!more) break;
        __syncthreads();       // sums and refs are read
        cur = next;
    }
}

template <bool GRAD>
__global__ __launch_bounds__(256, 1) void loss_logits_kernel(LogitsArgs g) {
    // one LDS object per stage: a fragment read of one stage provably never aliases the
    // direct-to-LDS loads in flight into the other
    __shared__ __align__(16) uint8_t S0[2 * LOPB];
    __shared__ __align__(16) uint8_t S1[2 * LOPB];
    __shared__ float refs[LT], sums[2][LT], psums[GRAD ? 2 : 1][LT], tops[2][LT];
    __shared__ int labs[LT];
    const LossStages st{S0, S1, refs, labs, sums, psums, tops};

    const int count = __builtin_amdgcn_readfirstlane(g.r.count[0]);
    const LossTiles tiles((count + LT - 1) / LT, g.ntile);
    // each XCD (blockIdx % 8) takes a contiguous run of the whole tiles, its 32 workgroups 32 of them at a time
    const int xcd = (int)blockIdx.x & 7, slot = (int)blockIdx.x >> 3;
    const int first = (int)((int64_t)tiles.whole * xcd / 8), last = (int)((int64_t)tiles.whole * (xcd + 1) / 8);
    logits_tiles<GRAD, 4>(g, st, count, (last - first - slot + 31) / 32, [&](int i) {
        LossPlace p;
        int tn;
        tiles.place(first + slot + 32 * i, p.tm, tn);
        p.n0 = (int64_t)(g.tile0 + tn) * LT;
        p.entry = tn;
        p.p0 = 4 * tn;
        return p;
    });
    // halves of the tiles that are cut: at most one a workgroup
    const int cut = tiles.ntm * tiles.ntn - tiles.whole;
    if ((int)blockIdx.x >= 2 * cut) return;
    __syncthreads();
    logits_tiles<GRAD, 2>(g, st, count, 1, [&](int) {
        LossPlace p;
        int tn;
        const int h = (int)blockIdx.x / cut;
        tiles.place(tiles.whole + (int)blockIdx.x - h * cut, p.tm, tn);
        p.n0 = (int64_t)(g.tile0 + tn) * LT + 128 * h;
        p.entry = tn + h * g.ntile;
        p.p0 = 4 * tn + 2 * h;
        return p;
    });
}

}  // namespace

hipError_t launch_loss_logits(const LogitsArgs &a, hipStream_t stream) {
    const uint32_t grid = 256;      // a workgroup on each CU
    if (a.P) hipLaunchKernelGGL(loss_logits_kernel<true>, dim3(grid), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(loss_logits_kernel<false>, dim3(grid), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nf4k
