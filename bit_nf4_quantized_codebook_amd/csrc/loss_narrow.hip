// The loss for few tokens, forward (from 17) and with its gradient (gfx950): both products stream the weight, and tiles of
// 256 x 256 with two stages in flight leave the memory idle.  Tiles here are narrow and their stages many:
//   1. logits: 64 vocabulary rows a workgroup (more than 128 live tokens: 64 or 128).  Each makes the list of live rows for
//      itself, from at most 256 labels;
//   2. the join of the blocks of 64 rows (loss.hip; forward: and the mean);
//   3. dX's product: 128 columns over a part of the vocabulary, float32 partials;
//   4. their sum, dX, and the mean.
// A launch is made for the M tokens there may be (MT = 64, 128 or 256: its LDS and its grid), a tile for those that are
// live (TT): 60 labelled of 200 cost what 60 do.
// The layouts of p (in blocks of MT tokens), of the LDS stages and of the fragments are those of loss_logits.hip and loss_dx.hip.
//
// Bound by HBM: forward 37 x 50001 x 4096 101 us a call (logits 90: 4.5 TB/s), 100 x 32000 x 4096 71 (90 on tiles of 256),
// 200 88 (101); with the gradient, which reads the weight twice, 16, 64, 100 and 200 x 32000 x 4096 108, 120, 131 and 183
// (147, 156, 169 and 189 on tiles of 256), 129 with 39 labelled 117 (155), 100 x 4000 x 1024 29 (57).

#include "common.h"
#include "dqtile.h"
#include "loss.h"
#include "loss_tile.h"

namespace nf4k {

namespace {

// A step's wait: at most LEFT of this wave's loads still on their way, its LDS reads done; then the workgroup's barrier
// alone (__syncthreads would wait for the later stages' loads too).
template <int LEFT>
__device__ __forceinline__ void step_barrier() {
    static_assert(LEFT < 64, "vmcnt's range");
    __builtin_amdgcn_s_waitcnt((LEFT & 15) | (7 << 4) | (0 << 8) | ((LEFT >> 4) << 14));
    asm volatile("s_barrier" ::: "memory");
}

template <int MT>
struct NarrowLds {
    uint8_t *S[6];                                   // LDS objects (a stage is one, or two of them)
    float (*refs)[MT], (*sums)[MT], (*psums)[MT], (*tops)[MT];      // psums: of p
    int *labs, *rows;
};

// 64 VI vocabulary rows by TT tokens.  VI = 2: two blocks of 64, a wave's rows (64 of them) are of one block.
template <int TT, int MT, int NST, int VI, bool GRAD>
struct NarrowLogits {
    static __device__ __forceinline__ void run(const LossNarrow &g, const NarrowLds<MT> &lds_, int count) {
        // NST: stages; NST - 1 of them in flight
        constexpr int VB = 64 * VI * LSTEP * 2;          // bytes of W in a stage, before the tokens'
        constexpr int JN = TT / 64;                      // 32-token tiles of a wave
        constexpr int QW = 2 * VI, QX = TT / 32;         // a wave's loads of W and X a step
        // a stage's W and tokens: with MT = 256 objects 0 .. 2 of 16 KB and 3 .. 5 of 32 take one each, or a whole stage
        // where it fits
        constexpr bool APART = MT == 256 && TT == 256;
        uint8_t *w[NST], *x[NST];
#pragma unroll
        for (int i = 0; i < NST; ++i) {
            w[i] = lds_.S[MT == 256 && TT == 128 ? 3 + i : i];
            x[i] = APART ? lds_.S[3 + i] : w[i] + VB;
        }
        float (*const refs)[MT] = lds_.refs, (*const sums)[MT] = lds_.sums, (*const psums)[MT] = lds_.psums, (*const tops)[MT] = lds_.tops;
        int *const labs = lds_.labs, *const rows = lds_.rows;

        const int tid = threadIdx.x;
        const int lane = tid & 63;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int wm = wave >> 1, wn = wave & 1;         // along the vocabulary, along the tokens
        const int r32 = lane & 31, hh = lane >> 5;
        const int64_t n0 = (int64_t)blockIdx.x * (64 * VI);

        // rows of W past V read zeros; dead tokens too
        const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + n0 * g.K, (g.V - n0) * g.K * 2);
        const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.X, 0x7FFFFFF0LL);
        const __amdgpu_buffer_rsrc_t none = make_rsrc(g.X, 0);
        const int l8 = lane >> 3;
        // instruction q of a wave writes stage rows 8u .. 8u+7 (u = Q wave + q, Q even); lane l takes row 8u + l/8 and
        // physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8)
        auto chunk = [&](int q) { return (uint32_t)(((lane & 7) ^ ((4 * q + (l8 >> 1)) & 7)) * 16); };
        uint32_t voff[QW], xoff[QX];
#pragma unroll
        for (int q = 0; q < QW; ++q) voff[q] = (uint32_t)(8 * (QW * wave + q) + l8) * (uint32_t)(g.K * 2) + chunk(q);
#pragma unroll
        for (int q = 0; q < QX; ++q) {
            const int row = rows[8 * (QX * wave + q) + l8];
            xoff[q] = row >= 0 ? (uint32_t)row * (uint32_t)(g.K * 2) + chunk(q) : 0x80000000u;
        }
        const int steps = (int)(g.K / LSTEP);
        auto load = [&](int step, uint8_t *sw, uint8_t *sx) {
            lds_u8 *da = (lds_u8 *)sw + wave * (QW * 1024), *db = (lds_u8 *)sx + wave * (QX * 1024);
            const int at = step * (LSTEP * 2);
            const bool past = step >= steps;             // zeros, without memory
#pragma unroll
            for (int q = 0; q < QW; ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(past ? none : rA, (lds_void *)(da + q * 1024), 16, voff[q], at, 0, 0);
#pragma unroll
            for (int q = 0; q < QX; ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(past ? none : rB, (lds_void *)(db + q * 1024), 16, xoff[q], at, 0, 0);
        };
        f32x16 acc[VI][JN];
#pragma unroll
        for (int i = 0; i < VI; ++i)
#pragma unroll
            for (int j = 0; j < JN; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        auto multiply = [&](const uint8_t *sw, const uint8_t *sx) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t o = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
                bf16x8 a[VI];
#pragma unroll
                for (int i = 0; i < VI; ++i) a[i] = *reinterpret_cast<const bf16x8 *>(sw + o + 32 * (VI * wm + i) * 128);
#pragma unroll
                for (int j = 0; j < JN; ++j) {
                    const bf16x8 b = *reinterpret_cast<const bf16x8 *>(sx + o + (32 * JN * wn + 32 * j) * 128);
#pragma unroll
                    for (int i = 0; i < VI; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b, acc[i][j], 0, 0, 0);
                }
            }
        };
        // The stage of step s is free for step s + NST after the barrier of step s + 1.  Steps past the last multiply zeros.
        constexpr int LEFT = (NST - 2) * (QW + QX);
#pragma unroll
        for (int i = 0; i < NST - 1; ++i) load(i, w[i], x[i]);
        for (int step = 0; step < steps; step += NST) {
#pragma unroll
            for (int i = 0; i < NST; ++i) {
                step_barrier<LEFT>();
                load(step + i + NST - 1, w[(i + NST - 1) % NST], x[(i + NST - 1) % NST]);
                multiply(w[i], x[i]);
            }
        }
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();

        // ---- epilogue, as in loss_logits.hip: each wave turns 32 vocabulary rows x 32 JN tokens at a time through LDS, rows of
        // 128 bytes; four lanes then hold a token's 32, eight each ----
        uint8_t *lds = (wave < 2 ? x[0] : x[1]) + (wave & 1) * (32 * JN * 128);
        auto piece = [](int p, int token) { return (p ^ ((token >> 1) & 7)) * 16; };
        constexpr int B = 2 * JN;                        // 16 tokens at a time
        const int q = lane & 3, tt = lane >> 2;
        float z[VI][B][8];
#pragma unroll
        for (int i = 0; i < VI; ++i) {
#pragma unroll
            for (int j = 0; j < JN; ++j)
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    const f32x16 &x = acc[i][j];
                    *reinterpret_cast<f32x4 *>(lds + (32 * j + r32) * 128 + piece(2 * v4 + hh, r32)) =
                        f32x4{x[4 * v4], x[4 * v4 + 1], x[4 * v4 + 2], x[4 * v4 + 3]};
                }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int token = 16 * b + tt;
                const f32x4 lo = *reinterpret_cast<const f32x4 *>(lds + token * 128 + piece(2 * q, token));
                const f32x4 hi = *reinterpret_cast<const f32x4 *>(lds + token * 128 + piece(2 * q + 1, token));
#pragma unroll
                for (int k = 0; k < 8; ++k) z[i][b][k] = k < 4 ? lo[k & 3] : hi[k & 3];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        // this wave's block of 64 vocabulary rows (there may be none), and its row of the arrays
        const int block = (int)blockIdx.x * VI + (VI == 2 ? wm : 0), half = VI == 2 ? wm : 0;
        int end[VI];                                     // of this lane's eight rows
#pragma unroll
        for (int i = 0; i < VI; ++i)
            end[i] = (int)min(max(g.V - n0 - 32 * (VI * wm + i) - 8 * q, (int64_t)0), (int64_t)8);
        auto largest = [&]() {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float x = -__builtin_inff();
                const int at = labs[32 * JN * wn + 16 * b + tt];
#pragma unroll
                for (int i = 0; i < VI; ++i) {
                    const int lab = at < 0 ? -1 : at - 32 * (VI * wm + i) - 8 * q;
#pragma unroll
                    for (int k = 0; k < 8; ++k) x = fmaxf(x, k < end[i] && k != lab ? z[i][b][k] : -__builtin_inff());
                }
                x = over_lanes<4>(x, [](float a, float b) { return fmaxf(a, b); });
                tops[wm][32 * JN * wn + 16 * b + tt] = x;
            }
        };
        const __amdgpu_buffer_rsrc_t rP = make_rsrc(GRAD && block < g.n.steps ? g.P + (int64_t)block * (MT * LSTEP) : nullptr,
                                                    GRAD && block < g.n.steps ? MT * LSTEP * 2 : 0);
        auto groups = [&](auto far) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int tl = 32 * JN * wn + 16 * b + tt;
                const float c = refs[half][tl];
                float s = 0.0f, sp = 0.0f;
#pragma unroll
                for (int i = 0; i < VI; ++i) {
                    const int lab = labs[tl] < 0 ? -1 : labs[tl] - 32 * (VI * wm + i) - 8 * q;
                    float e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (lab == k) g.r.zl[tl] = z[i][b][k] * kLog2e;
                        e[k] = lab == k || k >= end[i] ? 0.0f : __builtin_amdgcn_exp2f(loss_above(z[i][b][k], c, decltype(far)::value));
                        s += e[k];
                    }
                    if (GRAD) {
                        const u32x4 p = {pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7])};
#pragma unroll
                        for (int k = 0; k < 4; ++k) sp = add_bf16x2(sp, p[k]);
                        __builtin_amdgcn_raw_buffer_store_b128(
                            p, rP, (uint32_t)(tl * 128 + (((4 * (VI == 2 ? i : wm) + q) ^ ((tl >> 1) & 7)) * 16)), 0, 0);
                    }
                }
                const auto plus = [](float a, float b) { return a + b; };
                sums[wm][tl] = over_lanes<4>(s, plus);   // the same from all of a token's lanes
                if (GRAD) psums[wm][tl] = over_lanes<4>(sp, plus);
            }
            __syncthreads();
        };
        groups(std::false_type{});
        // thread: a token's one or two blocks
        const int t = tid < TT ? tid : 0;
        float sum[VI];
        bool ok[VI], all = true;
        auto collect = [&]() {
#pragma unroll
            for (int h = 0; h < VI; ++h) sum[h] = VI == 2 ? sums[h][t] : sums[0][t] + sums[1][t];
        };
        collect();
#pragma unroll
        for (int h = 0; h < VI; ++h) {
            ok[h] = t >= count || (int)blockIdx.x * VI + h >= g.n.steps ||
                    (sum[h] <= __builtin_ldexpf(1.0f, kLossSlack) && sum[h] >= __builtin_ldexpf(1.0f, -kLossSlack));
            all &= ok[h];
        }
        if (!__syncthreads_and(all)) {
            largest();
            __syncthreads();
#pragma unroll
            for (int h = 0; h < VI; ++h) {
                const float most = VI == 2 ? tops[h][t] : fmaxf(tops[0][t], tops[1][t]);
                if (tid < TT && !ok[h] && most > -__builtin_inff()) refs[h][t] = ceilf(most * kLog2e);
            }
            __syncthreads();
            groups(std::true_type{});
            collect();
        }
        if (tid < count)
#pragma unroll
            for (int h = 0; h < VI; ++h) {
                if ((int)blockIdx.x * VI + h >= g.n.steps) break;
                const int64_t o = (int64_t)tid * g.n.steps + (int)blockIdx.x * VI + h;
                g.tref[o] = refs[h][tid];
                g.tsum[o] = sum[h];
                if (GRAD) g.tp[o] = VI == 2 ? psums[h][tid] : psums[0][tid] + psums[1][tid];
            }
    }
};

// D[t, n] of 128 columns and all tokens over `per` steps of the vocabulary: workgroup (split, tn)
template <int TT, int MT, int NST>
struct NarrowDx {
    static __device__ __forceinline__ void run(const LossNarrow &g, uint8_t *S0, uint8_t *S1, uint8_t *S2, uint8_t *S3, int count) {
        constexpr int WB = LSTEP * 128 * 2;              // bytes of W in a stage, before P's
        constexpr int JN = TT / 32;
        constexpr int QP = TT / 32;                      // a wave's loads of P a step (of W: 4)
        constexpr int PB = MT * LSTEP * 2;               // bytes of one of P's blocks
        const int lane = threadIdx.x & 63;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int r32 = lane & 31, hh = lane >> 5;
        const int ntn = (int)((g.K + 127) / 128);
        const int split = (int)blockIdx.x / ntn, tn = (int)blockIdx.x % ntn;
        const int kb = split * g.n.per, steps = min(g.n.steps - kb, g.n.per);
        const int64_t n0 = (int64_t)tn * 128, v0 = (int64_t)kb * LSTEP;

        const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + v0 * g.K, (g.V - v0) * g.K * 2);
        const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.P + (int64_t)kb * (PB / 2), (int64_t)steps * PB);
        const __amdgpu_buffer_rsrc_t none = make_rsrc(g.W, 0);
        // W: instruction q of wave w writes stage rows 4u .. 4u+3 (u = 4w + q) of 256 bytes; lane l takes row 4u + l/16 and
        // physical 16-byte chunk l%16, whose granule (l%16)/4 holds logical granule ((l%16)/4) ^ (row%4)
        const int row4 = lane >> 4, col = ((((lane & 15) >> 2) ^ row4) * 4 + (lane & 3)) * 8;
        const uint32_t aoff = n0 + col < g.K ? (uint32_t)(((16 * wave + row4) * g.K + n0 + col) * 2) : 0x80000000u;
        const uint32_t row4_off = (uint32_t)(4 * g.K * 2), step_off = (uint32_t)(LSTEP * g.K * 2);
        uint32_t boff[QP];
#pragma unroll
        for (int q = 0; q < QP; ++q)
            boff[q] = 8 * (QP * wave + q) + (lane >> 3) < count ? (uint32_t)((QP * wave + q) * 1024 + lane * 16) : 0x80000000u;
        auto load = [&](int step, uint8_t *st) {
            lds_u8 *da = (lds_u8 *)st + wave * 4096, *db = (lds_u8 *)(st + WB) + wave * (QP * 1024);
            const bool past = step >= steps;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(past ? none : rA, (lds_void *)(da + q * 1024), 16,
                                                         aoff + (uint32_t)q * row4_off + (uint32_t)step * step_off, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < QP; ++q)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(past ? none : rB, (lds_void *)(db + q * 1024), 16, boff[q],
                                                         step * PB, 0, 0);
        };
        f32x16 acc[JN];
#pragma unroll
        for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
        const int i16 = lane & 15, half = (lane >> 4) & 1, rq = i16 >> 2;
        const uint32_t aread = (uint32_t)((8 * hh + rq) * 256 + ((wave ^ rq) * 64) + half * 32 + (i16 & 3) * 8);
        auto multiply = [&](const uint8_t *st) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint8_t *p = st + aread + s * 16 * 256;
                const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)p);
                const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(p + 4 * 256));
                const bf16x8 a = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                const uint32_t o = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
#pragma unroll
                for (int j = 0; j < JN; ++j) {
                    const bf16x8 b = *reinterpret_cast<const bf16x8 *>(st + WB + o + 32 * j * 128);
                    acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[j], 0, 0, 0);
                }
            }
        };
        constexpr int LEFT = (NST - 2) * (4 + QP);
        load(0, S0);
        load(1, S1);
        if (NST > 3) load(2, S2);
        for (int step = 0; step < steps; step += NST) {
            step_barrier<LEFT>();
            load(step + NST - 1, NST > 3 ? S3 : S2);
            multiply(S0);
            step_barrier<LEFT>();
            load(step + NST, S0);
            multiply(S1);
            step_barrier<LEFT>();
            load(step + NST + 1, S1);
            multiply(S2);
            if (NST > 3) {
                step_barrier<LEFT>();
                load(step + NST + 2, S2);
                multiply(S3);
            }
        }
        __builtin_amdgcn_s_waitcnt(0);
        // lane (r32, hh) of tile j holds token 32 j + r32 and columns 32 wave + 8 (v/4) + 4 hh + v%4
        float *out = g.part + (int64_t)blockIdx.x * (MT * 128);
#pragma unroll
        for (int j = 0; j < JN; ++j) {
            if (32 * j + r32 >= count) continue;
#pragma unroll
            for (int v4 = 0; v4 < 4; ++v4)
                *reinterpret_cast<f32x4 *>(out + (32 * j + r32) * 128 + 32 * wave + 8 * v4 + 4 * hh) =
                    f32x4{acc[j][4 * v4], acc[j][4 * v4 + 1], acc[j][4 * v4 + 2], acc[j][4 * v4 + 3]};
        }
    }
};

// More than 128 tokens: two blocks of the vocabulary at a time where single ones would be more than a round of the chip
// (forward, 200 tokens: 32000 x 4096 88 us, one at a time 112; 160 tokens at 4000 x 1024 33, one at a time 24)
__device__ __forceinline__ bool narrow_pairs(int steps) { return steps > 256; }

template <int MT, bool GRAD>
__device__ __forceinline__ void narrow_logits_any(const LossNarrow &g) {
    // 64 tokens: four stages of 16 KB; 128: three of 24 (two workgroups a CU); 256: see there
    constexpr int A = MT == 64 ? 16384 : MT == 128 ? 24576 : 16384, C = MT == 64 ? A : 16, D = MT == 256 ? 32768 : 16;
    __shared__ __align__(16) uint8_t S0[A];
    __shared__ __align__(16) uint8_t S1[A];
    __shared__ __align__(16) uint8_t S2[A];
    __shared__ __align__(16) uint8_t S3[MT == 256 ? D : C];
    __shared__ __align__(16) uint8_t S4[D];
    __shared__ __align__(16) uint8_t S5[D];
    __shared__ float refs[2][MT], sums[2][MT], psums[GRAD ? 2 : 1][MT], tops[2][MT];
    __shared__ int labs[MT], rows[MT], waves[4];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the live rows (M <= 256), by every workgroup for itself; the first writes the list for the launches after
    const int64_t lab64 = tid < g.M ? g.labels[tid] : (int64_t)-1;
    const uint64_t live = __builtin_amdgcn_ballot_w64(lab64 >= 0);
    if (lane == 0) waves[wave] = __popcll(live);
    if (tid < MT) {
        rows[tid] = -1;
        labs[tid] = -1;
        refs[0][tid] = refs[1][tid] = 0.0f;
    }
    __syncthreads();
    int before = 0, count = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        before += w < wave ? waves[w] : 0;
        count += waves[w];
    }
    if (lab64 >= 0) {
        const uint32_t lo = (uint32_t)live, hi = (uint32_t)(live >> 32);
        const int at = before + (int)__builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0u));
        const int size = MT == 256 && count > 128 && narrow_pairs(g.n.steps) ? 128 : 64;
        const int64_t in = lab64 - (int64_t)blockIdx.x * size;
        rows[at] = tid;
        labs[at] = in >= 0 && in < size && lab64 < g.V ? (int)in : -1;
        if (blockIdx.x == 0) {
            g.r.row[at] = tid;
            g.r.label[at] = lab64 < g.V ? (int32_t)lab64 : -1;
        }
    }
    if (blockIdx.x == 0) {
        if (tid == 0) {
            g.r.count[0] = count;
            g.r.count[1] = 0;
        }
        if (tid < g.M && lab64 < 0) g.loss[tid] = 0.0f;
    }
    __syncthreads();
    count = __builtin_amdgcn_readfirstlane(count);
    const NarrowLds<MT> l{{S0, S1, S2, S3, S4, S5}, refs, sums, psums, tops, labs, rows};
    if constexpr (MT > 128)
        if (count > 128) {
            if (!narrow_pairs(g.n.steps)) NarrowLogits<256, MT, 3, 1, GRAD>::run(g, l, count);
            else if (2 * (int)blockIdx.x < g.n.steps) NarrowLogits<256, MT, 3, 2, GRAD>::run(g, l, count);
            return;
        }
    if constexpr (MT > 64)
        if (count > 64) return NarrowLogits<128, MT, 3, 1, GRAD>::run(g, l, count);
    NarrowLogits<64, MT, MT == 64 ? 4 : MT == 128 ? 3 : 6, 1, GRAD>::run(g, l, count);
}

template <int MT>
__device__ __forceinline__ void narrow_dx_any(const LossNarrow &g) {
    constexpr int STAGE = LSTEP * 128 * 2 + MT * LSTEP * 2, NST = MT == 128 ? 4 : 3;
    __shared__ __align__(16) uint8_t S0[STAGE];
    __shared__ __align__(16) uint8_t S1[STAGE];
    __shared__ __align__(16) uint8_t S2[STAGE];
    __shared__ __align__(16) uint8_t S3[NST > 3 ? STAGE : 16];
    const int count = __builtin_amdgcn_readfirstlane(g.r.count[0]);
    if constexpr (MT > 128)
        if (count > 128) return NarrowDx<256, MT, NST>::run(g, S0, S1, S2, S3, count);
    if constexpr (MT > 64)
        if (count > 64) return NarrowDx<128, MT, NST>::run(g, S0, S1, S2, S3, count);
    NarrowDx<64, MT, NST>::run(g, S0, S1, S2, S3, count);
}

// (two workgroups a CU where their LDS allows it)
template <int MT, bool GRAD>
__global__ __launch_bounds__(256, MT <= 128 ? 2 : 1) void loss_narrow_logits_kernel(LossNarrow g) {
    narrow_logits_any<MT, GRAD>(g);
}
template <int MT>
__global__ __launch_bounds__(256, MT == 64 ? 2 : 1) void loss_narrow_dx_kernel(LossNarrow g) {
    narrow_dx_any<MT>(g);
}

// dX of the live rows from the partials, zero for the others (a workgroup for each token and 1024 columns), and by the last
// workgroup the mean
__global__ __launch_bounds__(256) void loss_narrow_fold_kernel(LossNarrow g) {
    const int count = g.r.count[0];
    if (blockIdx.x == gridDim.x - 1) {
        loss_write_mean(g.r.sums, (int)((g.M + kLossJoinRowsNarrow - 1) / kLossJoinRowsNarrow), count, g.mean);
        return;
    }
    const int cols = (int)((g.K + 1023) / 1024), t = (int)blockIdx.x / cols, lane = threadIdx.x & 63;
    const int64_t k = (int64_t)((int)blockIdx.x % cols) * 1024 + threadIdx.x * 4;
    // the token's place among the live ones
    const uint64_t bit = (uint64_t)1 << (t & 63);
    uint64_t own = 0;
    int m = 0;
    for (int w = 0; w <= t / 64; ++w) {
        const int i = 64 * w + lane;
        own = __builtin_amdgcn_ballot_w64(i < g.M && g.labels[i < g.M ? i : 0] >= 0);
        m += __popcll(w < t / 64 ? own : own & (bit - 1));
    }
    if (k >= g.K) return;
    if (!(own & bit)) {
        *reinterpret_cast<uint2 *>(g.dX + (int64_t)t * g.K + k) = uint2{0, 0};
        return;
    }
    const int ntn = (int)((g.K + 127) / 128), MT = g.n.MT, splits = g.n.splits;
    const float *p = g.part + ((k / 128) * MT + m) * 128 + k % 128;
    const int64_t stride = (int64_t)ntn * MT * 128;
    const int32_t lab = g.r.label[m];
    const float a = g.r.a[m], b = g.r.b[m];
    const uint2 w = *reinterpret_cast<const uint2 *>(g.W + (int64_t)max(lab, 0) * g.K + k);
    f32x4 x = {0, 0, 0, 0};
    for (int s0 = 0; s0 < splits; s0 += 8) {
        f32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s0 + u < splits) v[u] = *reinterpret_cast<const f32x4 *>(p + (s0 + u) * stride);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s0 + u < splits) x += v[u];
    }
    // a label out of the vocabulary: a and b are NaN
    *reinterpret_cast<uint2 *>(g.dX + (int64_t)t * g.K + k) = LossFinal{a, b}.value(x, w);
}

}  // namespace

LossNarrowPlan loss_narrow_plan(int64_t M, int64_t V, int64_t K) {
    LossNarrowPlan p;
    p.MT = M <= 64 ? 64 : M <= 128 ? 128 : 256;
    p.steps = (int32_t)((V + LSTEP - 1) / LSTEP);
    const int32_t ntn = (int32_t)((K + 127) / 128), wgs = p.MT == 64 ? 512 : 256;
    int32_t splits = ntn < wgs ? wgs / ntn : 1;
    // at least four steps a workgroup: a partial costs about as much as two
    if (splits > p.steps / 4) splits = p.steps / 4 > 0 ? p.steps / 4 : 1;
    p.per = (p.steps + splits - 1) / splits;
    p.splits = (p.steps + p.per - 1) / p.per;
    p.parts = (size_t)p.splits * ntn * p.MT * 128;
    return p;
}

namespace {
template <bool GRAD>
void narrow_logits_of(const LossNarrow &g, hipStream_t stream) {
    const dim3 grid((uint32_t)g.n.steps), block(256);
    if (g.n.MT == 64) hipLaunchKernelGGL((loss_narrow_logits_kernel<64, GRAD>), grid, block, 0, stream, g);
    else if (g.n.MT == 128) hipLaunchKernelGGL((loss_narrow_logits_kernel<128, GRAD>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((loss_narrow_logits_kernel<256, GRAD>), grid, block, 0, stream, g);
}
}  // namespace

hipError_t launch_loss_narrow_logits(const LossNarrow &g, hipStream_t stream) {
    if (g.P) narrow_logits_of<true>(g, stream);
    else narrow_logits_of<false>(g, stream);
    return hipGetLastError();
}

hipError_t launch_loss_narrow_dx(const LossNarrow &g, hipStream_t stream) {
    const dim3 grid((uint32_t)(g.n.splits * ((g.K + 127) / 128))), block(256);
    if (g.n.MT == 64) hipLaunchKernelGGL(loss_narrow_dx_kernel<64>, grid, block, 0, stream, g);
    else if (g.n.MT == 128) hipLaunchKernelGGL(loss_narrow_dx_kernel<128>, grid, block, 0, stream, g);
    else hipLaunchKernelGGL(loss_narrow_dx_kernel<256>, grid, block, 0, stream, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_narrow_fold_kernel, dim3((uint32_t)(g.M * ((g.K + 1023) / 1024) + 1)), dim3(256), 0, stream, g);
    return hipGetLastError();
}

}  // namespace nf4k
