// The loss for up to 128 tokens, forward (from 17) and with its gradient (gfx950): both products stream the weight, and
// tiles of 256 tokens with two stages in flight leave the memory idle.  Tiles here are narrow and their stages many:
//   1. logits: 64 vocabulary rows x TT tokens (64 or 128) a workgroup, two workgroups a CU.  Each makes the list of live
//      rows for itself, from at most 128 labels;
//   2. the join of the tiles (loss.hip);
//   3. dX's product: 128 columns x TT tokens over a part of the vocabulary, float32 partials;
//   4. their sum, dX, and the mean (forward: the mean alone).
// The layouts of p, of the LDS stages and of the fragments are those of loss_logits.hip and loss_dx.hip.
//
// Bound by HBM: forward 37 x 50001 x 4096 101 us a call (logits 90: 4.5 TB/s), 100 x 32000 x 4096 71 (90 on tiles of 256);
// with the gradient, which reads the weight twice, 16, 64 and 100 x 32000 x 4096 108, 120 and 131 (147, 156 and 169 on
// tiles of 256), 100 x 4000 x 1024 29 (57).

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
    static_assert(LEFT < 16, "vmcnt's low bits");
    __builtin_amdgcn_s_waitcnt(LEFT | (7 << 4) | (0 << 8));
    asm volatile("s_barrier" ::: "memory");
}

template <int TT, bool GRAD>
__device__ __forceinline__ void narrow_logits(const LossNarrow &g) {
    constexpr int NST = TT == 64 ? 4 : 3;            // stages; NST - 1 of them in flight
    constexpr int VB = 64 * LSTEP * 2;               // bytes of W in a stage, before the tokens'
    constexpr int JN = TT / 64;                      // 32-token tiles of a wave
    constexpr int QX = TT / 32;                      // a wave's loads of X a step (of W: 2)
    __shared__ __align__(16) uint8_t S0[VB + TT * LSTEP * 2];
    __shared__ __align__(16) uint8_t S1[VB + TT * LSTEP * 2];
    __shared__ __align__(16) uint8_t S2[VB + TT * LSTEP * 2];
    __shared__ __align__(16) uint8_t S3[NST > 3 ? VB + TT * LSTEP * 2 : 16];
    __shared__ float refs[TT], sums[2][TT], tops[2][TT];
    __shared__ int labs[TT], rows[TT], waves[4];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;         // along the vocabulary, along the tokens
    const int r32 = lane & 31, hh = lane >> 5;
    const int64_t n0 = (int64_t)blockIdx.x * 64;

    // the live rows (M <= TT), by every workgroup for itself; the first writes the list for the launches after
    const int64_t lab64 = tid < g.M ? g.labels[tid] : (int64_t)-1;
    const uint64_t live = __builtin_amdgcn_ballot_w64(lab64 >= 0);
    if (lane == 0) waves[wave] = __popcll(live);
    if (tid < TT) {
        rows[tid] = -1;
        labs[tid] = -1;
        refs[tid] = 0.0f;
    }
    __syncthreads();
    int before = 0, count = 0;
#pragma unroll
    for (int w = 0; w < TT / 64; ++w) {
        before += w < wave ? waves[w] : 0;
        count += waves[w];
    }
    if (lab64 >= 0) {
        const uint32_t lo = (uint32_t)live, hi = (uint32_t)(live >> 32);
        const int at = before + (int)__builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0u));
        const int64_t in = lab64 - n0;
        rows[at] = tid;
        labs[at] = in >= 0 && in < 64 && lab64 < g.V ? (int)in : -1;
        if (blockIdx.x == 0) {
            g.r.row[at] = tid;
            g.r.label[at] = lab64 < g.V ? (int32_t)lab64 : -1;
        }
    }
    if (blockIdx.x == 0 && tid == 0) g.r.count[0] = count;
    __syncthreads();

    // rows of W past V read zeros; dead tokens too
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + n0 * g.K, (g.V - n0) * g.K * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.X, 0x7FFFFFF0LL);
    const __amdgpu_buffer_rsrc_t none = make_rsrc(g.X, 0);
    const int l8 = lane >> 3;
    // instruction q of a wave writes stage rows 8u .. 8u+7 (u = Q wave + q, Q even); lane l takes row 8u + l/8 and
    // physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8)
    auto chunk = [&](int q) { return (uint32_t)(((lane & 7) ^ ((4 * q + (l8 >> 1)) & 7)) * 16); };
    uint32_t voff[2], xoff[QX];
#pragma unroll
    for (int q = 0; q < 2; ++q) voff[q] = (uint32_t)(8 * (2 * wave + q) + l8) * (uint32_t)(g.K * 2) + chunk(q);
#pragma unroll
    for (int q = 0; q < QX; ++q) {
        const int row = rows[8 * (QX * wave + q) + l8];
        xoff[q] = row >= 0 ? (uint32_t)row * (uint32_t)(g.K * 2) + chunk(q) : 0x80000000u;
    }
    const int steps = (int)(g.K / LSTEP);
    auto load = [&](int step, uint8_t *st) {
        lds_u8 *da = (lds_u8 *)st + wave * 2048, *db = (lds_u8 *)(st + VB) + wave * (QX * 1024);
        const int at = step * (LSTEP * 2);
        const bool past = step >= steps;             // zeros, without memory
#pragma unroll
        for (int q = 0; q < 2; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(past ? none : rA, (lds_void *)(da + q * 1024), 16, voff[q], at, 0, 0);
#pragma unroll
        for (int q = 0; q < QX; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(past ? none : rB, (lds_void *)(db + q * 1024), 16, xoff[q], at, 0, 0);
    };
    f32x16 acc[JN];
#pragma unroll
    for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
    auto multiply = [&](const uint8_t *st) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t o = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
            const bf16x8 a = *reinterpret_cast<const bf16x8 *>(st + o + 32 * wm * 128);
#pragma unroll
            for (int j = 0; j < JN; ++j) {
                const bf16x8 b = *reinterpret_cast<const bf16x8 *>(st + VB + o + (32 * JN * wn + 32 * j) * 128);
                acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc[j], 0, 0, 0);
            }
        }
    };
    // The stage of step s is free for step s + NST after the barrier of step s + 1.  Steps past the last multiply zeros.
    constexpr int LEFT = (NST - 2) * (2 + QX);
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
    __syncthreads();

    // ---- epilogue, as in loss_logits.hip: each wave turns its 32 vocabulary rows x 32 JN tokens through LDS, rows of 128
    // bytes; four lanes then hold a token's 32, eight each ----
    uint8_t *lds = (wave < 2 ? S0 : S1) + (wave & 1) * (32 * JN * 128);
    auto piece = [](int p, int token) { return (p ^ ((token >> 1) & 7)) * 16; };
#pragma unroll
    for (int j = 0; j < JN; ++j)
#pragma unroll
        for (int v4 = 0; v4 < 4; ++v4)
            *reinterpret_cast<f32x4 *>(lds + (32 * j + r32) * 128 + piece(2 * v4 + hh, r32)) =
                f32x4{acc[j][4 * v4], acc[j][4 * v4 + 1], acc[j][4 * v4 + 2], acc[j][4 * v4 + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int B = 2 * JN;                        // 16 tokens at a time
    const int q = lane & 3, tt = lane >> 2;
    const int64_t left = g.V - n0 - 32 * wm;
    const int end = (int)min(max(left - 8 * q, (int64_t)0), (int64_t)8);
    float z[B][8];
    int lab[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int token = 16 * b + tt, tl = 32 * JN * wn + token;
        const f32x4 lo = *reinterpret_cast<const f32x4 *>(lds + token * 128 + piece(2 * q, token));
        const f32x4 hi = *reinterpret_cast<const f32x4 *>(lds + token * 128 + piece(2 * q + 1, token));
        lab[b] = labs[tl] < 0 ? -1 : labs[tl] - 32 * wm - 8 * q;
#pragma unroll
        for (int k = 0; k < 8; ++k) z[b][k] = k < 4 ? lo[k & 3] : hi[k & 3];
    }
    auto largest = [&]() {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            float x = -__builtin_inff();
#pragma unroll
            for (int k = 0; k < 8; ++k) x = fmaxf(x, k < end ? z[b][k] : -__builtin_inff());
            x = over_lanes<4>(x, [](float a, float b) { return fmaxf(a, b); });
            tops[wm][32 * JN * wn + 16 * b + tt] = x;
        }
    };
    const __amdgpu_buffer_rsrc_t rP = make_rsrc(GRAD ? g.P + (int64_t)blockIdx.x * LBLOCK : nullptr, GRAD ? LBLOCK * 2 : 0);
    auto groups = [&]() {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int tl = 32 * JN * wn + 16 * b + tt;
            const float c = refs[tl];
            float e[8], s = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (lab[b] == k) g.r.zl[tl] = z[b][k] * kLog2e;
                e[k] = lab[b] == k || k >= end ? 0.0f : __builtin_amdgcn_exp2f(__builtin_fmaf(z[b][k], kLog2e, -c));
                s += e[k];
            }
            s = over_lanes<4>(s, [](float a, float b) { return a + b; });
            sums[wm][tl] = s;                        // the same from all of a token's lanes
            if (GRAD) __builtin_amdgcn_raw_buffer_store_b128(
                u32x4{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]), pack_bf16x2(e[6], e[7])}, rP,
                (uint32_t)(tl * 128 + (((4 * wm + q) ^ ((tl >> 1) & 7)) * 16)), 0, 0);
        }
        __syncthreads();
    };
    groups();
    const int t = tid < TT ? tid : 0;
    float sum = sums[0][t] + sums[1][t];
    const bool ok = t >= count || (sum <= __builtin_ldexpf(1.0f, kLossSlack) && sum >= __builtin_ldexpf(1.0f, -kLossSlack));
    if (!__syncthreads_and(ok)) {
        largest();
        __syncthreads();
        const float most = fmaxf(tops[0][t], tops[1][t]);
        if (tid < TT && !ok && most > -__builtin_inff()) refs[t] = ceilf(most * kLog2e);
        __syncthreads();
        groups();
        sum = sums[0][t] + sums[1][t];
    }
    if (tid < count) {
        const int64_t o = (int64_t)tid * g.steps + blockIdx.x;
        g.tref[o] = refs[tid];
        g.tsum[o] = sum;
    }
}

// D[t, n] of 128 columns and all tokens over `per` steps of the vocabulary: workgroup (split, tn)
template <int TT>
__device__ __forceinline__ void narrow_dx(const LossNarrow &g) {
    constexpr int NST = TT == 64 ? 3 : 4;
    constexpr int WB = LSTEP * 128 * 2;              // bytes of W in a stage, before P's
    constexpr int JN = TT / 32;
    constexpr int QP = TT / 32;                      // a wave's loads of P a step (of W: 4)
    __shared__ __align__(16) uint8_t S0[WB + TT * LSTEP * 2];
    __shared__ __align__(16) uint8_t S1[WB + TT * LSTEP * 2];
    __shared__ __align__(16) uint8_t S2[WB + TT * LSTEP * 2];
    __shared__ __align__(16) uint8_t S3[NST > 3 ? WB + TT * LSTEP * 2 : 16];
    const int count = __builtin_amdgcn_readfirstlane(g.r.count[0]);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r32 = lane & 31, hh = lane >> 5;
    const int ntn = (int)((g.K + 127) / 128);
    const int split = (int)blockIdx.x / ntn, tn = (int)blockIdx.x % ntn;
    const int kb = split * g.per, steps = min(g.steps - kb, g.per);
    const int64_t n0 = (int64_t)tn * 128, v0 = (int64_t)kb * LSTEP;

    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + v0 * g.K, (g.V - v0) * g.K * 2);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.P + (int64_t)kb * LBLOCK, (int64_t)steps * LBLOCK * 2);
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
                                                     step * (int)(LBLOCK * 2), 0, 0);
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
        step_barrier<(LEFT < 16 ? LEFT : 15)>();
        load(step + NST - 1, NST > 3 ? S3 : S2);
        multiply(S0);
        step_barrier<(LEFT < 16 ? LEFT : 15)>();
        load(step + NST, S0);
        multiply(S1);
        step_barrier<(LEFT < 16 ? LEFT : 15)>();
        load(step + NST + 1, S1);
        multiply(S2);
        if (NST > 3) {
            step_barrier<(LEFT < 16 ? LEFT : 15)>();
            load(step + NST + 2, S2);
            multiply(S3);
        }
    }
    __builtin_amdgcn_s_waitcnt(0);
    // lane (r32, hh) of tile j holds token 32 j + r32 and columns 32 wave + 8 (v/4) + 4 hh + v%4
    float *out = g.part + (int64_t)blockIdx.x * (TT * 128);
#pragma unroll
    for (int j = 0; j < JN; ++j) {
        if (32 * j + r32 >= count) continue;
#pragma unroll
        for (int v4 = 0; v4 < 4; ++v4)
            *reinterpret_cast<f32x4 *>(out + (32 * j + r32) * 128 + 32 * wave + 8 * v4 + 4 * hh) =
                f32x4{acc[j][4 * v4], acc[j][4 * v4 + 1], acc[j][4 * v4 + 2], acc[j][4 * v4 + 3]};
    }
}

template <int TT, bool GRAD>
__global__ __launch_bounds__(256, 2) void loss_narrow_logits_kernel(LossNarrow g) {
    narrow_logits<TT, GRAD>(g);
}
template <int TT>
__global__ __launch_bounds__(256, TT == 64 ? 2 : 1) void loss_narrow_dx_kernel(LossNarrow g) {
    narrow_dx<TT>(g);
}

// dX of the live rows from the partials, zero for the others (a workgroup for each token and 1024 columns), and by the last
// workgroup the mean
__global__ __launch_bounds__(256) void loss_narrow_fold_kernel(LossNarrow g, int TT) {
    const int count = g.r.count[0];
    if (blockIdx.x == gridDim.x - 1) {
        loss_write_mean(g.r.sums, (int)((g.M + kLossJoinRowsNarrow - 1) / kLossJoinRowsNarrow), count, g.mean);
        return;
    }
    const int cols = (int)((g.K + 1023) / 1024), t = (int)blockIdx.x / cols, lane = threadIdx.x & 63;
    const int64_t k = (int64_t)((int)blockIdx.x % cols) * 1024 + threadIdx.x * 4;
    // the token's place among the live ones
    const uint64_t live0 = __builtin_amdgcn_ballot_w64(lane < g.M && g.labels[lane < g.M ? lane : 0] >= 0);
    const uint64_t live1 = __builtin_amdgcn_ballot_w64(64 + lane < g.M && g.labels[64 + lane < g.M ? 64 + lane : 0] >= 0);
    const uint64_t own = t < 64 ? live0 : live1, bit = (uint64_t)1 << (t & 63);
    const int m = __popcll(own & (bit - 1)) + (t < 64 ? 0 : __popcll(live0));
    if (k >= g.K) return;
    if (!(own & bit)) {
        *reinterpret_cast<uint2 *>(g.dX + (int64_t)t * g.K + k) = uint2{0, 0};
        if (k == 0) g.loss[t] = 0.0f;
        return;
    }
    const int ntn = (int)((g.K + 127) / 128), splits = (g.steps + g.per - 1) / g.per;
    const float *p = g.part + ((k / 128) * TT + m) * 128 + k % 128;
    const int64_t stride = (int64_t)ntn * TT * 128;
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

// forward: the mean, and the losses of tokens without a label
__global__ __launch_bounds__(256) void loss_narrow_mean_kernel(LossNarrow g) {
    if ((int)threadIdx.x < g.M && g.labels[threadIdx.x] < 0) g.loss[threadIdx.x] = 0.0f;
    loss_write_mean(g.r.sums, (int)((g.M + kLossJoinRowsNarrow - 1) / kLossJoinRowsNarrow), g.r.count[0], g.mean);
}

}  // namespace

LossNarrowPlan loss_narrow_plan(int64_t M, int64_t V, int64_t K) {
    LossNarrowPlan p;
    p.TT = M <= 64 ? 64 : 128;
    p.steps = (int32_t)((V + LSTEP - 1) / LSTEP);
    const int32_t ntn = (int32_t)((K + 127) / 128), wgs = p.TT == 64 ? 512 : 256;
    int32_t splits = ntn < wgs ? wgs / ntn : 1;
    // at least four steps a workgroup: a partial costs about as much as two
    if (splits > p.steps / 4) splits = p.steps / 4 > 0 ? p.steps / 4 : 1;
    p.per = (p.steps + splits - 1) / splits;
    p.splits = (p.steps + p.per - 1) / p.per;
    p.parts = (size_t)p.splits * ntn * p.TT * 128;
    return p;
}

hipError_t launch_loss_narrow_logits(const LossNarrow &g, hipStream_t stream) {
    const dim3 grid((uint32_t)g.steps), block(256);
    if (g.P && g.M <= 64) hipLaunchKernelGGL((loss_narrow_logits_kernel<64, true>), grid, block, 0, stream, g);
    else if (g.P) hipLaunchKernelGGL((loss_narrow_logits_kernel<128, true>), grid, block, 0, stream, g);
    else if (g.M <= 64) hipLaunchKernelGGL((loss_narrow_logits_kernel<64, false>), grid, block, 0, stream, g);
    else hipLaunchKernelGGL((loss_narrow_logits_kernel<128, false>), grid, block, 0, stream, g);
    return hipGetLastError();
}

hipError_t launch_loss_narrow_mean(const LossNarrow &g, hipStream_t stream) {
    hipLaunchKernelGGL(loss_narrow_mean_kernel, dim3(1), dim3(256), 0, stream, g);
    return hipGetLastError();
}

hipError_t launch_loss_narrow_dx(const LossNarrow &g, hipStream_t stream) {
    const int ntn = (int)((g.K + 127) / 128), splits = (g.steps + g.per - 1) / g.per, TT = g.M <= 64 ? 64 : 128;
    if (TT == 64) hipLaunchKernelGGL(loss_narrow_dx_kernel<64>, dim3((uint32_t)(splits * ntn)), dim3(256), 0, stream, g);
    else hipLaunchKernelGGL(loss_narrow_dx_kernel<128>, dim3((uint32_t)(splits * ntn)), dim3(256), 0, stream, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_narrow_fold_kernel, dim3((uint32_t)(g.M * ((g.K + 1023) / 1024) + 1)), dim3(256), 0, stream, g, TT);
    return hipGetLastError();
}

}  // namespace nf4k
