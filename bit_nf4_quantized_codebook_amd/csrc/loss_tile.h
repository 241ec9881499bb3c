// The MFMA loop of the two products of the loss over the vocabulary: a 256 x 256 tile, 4 waves in 2 x 2,
// each 128 x 128 with v_mfma_f32_32x32x16_bf16 (16 tiles, 256 float32 accumulators), reduction step 64,
// both operands straight from global memory to LDS, two 32 KB stages each.  The schedule is the bf16
// GEMM's (gemm_bf16.hip): fragments are read one sub-step ahead of the MFMAs, the workgroup barrier
// stands before the last sub-step, and a step's loads go out in two halves, spread over the MFMAs.
#pragma once

#include <type_traits>

#include "common.h"
#include "dqtile.h"
#include "loss.h"

namespace nf4k {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// A row's reference is kept while no logit exceeds it by more than about this (log2 units): p stays far from bf16's
// and float32's limits (2^127).  The first is 0, which lies within this of the largest logit of nearly every tile there
// is (33 in natural units); the sums tell where it does not, and such a tile is done once more against its own maxima
// and rescaled afterwards.  (The maximum first and then the sums, as two passes over the accumulators for every tile,
// was slower.)
constexpr int kLossSlack = 48;

// l - c for a logit z: one fma, which keeps the product l = z log2(e) whole.  c is such a product rounded to float32: from
// |c| = 2^28 on that moves it by 16 and more, and soon by more than 2^x takes (2^32: 256).  There the product is rounded as c was,
// so that the largest logit stands within 1 of its reference again.  A tile's first pass, against references below that, needs
// no such choice (far false).
constexpr float kLossFar = 0x1p28f;
__device__ __forceinline__ float loss_above(float z, float c, bool far) {
#pragma clang fp contract(off)
    const float l = z * kLog2e;
    return far && !(fabsf(c) < kLossFar) ? l - c : __builtin_fmaf(z, kLog2e, -c);
}

// the sum or maximum over groups of N lanes (4, 8 or 16), in all of them
template <int N, class Op>
__device__ __forceinline__ float over_lanes(float x, Op op) {
    auto dpp = [](float v, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    x = op(x, dpp(x, std::integral_constant<int, 0xB1>{}));       // lane ^ 1
    x = op(x, dpp(x, std::integral_constant<int, 0x4E>{}));       // lane ^ 2
    if (N >= 8) x = op(x, dpp(x, std::integral_constant<int, 0x141>{}));      // mirrored within 8
    if (N == 16) x = op(x, dpp(x, std::integral_constant<int, 0x140>{}));      // mirrored within 16
    return x;
}

// s + the two bf16 values of v
__device__ __forceinline__ float add_bf16x2(float s, uint32_t v) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, v), bf16x2{(__bf16)1.0f, (__bf16)1.0f}, s, false);
}

// A token's last step: dX = b (a sum P W - W[label]), a = 1 / sum P, rounded once.
struct LossFinal {
    float a, b;
    __device__ __forceinline__ uint2 value(const f32x4 &x, const uint2 &v) const {
        return uint2{pack_bf16x2(b * (a * x[0] - bf16_to_f32(v.x & 0xFFFFu)), b * (a * x[1] - __uint_as_float(v.x & 0xFFFF0000u))),
                     pack_bf16x2(b * (a * x[2] - bf16_to_f32(v.y & 0xFFFFu)), b * (a * x[3] - __uint_as_float(v.y & 0xFFFF0000u)))};
    }
};

// IA: 32-row tiles of a wave along the first operand, 4 or 2 (a tile of 256 or 128 rows there)
template <int IA>
struct LossFrags {
    bf16x8 a[IA], b[4];
};

template <int IA>
__device__ __forceinline__ void loss_mma(const LossFrags<IA> &f, f32x16 acc[IA][4]) {
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// One sub-step's order: an LDS read (of NDS) after each of the first MFMAs, and one of nvmem loads after every second
// (IA = 2: after each).
template <int IA, int NDS>
__device__ __forceinline__ void loss_interleave(int nvmem) {
#pragma unroll
    for (int k = 0; k < 4 * IA; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                             // 1 MFMA
        if (k < NDS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                // 1 DS read
        const int at = IA == 4 ? ((k & 1) ? k >> 1 : 16) : k;
        if (at < nvmem) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);             // 1 VMEM
    }
}

// A stage holds a step's two operands: 32 KB for the first, from LOPB on the second.
constexpr int LOPB = LBLOCK * 2;

// load(step, stage, half): issues half (0 or 1; NV loads) of the loads of both operands of a step; past the last step
// anything that is in range.  read(stage, s, frags): fragments of sub-step s (NDS LDS reads).  On entry step 0 is
// on its way into stage c; where `younger` is set, YOUNGER memory operations were surely issued after its loads.  At the
// end both stages are free.
template <int IA, int NDS, int NV, int YOUNGER, class Load, class Read>
__device__ __forceinline__ void loss_loop(int steps, bool younger, uint8_t *c, uint8_t *n, f32x16 acc[IA][4], Load load, Read read) {
    LossFrags<IA> f0, f1;
    auto step_body = [&](int step, uint8_t *sc, uint8_t *sn) {
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            LossFrags<IA> &cur = (s & 1) ? f1 : f0;
            LossFrags<IA> &nxt = (s & 1) ? f0 : f1;
            if (s == 0) load(step + 1, sn, 1);
            read(sc, s + 1, nxt);
            loss_mma<IA>(cur, acc);
            loss_interleave<IA, NDS>(s == 0 ? NV : 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // step + 1 landed (this wave's loads) and this wave's fragment reads of stage c are done
        __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (0 << 8));
        __syncthreads();
        read(sn, 0, f0);
        load(step + 2, sc, 0);
        loss_mma<IA>(f1, acc);
        loss_interleave<IA, NDS>(NV);
        __builtin_amdgcn_sched_barrier(0);
    };
    load(1, n, 0);
    // gfx9 layout: vmcnt[3:0] | expcnt << 4 | lgkmcnt << 8 | vmcnt[5:4] << 14
    constexpr int left = NV + YOUNGER;
    static_assert(left < 64, "vmcnt's range");
    if (YOUNGER && younger) __builtin_amdgcn_s_waitcnt((left & 15) | (7 << 4) | (0 << 8) | ((left >> 4) << 14));
    else __builtin_amdgcn_s_waitcnt(NV | (7 << 4) | (0 << 8));
    __syncthreads();
    read(c, 0, f0);
    int step = 0;
    for (; step + 1 < steps; step += 2) {
        step_body(step, c, n);
        step_body(step + 1, n, c);
    }
    if (step < steps) step_body(step, c, n);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
}

}  // namespace nf4k
