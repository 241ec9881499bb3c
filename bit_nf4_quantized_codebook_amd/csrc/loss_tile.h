// The MFMA loop of the two products of the loss over the vocabulary: a 256 x 256 tile, 4 waves in 2 x 2,
// each 128 x 128 with v_mfma_f32_32x32x16_bf16 (16 tiles, 256 float32 accumulators), reduction step 64,
// both operands straight from global memory to LDS, two 32 KB stages each.  The schedule is the bf16
// GEMM's (gemm_bf16.hip): fragments are read one sub-step ahead of the MFMAs, the workgroup barrier
// stands before the last sub-step, and a step's loads go out in two halves, spread over the MFMAs.
#pragma once

#include "common.h"
#include "dqtile.h"
#include "loss.h"

namespace nf4k {

typedef __attribute__((address_space(3))) uint8_t lds_u8;

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

// load(step, a, b, half): issues half (0 or 1; NV loads) of the loads of both operands of a step; past the last step they
// read zeros.  read(a, b, s, frags): fragments of sub-step s (NDS LDS reads).
template <int IA, int NDS, int NV, class Load, class Read>
__device__ __forceinline__ void loss_loop(int steps, uint8_t *As0, uint8_t *Bs0, uint8_t *As1, uint8_t *Bs1,
                                          f32x16 acc[IA][4], Load load, Read read) {
    LossFrags<IA> f0, f1;
    auto step_body = [&](int step, uint8_t *Ac, uint8_t *Bc, uint8_t *An, uint8_t *Bn) {
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            LossFrags<IA> &cur = (s & 1) ? f1 : f0;
            LossFrags<IA> &nxt = (s & 1) ? f0 : f1;
            if (s == 0) load(step + 1, An, Bn, 1);
            read(Ac, Bc, s + 1, nxt);
            loss_mma<IA>(cur, acc);
            loss_interleave<IA, NDS>(s == 0 ? NV : 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // step + 1 landed (this wave's loads) and this wave's fragment reads of stage c are done
        __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (0 << 8));
        __syncthreads();
        read(An, Bn, 0, f0);
        load(step + 2, Ac, Bc, 0);
        loss_mma<IA>(f1, acc);
        loss_interleave<IA, NDS>(NV);
        __builtin_amdgcn_sched_barrier(0);
    };
    load(0, As0, Bs0, 0);
    load(0, As0, Bs0, 1);
    load(1, As1, Bs1, 0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    read(As0, Bs0, 0, f0);
    int step = 0;
    for (; step + 1 < steps; step += 2) {
        step_body(step, As0, Bs0, As1, Bs1);
        step_body(step + 1, As1, Bs1, As0, Bs0);
    }
    if (step < steps) step_body(step, As0, Bs0, As1, Bs1);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
}

}  // namespace nf4k
