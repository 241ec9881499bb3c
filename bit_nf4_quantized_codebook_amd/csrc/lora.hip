// Low-rank (LoRA) side products of the QLoRA linear layer (gfx950).
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net),
// section 4 eq. (3) (Y = XW + s X L1 L2) and section 3.5 (gradients for L1, L2 only).
//
// Each product is one streaming pass over an [M, K] or [M, N] activation with a rank-r (<= 128)
// partner, so the kernels are built for HBM bandwidth: a block tile is 64 x 64 outputs, the
// reduction is split over enough block tiles to fill the 256 CUs, every thread keeps four
// reduction steps of 16-byte loads in flight, and float32 partials are summed afterwards in a
// fixed order (deterministic).  Operands sit in LDS in their natural row-major layout; when the
// reduction runs along rows, fragments are read with ds_read_b64_tr_b16 (4 x 16 transposes per
// 16-lane group), so no operand is ever transposed in memory.
//   skinny_nt:  P[ks] = A[:, chunk ks] . B          A [M, Kred];  B = Bk [Kred, R] or Bt [R, Kred]
//   skinny_tn:  P[ms] = U[rows ms, :]^T . V[rows ms, :]    U [M, Pn], V [M, Qn]
// MFMA v_mfma_f32_32x32x16_bf16, 4 waves of 32 x 32.

#include "common.h"
#include "dqtile.h"
#include "launch.h"
#include "reduce.h"
#include "skinny.h"

namespace nf4k {

namespace {

template <bool B_ROWS_K>
__global__ __launch_bounds__(256) void skinny_nt_kernel(const uint16_t *__restrict__ A,
                                                        const uint16_t *__restrict__ B,
                                                        float *__restrict__ P, int64_t M, int32_t R,
                                                        int64_t Kred, int64_t kchunk) {
    skinny_nt_block<B_ROWS_K>(A, B, P, M, R, Kred, kchunk, blockIdx.x, blockIdx.y, blockIdx.z);
}

// P[ms][p][q] = sum_{m in chunk ms} U[m][p] * V[m][q];  U [M, Pn], V [M, Qn] (row-major).
// Both tiles are stored [m][p] / [m][q] and read with transposing fragment loads.
// One launch serves one or two independent products (the backward runs dL2 and dL1 together):
// blocks [0, nb0) take product 0, the rest product 1; within a product, block b is tile
// (b % tx, (b / tx) % ty) of reduction chunk b / (tx ty).
struct TnProb {
    const uint16_t *U, *V;
    float *P;
    uint16_t *out;           // unsplit: bf16(scale * product) here instead of P
    float scale;
    int64_t Pn, Qn, mchunk;
    int32_t tx, ty;
    const uint16_t *Vlo;
};
struct TnGroup {
    TnProb p[2];
    int64_t M;
    uint32_t nb0;
};
// LO: a product may have its V as two bf16 halves; the second is loaded with the first and takes its
// place in LDS after it, so that U is still read once (a tile of its own in LDS: two workgroups a CU
// instead of four, 23.9 against 21.6 us for dL2 + dL1 at 4096 tokens).
template <bool LO>
__global__ __launch_bounds__(256) void skinny_tn_kernel(TnGroup grp) {
    __shared__ __align__(16) uint8_t Us[NSTAGE_TN][ST * ROWB];
    __shared__ __align__(16) uint8_t Vs[NSTAGE_TN][ST * ROWB];
    const int second = blockIdx.x >= grp.nb0;
    const TnProb &pr = grp.p[second];
    const uint16_t *__restrict__ U = pr.U;
    const uint16_t *__restrict__ V = pr.V;
    float *__restrict__ P = pr.P;
    const int64_t M = grp.M, Pn = pr.Pn, Qn = pr.Qn, mchunk = pr.mchunk;
    const uint32_t b = blockIdx.x - (second ? grp.nb0 : 0u);
    const uint32_t bx = b % (uint32_t)pr.tx, by = (b / (uint32_t)pr.tx) % (uint32_t)pr.ty;
    const uint32_t bz = b / ((uint32_t)pr.tx * (uint32_t)pr.ty);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1, r32 = lane & 31, hh = lane >> 5;
    const int64_t p0 = (int64_t)bx * ST;
    const int64_t q0 = (int64_t)by * ST;
    const int64_t mbeg = (int64_t)bz * mchunk;
    const int64_t mend = (mbeg + mchunk < M) ? mbeg + mchunk : M;
    const int64_t rows = mend > mbeg ? mend - mbeg : 0;
    const int nsteps = (int)((rows + ST - 1) / ST);
    // descriptors of this chunk of rows alone: T and dT, [M, r], may pass 2 GiB where X and dY do not (then
    // N and K are below 128, the rows are split 64 ways, and a chunk stays below 2^27 bytes)
    const __amdgpu_buffer_rsrc_t rU = make_rsrc(U + mbeg * Pn, rows * Pn * 2);
    const __amdgpu_buffer_rsrc_t rV = make_rsrc(V + mbeg * Qn, rows * Qn * 2);
    const int trow = tid >> 3, tch = tid & 7;
    const bool pok = p0 + tch * 8 < Pn, qok = q0 + tch * 8 < Qn;

    const bool lo = LO && pr.Vlo;
    const __amdgpu_buffer_rsrc_t rL = make_rsrc((lo ? pr.Vlo : V) + mbeg * Qn, lo ? rows * Qn * 2 : 0);
    auto load = [&](int step, TileLoad &a, TileLoad &b, TileLoad &c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t gm = (int64_t)step * ST + trow + 32 * h;      // row of the chunk
            const bool ok = gm < rows;
            a.v[h] = bload16(rU, (ok && pok) ? (uint32_t)((gm * Pn + p0 + tch * 8) * 2) : 0xFFFFFFF0u);
            b.v[h] = bload16(rV, (ok && qok) ? (uint32_t)((gm * Qn + q0 + tch * 8) * 2) : 0xFFFFFFF0u);
            if (LO) c.v[h] = bload16(rL, (ok && qok && lo) ? (uint32_t)((gm * Qn + q0 + tch * 8) * 2) : 0xFFFFFFF0u);
        }
    };
    auto store = [&](int slot, const TileLoad &a, const TileLoad &b) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = trow + 32 * h;
            *reinterpret_cast<u32x4 *>(&Us[slot][row * ROWB + tch * 16]) = a.v[h];
            *reinterpret_cast<u32x4 *>(&Vs[slot][row * ROWB + tch * 16]) = b.v[h];
        }
    };

    f32x16 acc = {};
    TileLoad la[NSTAGE_TN], lb[NSTAGE_TN], lc[NSTAGE_TN];
    for (int g0 = 0; g0 < nsteps; g0 += NSTAGE_TN) {
#pragma unroll
        for (int u = 0; u < NSTAGE_TN; ++u) load(g0 + u, la[u], lb[u], lc[u]);
#pragma unroll
        for (int u = 0; u < NSTAGE_TN; ++u) store(u, la[u], lb[u]);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NSTAGE_TN; ++u) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const bf16x8 fa = frag_tr(Us[u], wm * 32, s, lane);
                const bf16x8 fb = frag_tr(Vs[u], wn * 32, s, lane);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
            }
        }
        __syncthreads();
        if (LO && lo) {
#pragma unroll
            for (int u = 0; u < NSTAGE_TN; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<u32x4 *>(&Vs[u][(trow + 32 * h) * ROWB + tch * 16]) = lc[u].v[h];
            __syncthreads();
#pragma unroll
            for (int u = 0; u < NSTAGE_TN; ++u)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag_tr(Us[u], wm * 32, s, lane),
                                                                 frag_tr(Vs[u], wn * 32, s, lane), acc, 0, 0, 0);
            __syncthreads();
        }
    }
    const int64_t col = q0 + wn * 32 + r32;
    if (col < Qn && pr.out) {
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int64_t row = p0 + wm * 32 + (v >> 2) * 8 + hh * 4 + (v & 3);
            if (row < Pn) pr.out[row * Qn + col] = (uint16_t)f32_to_bf16(pr.scale * acc[v]);
        }
    } else if (col < Qn) {
        float *Pk = P + (int64_t)bz * Pn * Qn;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
            const int64_t row = p0 + wm * 32 + (v >> 2) * 8 + hh * 4 + (v & 3);
            if (row < Pn) Pk[row * Qn + col] = acc[v];
        }
    }
}

// One launch serves one to three reductions: blocks [0, nb[0]) take the first, the next nb[1] the
// second, the rest the third.
struct RedGroup {
    RedProb p[3];
    uint32_t nb[3];
};
__global__ __launch_bounds__(256) void reduce_partials_kernel(RedGroup grp) {
    uint32_t b = blockIdx.x;
    const int i = b < grp.nb[0] ? 0 : (b < grp.nb[0] + grp.nb[1] ? 1 : 2);
    if (i >= 1) b -= grp.nb[0];
    if (i == 2) b -= grp.nb[1];
    reduce_partials_block(grp.p[i], b, grp.nb[i]);
}

}  // namespace

int choose_split(int64_t tiles, int64_t red_steps) {
    // aim for >= 512 block tiles in flight, each with >= 8 reduction steps
    int64_t s = (512 + tiles - 1) / tiles;
    if (s > red_steps / 8) s = red_steps / 8;
    if (s < 1) s = 1;
    if (s > 64) s = 64;
    return (int)s;
}

hipError_t launch_skinny_nt(const uint16_t *A, const uint16_t *B, bool b_rows_k, float *P, int64_t M,
                            int32_t R, int64_t Kred, int nsplit, hipStream_t stream) {
    const int64_t steps = (Kred + ST - 1) / ST;
    const int64_t per = (steps + nsplit - 1) / nsplit;
    dim3 grid((unsigned)((M + ST - 1) / ST), (unsigned)((R + ST - 1) / ST), (unsigned)nsplit);
    if (b_rows_k)
        hipLaunchKernelGGL(skinny_nt_kernel<true>, grid, dim3(256), 0, stream, A, B, P, M, R, Kred, per * ST);
    else
        hipLaunchKernelGGL(skinny_nt_kernel<false>, grid, dim3(256), 0, stream, A, B, P, M, R, Kred, per * ST);
    return hipGetLastError();
}

namespace {
TnProb tn_prob(const TnProduct &t, int64_t M, uint32_t &nblocks) {
    const int64_t steps = (M + ST - 1) / ST;
    const int64_t per = (steps + t.nsplit - 1) / t.nsplit;
    TnProb p;
    p.U = t.U; p.V = t.V; p.P = t.P; p.Pn = t.Pn; p.Qn = t.Qn; p.mchunk = per * ST;
    p.out = t.nsplit == 1 ? t.out : nullptr;
    p.scale = t.scale;
    p.Vlo = t.Vlo;
    p.tx = (int32_t)((t.Pn + ST - 1) / ST);
    p.ty = (int32_t)((t.Qn + ST - 1) / ST);
    nblocks = (uint32_t)p.tx * (uint32_t)p.ty * (uint32_t)t.nsplit;
    return p;
}
}  // namespace

RedProb red_prob(const Reduction &r, uint32_t &nblocks) {
    RedProb p;
    p.P = r.P; p.n = r.n; p.out = r.out; p.out2 = r.out2; p.s1 = r.s1; p.s2 = r.s2; p.nsplit = r.nsplit;
    p.stride = r.stride ? r.stride : r.n;
    p.accum = r.accum ? 1u : 0u;
    p.lo2 = r.lo2;
    nblocks = reduce_blocks(r.n);
    return p;
}

SplitPlan gemm_split(int64_t tiles, int64_t steps, int quantum) {
    int64_t s = tiles > 0 ? 256 / tiles : 1;
    const int64_t smax = steps / quantum;
    if (s > smax) s = smax;
    if (s > 16) s = 16;
    if (s < 1) s = 1;
    int64_t per = (steps + s - 1) / s;
    per = (per + quantum - 1) / quantum * quantum;
    s = (steps + per - 1) / per;   // rounding per up may leave the last splits empty: drop them
    if (s <= 1) return SplitPlan{1, steps};
    return SplitPlan{(int)s, per};
}

hipError_t launch_skinny_tn(const TnProduct &a, const TnProduct *b, int64_t M, hipStream_t stream) {
    TnGroup g;
    uint32_t n0 = 0, n1 = 0;
    g.p[0] = tn_prob(a, M, n0);
    g.p[1] = b ? tn_prob(*b, M, n1) : g.p[0];
    g.M = M;
    g.nb0 = n0;
    if (a.Vlo || (b && b->Vlo))
        hipLaunchKernelGGL(skinny_tn_kernel<true>, dim3(n0 + (b ? n1 : 0u)), dim3(256), 0, stream, g);
    else
        hipLaunchKernelGGL(skinny_tn_kernel<false>, dim3(n0 + (b ? n1 : 0u)), dim3(256), 0, stream, g);
    return hipGetLastError();
}

hipError_t launch_reduce_partials(const Reduction &a, const Reduction *b, hipStream_t stream, const Reduction *c) {
    RedGroup g;
    const Reduction *rs[3] = {&a, b, c};
    uint32_t total = 0;
    int used = 0;
    for (int i = 0; i < 3; ++i) {
        if (!rs[i]) continue;
        g.p[used] = red_prob(*rs[i], g.nb[used]);
        total += g.nb[used];
        ++used;
    }
    for (int i = used; i < 3; ++i) {
        g.p[i] = g.p[0];
        g.nb[i] = 0;
    }
    hipLaunchKernelGGL(reduce_partials_kernel, dim3(total), dim3(256), 0, stream, g);
    return hipGetLastError();
}

}  // namespace nf4k
