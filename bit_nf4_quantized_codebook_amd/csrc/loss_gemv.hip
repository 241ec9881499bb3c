// Loss over the vocabulary for up to 16 tokens, forward (gfx950): W's 2 V K bytes stream once from HBM, and
// everything else stays out of the way of those loads.  Two launches:
//   1. logits and statistics.  A workgroup of 4 waves owns 16 RG vocabulary rows; the waves take turns along K
//      (256-byte chunks, wave w takes chunks w, w + 4, ..), a chunk loaded while the one before it is multiplied
//      (v_mfma_f32_16x16x32_bf16: 16 vocabulary rows by 16 tokens).  A row's bytes go from the load
//      straight into the MFMA.  The waves' sums meet in LDS in a fixed order; then each token's maximum and its sum of
//      2^(l - c) over the 16 rows;
//   2. a workgroup per token joins its tiles, and the one that ends last sums the losses.
// All tokens are computed, also those without a label: the weight's stream costs the same.
//
// Bound by HBM: one token at 32000 x 4096 43 us (6.1 TB/s) and 4 for the join.

#include "common.h"
#include "dqtile.h"
#include "loss.h"
#include "loss_tile.h"

namespace nf4k {

namespace {

constexpr int CHUNK = 256;         // bytes of K per wave and turn
constexpr int CS = CHUNK / 64;     // MFMA steps of a chunk
constexpr int NW = 4;

// DIRECT (up to 4 tokens): the tokens are loaded in the operands' own layout, too few lines to matter.
template <int RG, bool DIRECT>
__global__ __launch_bounds__(NW * 64) void loss_gemv_kernel(LossGemv g) {
    // a wave's tokens of a chunk, and after the last its sums [16 rows][4][lane]
    constexpr int XW = DIRECT ? RG * 1024 : 4096;
    static_assert(RG <= 4, "a wave's sums fit where its tokens were");
    __shared__ __align__(16) uint8_t xtile[NW * XW];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ln = lane & 15, lg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RG);
    const uint32_t KB = (uint32_t)(g.K * 2);           // bytes of a row
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(g.W + n0 * g.K, (g.V - n0) * g.K * 2);
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(g.X, g.M * g.K * 2);
    const int nchunk = (int)((KB + CHUNK - 1) / CHUNK);
    if (blockIdx.x == 0 && tid == 0) g.done[0] = 0;

    // Vocabulary rows: lane (ln, lg) of step s loads bytes 64 s + 16 lg .. +15 of row ln, which is its
    // operand.  Rows past V, tokens past M and bytes past K read zeros.
    struct WStage {
        u32x4 w[CS][RG];
    };
    const uint32_t lane_off = (uint32_t)ln * KB + lg * 16;
    auto load_w = [&](int c, WStage &st) {
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            const uint32_t k = (uint32_t)c * CHUNK + s * 64;
#pragma unroll
            for (int q = 0; q < RG; ++q) st.w[s][q] = bload16(rW, k < KB ? lane_off + k + q * 16 * KB : 0xFFFFFFF0u);
        }
    };
    // Tokens: 16 lanes load a row's 256 bytes (four rows per load), and the wave turns them into operands through
    // its own LDS tile, 16-byte pieces XOR-ed with the row so that neither side has bank conflicts.
    u32x4 xr[4];
    auto load_x = [&](int c) {
        if (DIRECT) {
#pragma unroll
            for (int s = 0; s < CS; ++s) {
                const uint32_t k = (uint32_t)c * CHUNK + s * 64;
                xr[s] = bload16(rX, k < KB ? lane_off + k : 0xFFFFFFF0u);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * i + lg;
            const uint32_t k = (uint32_t)c * CHUNK + ((ln ^ row) * 16);
            xr[i] = bload16(rX, k < KB ? (uint32_t)row * KB + k : 0xFFFFFFF0u);
        }
    };
    uint8_t *xt = xtile + wave * XW;
    f32x4 acc[RG];
#pragma unroll
    for (int a = 0; a < RG; ++a) acc[a] = f32x4{0, 0, 0, 0};
    // The tile is the wave's own: its LDS operations complete in order, so no barrier is needed, only that the
    // compiler keeps the order of one lane's writes and another's reads.
    auto wave_order = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    u32x4 xd[CS];
    auto put_x = [&]() {
        if (DIRECT) {
#pragma unroll
            for (int s = 0; s < CS; ++s) xd[s] = xr[s];
            return;
        }
        wave_order();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4 *>(xt + i * 1024 + lane * 16) = xr[i];
        wave_order();
    };
    auto mul = [&](const WStage &st) {
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            const bf16x8 x = DIRECT ? __builtin_bit_cast(bf16x8, xd[s])
                                    : *reinterpret_cast<const bf16x8 *>(xt + ln * 256 + (((4 * s + lg) ^ ln) * 16));
#pragma unroll
            for (int a = 0; a < RG; ++a)
                acc[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, st.w[s][a]), x, acc[a], 0, 0, 0);
        }
    };

    WStage s0, s1;
    load_w(wave, s0);
    load_x(wave);
    // Chunks past the end load nothing and add zeros.
    for (int c = wave; c < nchunk; c += 2 * NW) {
        put_x();
        load_x(c + NW);
        load_w(c + NW, s1);
        mul(s0);
        put_x();
        load_x(c + 2 * NW);
        load_w(c + 2 * NW, s0);
        mul(s1);
    }
    wave_order();
#pragma unroll
    for (int a = 0; a < RG; ++a) *reinterpret_cast<f32x4 *>(xt + a * 1024 + lane * 16) = acc[a];
    __syncthreads();

    // wave 0: lane (ln, lg) holds token ln, vocabulary rows 16 a + 4 lg + v
    if (wave) return;
    const int t = ln;
    f32x4 z[RG];
    const int64_t lab = t < g.M ? g.labels[t] : -1;
    float top = -__builtin_inff(), s = 0.0f;
#pragma unroll
    for (int a = 0; a < RG; ++a) {
        z[a] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < NW; ++w) z[a] += *reinterpret_cast<const f32x4 *>(xtile + w * XW + a * 1024 + lane * 16);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t n = n0 + 16 * a + 4 * lg + v;
            if (n < g.V && n != lab) top = fmaxf(top, z[a][v]);
            if (n == lab) g.zl[t] = z[a][v] * kLog2e;
        }
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    top = top > -__builtin_inff() ? ceilf(top * kLog2e) : 0.0f;      // none: a sum of zero, which the join passes over
#pragma unroll
    for (int a = 0; a < RG; ++a)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t n = n0 + 16 * a + 4 * lg + v;
            s += n < g.V && n != lab ? __builtin_amdgcn_exp2f(loss_above(z[a][v], top, true)) : 0.0f;
        }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lg == 0 && t < g.M) g.table[(int64_t)t * gridDim.x + blockIdx.x] = float2{top, s};
}

__global__ __launch_bounds__(256) void loss_gemv_join_kernel(LossGemv g, int ntile) {
    __shared__ float pc[4], ps[4];
    const int t = blockIdx.x, tid = threadIdx.x;
    const int64_t lab = g.labels[t];
    const float NEG = -__builtin_inff();
    const float2 *tab = g.table + (int64_t)t * ntile;
    float c = NEG, sum = 0.0f;
    for (int i0 = tid; i0 < ntile; i0 += 256 * 8) {
        float2 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = i0 + 256 * u < ntile ? tab[i0 + 256 * u] : float2{NEG, 0.0f};
        float m = c;
#pragma unroll
        for (int u = 0; u < 8; ++u) m = fmaxf(m, v[u].y != 0.0f ? v[u].x : NEG);
        sum *= m == c ? 1.0f : __builtin_amdgcn_exp2f(c - m);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (v[u].y != 0.0f) sum += v[u].y * __builtin_amdgcn_exp2f(v[u].x - m);
        c = m;
    }
    auto join = [&](float c2, float s2) {
        const float m = fmaxf(c, c2);
        sum = (c == m ? sum : sum * __builtin_amdgcn_exp2f(c - m)) + (c2 == m ? s2 : s2 * __builtin_amdgcn_exp2f(c2 - m));
        c = m;
    };
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float c2 = __shfl_xor(c, d), s2 = __shfl_xor(sum, d);
        join(c2, s2);
    }
    if ((tid & 63) == 0) {
        pc[tid >> 6] = c;
        ps[tid >> 6] = sum;
    }
    __syncthreads();
    if (tid >= 64) return;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w == 0) {
            c = pc[0];
            sum = ps[0];
        } else {
            join(pc[w], ps[w]);
        }
    }
    // (a label's logit that is not finite: NaN; d would be infinite)
    const float zl = g.zl[t];
    const float d = (log2f(sum) + (c - zl)) * kLn2;
    const float loss = lab < 0 ? 0.0f : (lab < g.V && fabsf(zl) < __builtin_inff() ? fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d))) : __builtin_nanf(""));
    if (tid == 0) g.loss[t] = loss;
    if (g.M == 1) {
        if (tid == 0) g.mean[0] = loss;
        return;
    }
    int last = 0;
    if (tid == 0) {
        __hip_atomic_store(&g.each[t], loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = __hip_atomic_fetch_add(g.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1 == (int)gridDim.x;
    }
    if (!__builtin_amdgcn_readfirstlane(last)) return;
    // the workgroup that ends last: one loss a lane, summed in a fixed order
    __shared__ double each[64];
    const bool has = tid < g.M && g.labels[tid < g.M ? tid : 0] >= 0;
    const int count = __popcll(__builtin_amdgcn_ballot_w64(has));
    each[tid] = tid < g.M ? (double)__hip_atomic_load(&g.each[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (tid) return;
    double total = 0.0;
    for (int i = 0; i < (int)g.M; ++i) total += each[i];
    g.mean[0] = count ? (float)(total / count) : 0.0f;
}

template <int RG, bool DIRECT>
hipError_t run(const LossGemv &g, hipStream_t stream) {
    const uint32_t tiles = (uint32_t)((g.V + 16 * RG - 1) / (16 * RG));
    hipLaunchKernelGGL((loss_gemv_kernel<RG, DIRECT>), dim3(tiles), dim3(NW * 64), 0, stream, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(loss_gemv_join_kernel, dim3((uint32_t)g.M), dim3(256), 0, stream, g, (int)tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_loss_gemv(const LossGemv &g, hipStream_t stream) {
    // Weight rows of a workgroup: 16 while the weight's stream is all there is (many small workgroups hide its latency:
    // one token at 50001 x 4096 takes 77 us with 16 rows, 90 with 48), more where the tokens' LDS traffic counts (16
    // tokens at 131072 x 4096 230 us with 16 rows, 204 with 48).  Beyond 16 tokens the narrow tiles are faster (33 at
    // 32000 x 4096 61 us, 70 here).
    if (g.M <= 4) return run<1, true>(g, stream);
    if (g.M <= 8) return run<1, false>(g, stream);
    return run<3, false>(g, stream);
}

}  // namespace nf4k
