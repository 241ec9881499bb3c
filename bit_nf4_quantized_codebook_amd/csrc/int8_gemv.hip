// Int8 QLoRA linear forward for up to 64 tokens (gfx950):
//   Y[m, n] = xs[m] ws[n] sum_k Xq[m, k] Wq[n, k] + s (T L2)[m, n],   T = X L1
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net), section 3.1
// eq. (1) (8-bit integers), section 3.5 eq. (5), section 4 eq. (3).
//
// The shape streams the weight's N K bytes once from HBM; everything else has to stay out of the way
// of those loads.  Two launches:
//   1. X's rows to codes, and T's float32 split partials (independent of each other);
//   2. the product.  A workgroup of 8 waves owns 16 RG weight rows and its waves take turns along K
//      (256-byte chunks, wave w takes chunks w, w + 8, ..), so that a few thousand rows already keep
//      every CU loading; a chunk is loaded while the one before it is multiplied
//      (v_mfma_i32_16x16x64_i8; the 16 columns of the MFMA hold 16 tokens, G groups of them).  A
//      weight fragment's bytes go from the load straight into the MFMA: no LDS, no decode.  The
//      codes of X (at most 64 K bytes) come from L2 with the same addressing.
//      The waves' int32 sums meet in LDS by integer adds, exact in any order; then the constants, the
//      adapter's MFMAs (s T from T's partials, summed in the prologue in a fixed order) and one
//      rounding to bf16.

#include "common.h"
#include "dqtile.h"
#include "int8.h"
#include "launch.h"
#include "skinny.h"

namespace nf4k {

namespace {

constexpr int NW = 8;              // waves
constexpr int NT = NW * 64;
constexpr int CHUNK = 256;         // bytes of K per wave and turn
constexpr int CS = CHUNK / 64;     // MFMA steps of a chunk
constexpr int R_MAX = 128;

template <int RG, int G>
__global__ __launch_bounds__(NT) void int8_gemv_kernel(Int8Gemv g) {
    __shared__ int32_t sums[RG * G * 256];                 // [tile][lane][4]
    __shared__ __align__(16) uint16_t sTs[16 * G * R_MAX];  // s T, bf16 [M][r]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ln = lane & 15, lg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RG);
    const uint32_t K = (uint32_t)g.K;
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(g.Wq + n0 * g.K, (g.N - n0) * g.K);
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(g.Xq, g.M * g.K);
    const int nchunk = (int)((g.K + CHUNK - 1) / CHUNK);

    struct Stage {
        u32x4 w[CS][RG], x[CS][G];
    };
    // rows past N, tokens past M and steps past K read zeros
    const uint32_t lane_off = (uint32_t)ln * K + lg * 16;
    auto load = [&](int c, Stage &st) {
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            const uint32_t k = (uint32_t)c * CHUNK + s * 64;
            const bool live = k < K;
#pragma unroll
            for (int q = 0; q < RG; ++q) st.w[s][q] = bload16(rW, live ? lane_off + k + q * 16 * K : 0xFFFFFFF0u);
#pragma unroll
            for (int q = 0; q < G; ++q) st.x[s][q] = bload16(rX, live ? lane_off + k + q * 16 * K : 0xFFFFFFF0u);
        }
    };
    i32x4 acc[RG][G];
#pragma unroll
    for (int a = 0; a < RG; ++a)
#pragma unroll
        for (int b = 0; b < G; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    auto mul = [&](const Stage &st) {
#pragma unroll
        for (int s = 0; s < CS; ++s)
#pragma unroll
            for (int a = 0; a < RG; ++a)
#pragma unroll
                for (int b = 0; b < G; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, st.x[s][b]),
                                                                      __builtin_bit_cast(i32x4, st.w[s][a]), acc[a][b], 0, 0, 0);
    };

    Stage s0, s1;
    load(wave, s0);
    // prologue, while the first chunk streams in: the sums' zeros, s T (and T, by workgroup 0)
    for (int i = tid; i < RG * G * 256; i += NT) sums[i] = 0;
    if (g.r && !g.Tp) {
        const uint2 *src = reinterpret_cast<const uint2 *>(g.sT);
        for (int i = tid; i < (int)((g.M * g.r) >> 2); i += NT) reinterpret_cast<uint2 *>(sTs)[i] = src[i];
    } else if (g.r) {
        const int64_t E4 = (g.M * g.r) >> 2;
        const f32x4 *Tp = reinterpret_cast<const f32x4 *>(g.Tp);
        for (int i = tid; i < (int)E4; i += NT) {
            f32x4 t = Tp[i];
            for (int k0 = 1; k0 < g.ksT; k0 += 8) {
                f32x4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (k0 + u < g.ksT) v[u] = Tp[(int64_t)(k0 + u) * E4 + i];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (k0 + u < g.ksT) t += v[u];
            }
            const float s = g.scale;
            *reinterpret_cast<uint2 *>(sTs + 4 * i) = uint2{pack_bf16x2(s * t.x, s * t.y), pack_bf16x2(s * t.z, s * t.w)};
            if (blockIdx.x == 0 && g.T_out)
                reinterpret_cast<uint2 *>(g.T_out)[i] = uint2{pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w)};
        }
    }
    __syncthreads();

    for (int c = wave; c < nchunk; c += 2 * NW) {      // chunks past the end load nothing and add zeros
        load(c + NW, s1);
        mul(s0);
        load(c + 2 * NW, s0);
        mul(s1);
    }

    if (nchunk > wave) {
#pragma unroll
        for (int a = 0; a < RG; ++a)
#pragma unroll
            for (int b = 0; b < G; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v) atomicAdd(&sums[(a * G + b) * 256 + v * 64 + lane], acc[a][b][v]);
    }
    __syncthreads();

    // wave w finishes tiles w, w + 8, ..: lane (ln, lg) holds weight row n and tokens 16 b + 4 lg + v
    const __amdgpu_buffer_rsrc_t rL2 = make_rsrc(g.L2, (int64_t)g.r * g.N * 2);
    for (int t = wave; t < RG * G; t += NW) {
        const int a = t / G, b = t % G;
        const int64_t n = n0 + a * 16 + ln;
        if (16 * b >= g.M) continue;
        f32x4 lora = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int j0 = 0; j0 < g.r; j0 += 32) {
            const int jj = j0 + lg * 8;
            uint32_t bw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool ok = jj < g.r && n < g.N;       // r % 8 == 0: a group of 8 is inside or outside
                const uint32_t o = (uint32_t)(((jj + 2 * i) * g.N + n) * 2);
                const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b16(rL2, ok ? o : 0xFFFFFFF0u, 0, 0);
                const uint32_t hi = __builtin_amdgcn_raw_buffer_load_b16(rL2, ok ? o + (uint32_t)(g.N * 2) : 0xFFFFFFF0u, 0, 0);
                bw[i] = (lo & 0xFFFFu) | (hi << 16);
            }
            const int64_t m = 16 * b + ln;
            const u32x4 av = (m < g.M && jj < g.r) ? *reinterpret_cast<const u32x4 *>(sTs + m * g.r + jj) : u32x4{0u, 0u, 0u, 0u};
            lora = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av),
                                                           __builtin_bit_cast(bf16x8, u32x4{bw[0], bw[1], bw[2], bw[3]}), lora, 0, 0, 0);
        }
        if (n >= g.N) continue;
        const float w = g.ws[n];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t m = 16 * b + 4 * lg + v;
            if (m < g.M) {
                const float y = ((float)sums[t * 256 + v * 64 + lane] * g.xs[m]) * w + lora[v];
                g.Y[m * g.N + n] = (uint16_t)f32_to_bf16(y);
            }
        }
    }
}

// Launch 1: T's partials (skinny workgroups first, they take longer) and X's rows to codes.
struct RowsT {
    const uint16_t *X, *L1;
    float *P;
    int64_t M, K, kchunk;
    int32_t r;
    uint32_t nt, nty;          // T's workgroups, and how many of them lie along r
    int8_t *Xq;
    float *xs;
};
__global__ __launch_bounds__(256) void int8_rows_t_kernel(RowsT g) {
    if (blockIdx.x < g.nt) {
        skinny_nt_block<true>(g.X, g.L1, g.P, g.M, g.r, g.K, g.kchunk, 0, blockIdx.x % g.nty, blockIdx.x / g.nty);
        return;
    }
    int8_rows_block<false>(g.X, blockIdx.x - g.nt, g.M, g.K, g.Xq, g.xs);
}

template <int RG>
void launch_rg(const Int8Gemv &a, hipStream_t s) {
    const dim3 gd((unsigned)((a.N + 16 * RG - 1) / (16 * RG)));
    if (a.M <= 16) hipLaunchKernelGGL((int8_gemv_kernel<RG, 1>), gd, dim3(NT), 0, s, a);
    else if (a.M <= 32) hipLaunchKernelGGL((int8_gemv_kernel<RG, 2>), gd, dim3(NT), 0, s, a);
    else hipLaunchKernelGGL((int8_gemv_kernel<RG, 4>), gd, dim3(NT), 0, s, a);
}

}  // namespace

hipError_t launch_int8_rows_t(const uint16_t *X, const uint16_t *L1, float *P, int64_t M, int32_t r, int64_t K, int nsplit,
                              int8_t *Xq, float *xs, hipStream_t stream) {
    if (M < 1 || M > 64) return hipErrorInvalidValue;
    RowsT a{};
    a.X = X; a.L1 = L1; a.P = P; a.M = M; a.K = K; a.r = r; a.Xq = Xq; a.xs = xs;
    if (r) {
        if (nsplit < 1) return hipErrorInvalidValue;
        const int64_t steps = (K + ST - 1) / ST;
        a.kchunk = (steps + nsplit - 1) / nsplit * ST;
        a.nty = (uint32_t)((r + ST - 1) / ST);
        a.nt = a.nty * (uint32_t)nsplit;
    }
    const uint32_t rows = Xq ? (uint32_t)int8_rows_blocks(M, K) : 0u;
    if (a.nt + rows == 0) return hipSuccess;
    hipLaunchKernelGGL(int8_rows_t_kernel, dim3(a.nt + rows), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_int8_gemv(const Int8Gemv &p, hipStream_t stream) {
    if (p.M < 1 || p.M > 64 || p.r < 0 || p.r > R_MAX || (p.r && !p.Tp == !p.sT)) return hipErrorInvalidValue;
    // as many rows per workgroup (they share X's loads) as still leave one for every CU
    const int64_t groups = (p.N + 15) / 16;
    timing_before(stream, 2);
    if (groups >= 4 * 256) launch_rg<4>(p, stream);
    else if (groups >= 2 * 256) launch_rg<2>(p, stream);
    else launch_rg<1>(p, stream);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace nf4k
