// Int8 QLoRA linear forward for up to 64 tokens (gfx950):
//   Y[m, n] = xs[m] ws[n] sum_k Xq[m, k] Wq[n, k] + s (T L2)[m, n],   T = X L1
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net), section 3.1
// eq. (1) (8-bit integers), section 3.5 eq. (5), section 4 eq. (3).
//
// The shape streams the weight's N K bytes once from HBM; everything else has to stay out of the way
// of those loads.  Two launches:
//   1. X's rows to codes, and T's float32 split partials (independent of each other);
//   2. the product.  A workgroup of 4 or 8 waves owns 16 RG weight rows and its waves take turns along
//      K (256-byte chunks, wave w takes chunks w, w + waves, ..), so that a few thousand rows already
//      keep every CU loading; a chunk is loaded while the one before it is multiplied
//      (v_mfma_i32_16x16x64_i8; the 16 rows of its other operand hold 16 tokens, G groups of them).  A
//      weight fragment's bytes go from the load straight into the MFMA: no LDS, no decode.
//      The waves' int32 sums meet in LDS, exact in any order; then the constants, the
//      adapter's MFMAs (s T from T's partials, summed in a fixed order and held in two bf16 halves) and
//      one rounding to bf16.
// Measured (both launches): 47 us for one token x 28672 x 8192 with r = 64 (5.0 TB/s of weight bytes; a
// large copy reaches 5.2 here), 12 us at 4096 x 4096; 20 us for 23 tokens x 4096 x 11008 (16.5 where the
// weight stays in the 256 MB cache).  Bound by HBM at large weights, by the two launches at small ones.
// Small workgroups with few registers win, many waves hiding the loads' latency: one token at 28672 x
// 8192 took 45 us (r = 0) with 4 waves and 16 rows each, 57 with 32 rows, 55 with 8 waves and 64 rows.

#include "common.h"
#include "dqtile.h"
#include "int8.h"
#include "launch.h"
#include "skinny.h"

namespace nf4k {

namespace {

constexpr int CHUNK = 256;         // bytes of K per wave and turn
constexpr int CS = CHUNK / 64;     // MFMA steps of a chunk
constexpr int R_MAX = 128;

// DIRECT (up to 4 tokens): the tokens are loaded in the operands' own layout, too few lines to matter.
template <int NW, int RG, int G, bool DIRECT>
__global__ __launch_bounds__(NW * 64) void int8_gemv_kernel(Int8Gemv g) {
    constexpr int NT = NW * 64;
    // A wave's tokens of a chunk, and after the last its int32 sums [tile][4][lane]; with the tokens in
    // registers, the sums of all waves.
    constexpr int XW = G * 4096, SUMS = RG * G * 256;
    static_assert(SUMS * 4 <= XW, "a wave's sums fit where its tokens were");
    __shared__ __align__(16) uint8_t xtile[DIRECT ? SUMS * 4 : NW * XW];
    // s T as two bf16 halves, [2][M][r], and, where parts > 1 (below: 4 M r bytes of halves are then less
    // than 16 NT), sums over parts of T's partials
    constexpr int ST_MAX = 2 * 16 * G * R_MAX * 2, TPART = NT * 16;
    __shared__ __align__(16) uint8_t st[ST_MAX > 2 * TPART ? ST_MAX : 2 * TPART];
    uint16_t *sTs = reinterpret_cast<uint16_t *>(st);
    f32x4 *tpart = reinterpret_cast<f32x4 *>(st + TPART);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ln = lane & 15, lg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RG);
    const uint32_t K = (uint32_t)g.K;
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(g.Wq + n0 * g.K, (g.N - n0) * g.K);
    const __amdgpu_buffer_rsrc_t rX = make_rsrc(g.Xq, g.M * g.K);
    const int nchunk = (int)((g.K + CHUNK - 1) / CHUNK);

    // Weight rows: lane (ln, lg) of step s loads bytes 64 s + 16 lg .. +15 of row ln, which is its
    // operand.  Rows past N, tokens past M and bytes past K read zeros.
    struct WStage {
        u32x4 w[CS][RG];
    };
    const uint32_t lane_off = (uint32_t)ln * K + lg * 16;
    auto load_w = [&](int c, WStage &st) {
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            const uint32_t k = (uint32_t)c * CHUNK + s * 64;
            const bool live = k < K;
#pragma unroll
            for (int q = 0; q < RG; ++q) st.w[s][q] = bload16(rW, live ? lane_off + k + q * 16 * K : 0xFFFFFFF0u);
        }
    };
    // Tokens: 16 lanes load a row's 256 bytes (four rows per load), and the wave turns them into
    // operands through its own LDS tile, 16-byte pieces XOR-ed with the row so that neither side has
    // bank conflicts.  Loaded in the operands' own layout (16 rows by 64 bytes), the rows' separate
    // lines bound the kernel: 79.8 us for 16 tokens x 28672 x 8192, against 44.9 us for one.
    static_assert(CS == 4, "a chunk's pieces: 4 loads of 4 rows, or 4 steps");
    u32x4 xr[G][4];
    auto load_x = [&](int c) {
        if (DIRECT) {
#pragma unroll
            for (int s = 0; s < CS; ++s) {
                const uint32_t k = (uint32_t)c * CHUNK + s * 64;
                xr[0][s] = bload16(rX, k < K ? lane_off + k : 0xFFFFFFF0u);
            }
            return;
        }
        const int r4 = lane >> 4;
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 4 * i + r4;
                const uint32_t k = (uint32_t)c * CHUNK + ((ln ^ row) * 16);
                xr[q][i] = bload16(rX, k < K ? (uint32_t)(16 * q + row) * K + k : 0xFFFFFFF0u);
            }
    };
    uint8_t *xt = xtile + (DIRECT ? 0 : wave * XW);
    i32x4 acc[RG][G];
#pragma unroll
    for (int a = 0; a < RG; ++a)
#pragma unroll
        for (int b = 0; b < G; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
    // The tile is the wave's own: its LDS operations complete in order, so no barrier is needed, only
    // that the compiler keeps the order of one lane's writes and another's reads.
    auto wave_order = [&]() {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    };
    u32x4 xd[DIRECT ? CS : 1];
    auto put_x = [&]() {
        if (DIRECT) {
#pragma unroll
            for (int s = 0; s < CS; ++s) xd[DIRECT ? s : 0] = xr[0][s];
            return;
        }
        wave_order();
#pragma unroll
        for (int q = 0; q < G; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4 *>(xt + q * 4096 + i * 1024 + lane * 16) = xr[q][i];
        wave_order();
    };
    auto mul = [&](const WStage &st) {
#pragma unroll
        for (int s = 0; s < CS; ++s) {
            i32x4 x[G];
#pragma unroll
            for (int b = 0; b < G; ++b)
                x[b] = DIRECT ? __builtin_bit_cast(i32x4, xd[DIRECT ? s : 0])
                              : *reinterpret_cast<const i32x4 *>(xt + b * 4096 + ln * 256 + (((4 * s + lg) ^ ln) * 16));
#pragma unroll
            for (int a = 0; a < RG; ++a)
#pragma unroll
                for (int b = 0; b < G; ++b)
                    acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[b], __builtin_bit_cast(i32x4, st.w[s][a]), acc[a][b], 0, 0, 0);
        }
    };

    WStage s0, s1;
    load_w(wave, s0);
    load_x(wave);
    // Prologue, while the first chunk streams in: the sums' zeros, and s T (and T, by workgroup 0).
    // Where T has fewer pieces than the workgroup threads, `parts` threads share a piece's partials, so
    // that their loads are one latency, not one after the other; the parts are added in order below.
    int32_t *sums = reinterpret_cast<int32_t *>(xt);
    if (DIRECT)
        for (int i = tid; i < SUMS; i += NT) sums[i] = 0;
    const int E4 = (int)((g.M * g.r) >> 2);
    const int parts = E4 > 0 && E4 < NT ? min(NT / E4, 16) : 1;
    auto put_T = [&](int i, f32x4 t) {
        const float f[4] = {g.scale * t.x, g.scale * t.y, g.scale * t.z, g.scale * t.w};
        split_bf16x4(f, reinterpret_cast<uint2 *>(sTs)[i], reinterpret_cast<uint2 *>(sTs)[E4 + i]);
        if (blockIdx.x == 0 && g.T_out)
            reinterpret_cast<uint2 *>(g.T_out)[i] = uint2{pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w)};
    };
    if (g.r && !g.Tp) {
        for (int i = tid; i < E4; i += NT) {
            reinterpret_cast<uint2 *>(sTs)[i] = reinterpret_cast<const uint2 *>(g.sT)[i];
            reinterpret_cast<uint2 *>(sTs)[E4 + i] = reinterpret_cast<const uint2 *>(g.sTlo)[i];
        }
    } else if (g.r) {
        const f32x4 *Tp = reinterpret_cast<const f32x4 *>(g.Tp);
        for (int j = tid; j < E4 * parts; j += NT) {
            const int i = j % E4;
            f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
            for (int k0 = j / E4; k0 < g.ksT; k0 += 8 * parts) {
                f32x4 v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (k0 + u * parts < g.ksT) v[u] = Tp[(int64_t)(k0 + u * parts) * E4 + i];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (k0 + u * parts < g.ksT) t += v[u];
            }
            if (parts == 1) put_T(i, t);
            else tpart[j] = t;
        }
    }

    // One chunk ahead (two cost the registers of more waves: 45.5 -> 48.8 us for one token at
    // 28672 x 8192).  Chunks past the end load nothing and add zeros.
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

    auto put_sum = [&](auto put) {
#pragma unroll
        for (int a = 0; a < RG; ++a)
#pragma unroll
            for (int b = 0; b < G; ++b)
#pragma unroll
                for (int v = 0; v < 4; ++v) put(&sums[(a * G + b) * 256 + v * 64 + lane], acc[a][b][v]);
    };
    if (!DIRECT) {
        wave_order();
        put_sum([](int32_t *s, int32_t x) { *s = x; });
    }
    __syncthreads();
    if (parts > 1 && tid < E4 && g.Tp) {
        f32x4 t = tpart[tid];
        for (int p = 1; p < parts; ++p) t += tpart[p * E4 + tid];
        put_T(tid, t);
    }
    if (DIRECT && nchunk > wave) put_sum([](int32_t *s, int32_t x) { atomicAdd(s, x); });
    __syncthreads();

    // wave w finishes tiles w, w + NW, ..: lane (ln, lg) holds weight row n and tokens 16 b + 4 lg + v
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
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const u32x4 av = (m < g.M && jj < g.r) ? *reinterpret_cast<const u32x4 *>(sTs + (h * g.M + m) * g.r + jj) : u32x4{0u, 0u, 0u, 0u};
                lora = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, av),
                                                               __builtin_bit_cast(bf16x8, u32x4{bw[0], bw[1], bw[2], bw[3]}), lora, 0, 0, 0);
            }
        }
        if (n >= g.N) continue;
        const float w = g.ws[n];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t m = 16 * b + 4 * lg + v;
            if (m < g.M) {
                int32_t sum = 0;
#pragma unroll
                for (int u = 0; u < (DIRECT ? 1 : NW); ++u)
                    sum += reinterpret_cast<const int32_t *>(xtile + u * XW)[t * 256 + v * 64 + lane];
                const float y = ((float)sum * g.xs[m]) * w + lora[v];
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

template <int NW, int RG, int G, bool DIRECT = false>
void launch_one(const Int8Gemv &a, hipStream_t s) {
    hipLaunchKernelGGL((int8_gemv_kernel<NW, RG, G, DIRECT>), dim3((unsigned)((a.N + 16 * RG - 1) / (16 * RG))), dim3(NW * 64), 0, s, a);
}
// More than 16 tokens: 32 weight rows share the tokens' loads where that leaves a workgroup for every
// CU (32 x 8192 x 22016: 56.5 against 64.1 us with 16 rows; 64 x 8192 x 8192 27.0 against 33.3).
template <int G>
void launch_g(const Int8Gemv &a, hipStream_t s) {
    const int64_t groups = (a.N + 15) / 16;
    if (groups >= 4 * 256) launch_one<4, 2, G>(a, s);
    else if (groups >= 2 * 256) launch_one<8, 2, G>(a, s);
    else launch_one<8, 1, G>(a, s);
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
    if (p.M < 1 || p.M > 64 || p.r < 0 || p.r > R_MAX || (p.r && !p.Tp == !p.sT) || !p.sT != !p.sTlo) return hipErrorInvalidValue;
    // Four waves where the rows make at least two workgroups a CU, else eight (8192 x 22016, one token:
    // 45.5 against 47.5 us; 4096 x 4096: 8.4 us with eight, 10.0 with sixteen).
    const int64_t groups = (p.N + 15) / 16;
    timing_before(stream, 2);
    if (p.M > 32) launch_g<4>(p, stream);
    else if (p.M > 16) launch_g<2>(p, stream);
    else if (p.M > 4 && groups >= 512) launch_one<4, 1, 1>(p, stream);
    else if (p.M > 4) launch_one<8, 1, 1>(p, stream);
    else if (groups >= 512) launch_one<4, 1, 1, true>(p, stream);
    else launch_one<8, 1, 1, true>(p, stream);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace nf4k
