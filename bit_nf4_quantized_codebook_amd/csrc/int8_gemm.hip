// Int8 product of the Int8 QLoRA linear forward from 65 tokens (gfx950):
//   Y[m, n] = xs[m] ws[n] sum_k Xq[m, k] Wq[n, k] + ((sT + sTlo) L2)[m, n]
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net), section 3.1
// eq. (1) (8-bit integers), section 3.5 eq. (5), section 4 eq. (3).
//
// The integer sums are exact in any order (K * 2^14 < 2^31), so only the epilogue rounds: the sum to
// float32, times the two constants, plus the adapter's product, once to bf16.
//
// Block tile 256 x 256 outputs, reduction step 128 (128-byte LDS rows), 4 waves in 2 x 2, each
// 128 x 128 with v_mfma_i32_32x32x32_i8 (16 tiles, 256 int32 accumulators): a 32 x 32 x 32 int8 MFMA
// takes the operand bytes and the cycles of a 32 x 32 x 16 bf16 one, so the loop moves the same bytes
// per cycle as the bf16 GEMM's and does twice its products.  Both operands go straight from global
// memory to LDS (buffer_load ... lds), two 32 KB stages each, 16-byte chunks XOR-swizzled by
// (row / 2) so that the fragment reads are free of bank conflicts.  After the last step the
// accumulators are turned to float32 four tiles at a time and the adapter's r/64 steps run on them with
// v_mfma_f32_32x32x16_bf16, whose output layout is the same.  (All 16 tiles turned first and then
// multiplied, the kernel spilled 70 registers.)  s T comes as two bf16 halves, each with its own MFMAs: one
// half alone would lose as much of the adapter's term as Y's own rounding.  (Tile by tile, with the
// fragments read again for each, the second halves cost 3.3 us at 4096 x 4096 x 4096, r = 64; as it is,
// 0.5.)
//
// Bound by the MFMA loop at the clock its power allows: 63 us at 4096 x 4096 x 4096 with r = 64 (2.2
// POPS; a library int8 product of 8192 x 8192 x 8192 reaches 2.33 here) and 331 us at 2048 tokens x 22016 x
// 8192 (2.2 POPS).  The whole forward call (codes of X, T, this product) takes 82 and 345 us; a 64 x 64
// tile with one LDS stage took 420 and 1667 us.
//
// Few output tiles (at most half the CUs): the reduction is split over up to 16 workgroups per
// tile, each writing its int32 sums; a second launch adds them, still exact, and has the epilogue.  So
// without an adapter a token's Y is the same bits whatever the batch it comes in.  The price is the
// partials' way through memory and, below 256 tokens, a tile that is mostly padding: with r = 64 and a weight of
// 4096 x 4096, 65 tokens take 29 us, 300 34, 1024 51 and 2048 71 (floors 4, 5, 15 and 31).

#include "common.h"
#include "dqtile.h"
#include "int8.h"
#include "launch.h"

namespace nf4k {

namespace {

constexpr int TM = 256, TN = 256;
constexpr int TKB = 128;                    // bytes of a reduction step: 128 codes, or 64 bf16 of the adapter
constexpr int STAGE = TM * TKB;             // 32 KB per operand stage

__global__ __launch_bounds__(256, 1) void int8_gemm_kernel(Int8Product g) {
    // one LDS object per stage: a fragment read of one stage provably never aliases the
    // direct-to-LDS loads in flight into the other
    __shared__ __align__(16) uint8_t As0[STAGE];
    __shared__ __align__(16) uint8_t As1[STAGE];
    __shared__ __align__(16) uint8_t Bs0[STAGE];
    __shared__ __align__(16) uint8_t Bs1[STAGE];
    __shared__ __align__(16) float xs_l[TM];
    __shared__ float ws_l[TN];
    typedef __attribute__((address_space(3))) uint8_t lds_u8;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int r32 = lane & 31, hh = lane >> 5;

    const int ntm = (int)((g.M + TM - 1) / TM);
    const int ntn = (int)((g.N + TN - 1) / TN);
    const int ntiles = ntm * ntn;
    const int split = (int)(blockIdx.x / (uint32_t)ntiles);
    int tm, tn;
    tile_coords_grouped<4>(ntm, ntn, (int)blockIdx.x - split * ntiles, tm, tn);
    const int64_t m0 = (int64_t)tm * TM;
    const int64_t n0 = (int64_t)tn * TN;
    // this workgroup's reduction steps: kb .. kb + steps - 1
    const int all_steps = (int)((g.K + TKB - 1) / TKB);
    const int kb = split * g.split_per;
    const int steps = min(all_steps - kb, g.split_per);
    const bool part = g.ksplit > 1;
    const int ext_steps = part ? 0 : (g.r + 63) / 64;

    // tile-relative descriptors: rows past M (or N) read zeros
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.Xq + m0 * g.K, (g.M - m0) * g.K);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.Wq + n0 * g.K, (g.N - n0) * g.K);

    // Loads: instruction q of wave w writes stage rows 8u .. 8u+7 (u = 8w + q); lane l takes row
    // 8u + l/8 and physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8); (row/2)%8 =
    // (4q + l/16)%8, so the lane's chunk depends only on the parity of q.
    int a_col[2];
    uint32_t voff[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = 8 * (8 * wave + q) + (lane >> 3);
        a_col[q] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
        voff[q] = (uint32_t)((lane >> 3) * g.K + a_col[q]);
    }
    const uint32_t wave_off = (uint32_t)(64 * wave * g.K);
    const uint32_t row8_off = (uint32_t)(8 * g.K);
    // Codes at or past the end of the split (the ragged last step, the steps past the end) read
    // zeros; the whole offset sits in the lane offset, so rows past the operand's end are out of
    // range for the descriptor's bound check.
    const int kend = (int)min(g.K, (int64_t)(kb + steps) * TKB);
    auto load = [&](__amdgpu_buffer_rsrc_t r, int step, uint8_t *st, int q0 = 0, int q1 = 8) {
        lds_u8 *dst = (lds_u8 *)st + wave * 8192;
        const int k0 = (kb + step) * TKB, rem = kend - k0;
        const uint32_t base = wave_off + (uint32_t)k0;
        const uint32_t v0 = a_col[0] < rem ? voff[0] + base : 0x80000000u;
        const uint32_t v1 = a_col[1] < rem ? voff[1] + base : 0x80000000u;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q < q0 || q >= q1) continue;
            const uint32_t v = ((q & 1) ? v1 : v0) + (uint32_t)q * row8_off;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(dst + q * 1024), 16, v, 0, 0, 0);
        }
    };

    i32x16 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;

    // fragment of sub-step s (32 bytes of the row): lane (r32, hh) takes its 16-byte chunk 2 s + hh
    uint32_t lds_off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) lds_off[s] = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
    struct Frags {
        i32x4 a[4], b[4];
    };
    auto read = [&](const uint8_t *Ast, const uint8_t *Bst, int s, Frags &f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f.a[i] = *reinterpret_cast<const i32x4 *>(Ast + lds_off[s] + (wm * 128 + 32 * i) * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f.b[j] = *reinterpret_cast<const i32x4 *>(Bst + lds_off[s] + (wn * 128 + 32 * j) * 128);
    };
    auto mma = [&](const Frags &f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
    };
    // The schedule is the bf16 GEMM's: fragment reads one sub-step ahead of the MFMAs, each of the
    // first 8 MFMAs of a sub-step followed by one read, and in a sub-step that carries loads every
    // second MFMA by one direct-to-LDS load.
    auto interleave = [&](int nvmem) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                             // 1 MFMA
            if (k < 8) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                  // 1 DS read
            if ((k & 1) && (k >> 1) < nvmem) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // 1 VMEM
        }
    };
    // One step computes stage (Ac, Bc) while step + 1 lands in (An, Bn).  The workgroup barrier sits
    // between sub-steps 2 and 3: by then every wave has its sub-step 3 fragments in registers, so
    // after it stage c is free for the loads of step + 2, and stage n is complete.
    Frags f0, f1;
    auto step_body = [&](int step, uint8_t *Ac, uint8_t *Bc, uint8_t *An, uint8_t *Bn) {
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            Frags &cur = (s & 1) ? f1 : f0;
            Frags &nxt = (s & 1) ? f0 : f1;
            if (s == 0) {
                load(rA, step + 1, An, 4, 8);
                load(rB, step + 1, Bn, 4, 8);
            }
            read(Ac, Bc, s + 1, nxt);
            mma(cur);
            interleave(s == 0 ? 8 : 0);
            __builtin_amdgcn_sched_barrier(0);
        }
        // step + 1 landed (this wave's loads) and this wave's fragment reads of stage c are done
        __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (0 << 8));
        __syncthreads();
        read(An, Bn, 0, f0);
        load(rA, step + 2, Ac, 0, 4);
        load(rB, step + 2, Bc, 0, 4);
        mma(f1);
        interleave(8);
        __builtin_amdgcn_sched_barrier(0);
    };

    load(rA, 0, As0);
    load(rB, 0, Bs0);
    load(rA, 1, As1, 0, 4);
    load(rB, 1, Bs1, 0, 4);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    read(As0, Bs0, 0, f0);
    int step = 0;
    for (; step + 1 < steps; step += 2) {
        step_body(step, As0, Bs0, As1, Bs1);
        step_body(step + 1, As1, Bs1, As0, Bs0);
    }
    if (step < steps) step_body(step, As0, Bs0, As1, Bs1);   // odd count: the last one
    __builtin_amdgcn_s_waitcnt(0);
    if (!part) __syncthreads();

    // lane indices for the code after the main loop, recomputed (mbcnt) rather than kept live
    // across it
    const int lane_e = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    const int r32_e = lane_e & 31, hh_e = lane_e >> 5;
    const int tid_e = wave * 64 + lane_e;

    // lane (r32, hh) of tile (i, j) holds column wn*128 + 32 j + r32 and rows wm*128 + 32 i + 8 (v/4) + 4 hh +
    // v%4; rows past M fall outside the descriptors
    const uint32_t row_bytes = (uint32_t)(g.N * (part ? 4 : 2));
    const uint32_t lane_off = (uint32_t)((wm * 128 + hh_e * 4) * row_bytes) + (uint32_t)((n0 + wn * 128 + r32_e) * (part ? 4 : 2));
    if (part) {
        const __amdgpu_buffer_rsrc_t rP = make_rsrc(g.P + (int64_t)split * g.M * g.N + m0 * g.N, (g.M - m0) * g.N * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n0 + wn * 128 + j * 32 + r32_e >= g.N) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    __builtin_amdgcn_raw_buffer_store_b32((uint32_t)acc[i][j][v], rP, lane_off + j * 128,
                                                          (uint32_t)(i * 32 + (v >> 2) * 8 + (v & 3)) * row_bytes, 0);
        }
        return;
    }

    // ---- epilogue operands into LDS: the tile's constants, and the adapter's steps (r <= 128: at most
    // two), zero padded past r: sT's rows in stage As0, sTlo's in As1, L2^T's rows of step e in Bs0 or Bs1.
    // With two steps an A stage holds both steps of half the tile's rows (64 of each wave row's 128), and
    // is loaded again for the other half ----
    const bool two = ext_steps > 1;
    const __amdgpu_buffer_rsrc_t rAe = make_rsrc(g.sT + m0 * g.r, ext_steps ? (g.M - m0) * (int64_t)g.r * 2 : 0);
    const __amdgpu_buffer_rsrc_t rAl = make_rsrc(g.sTlo + m0 * g.r, ext_steps ? (g.M - m0) * (int64_t)g.r * 2 : 0);
    // a_col of the main loop, in elements
    auto ext_col = [&](int q) { return ((lane_e & 7) ^ ((4 * q + (lane_e >> 4)) & 7)) * 8; };
    auto load_ext_A = [&](int half) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int r8 = 8 * q + (lane_e >> 3);
            const int row = two ? (wave & 1) * 128 + 64 * half + r8 : 64 * wave + r8;
            const int jj = (two ? (wave >> 1) * 64 : 0) + ext_col(q);
            const uint32_t off = jj < g.r ? (uint32_t)((row * (int64_t)g.r + jj) * 2) : 0x80000000u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rAe, (lds_void *)((lds_u8 *)As0 + wave * 8192 + q * 1024), 16, off, 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rAl, (lds_void *)((lds_u8 *)As1 + wave * 8192 + q * 1024), 16, off, 0, 0, 0);
        }
    };
    if (tid_e < TM) {
        xs_l[tid_e] = m0 + tid_e < g.M ? g.xs[m0 + tid_e] : 0.0f;
        ws_l[tid_e] = n0 + tid_e < g.N ? g.ws[n0 + tid_e] : 0.0f;
    }
    if (ext_steps > 0) {
        const __amdgpu_buffer_rsrc_t rBe = make_rsrc(g.L2T + n0 * g.r, (g.N - n0) * (int64_t)g.r * 2);
        auto load_ext_B = [&](int e, uint8_t *Bst) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int row = 8 * (8 * wave + q) + (lane_e >> 3);
                const int jj = e * 64 + ext_col(q);
                const uint32_t off = jj < g.r ? (uint32_t)((row * (int64_t)g.r + jj) * 2) : 0x80000000u;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rBe, (lds_void *)((lds_u8 *)Bst + wave * 8192 + q * 1024), 16, off, 0, 0, 0);
            }
        };
        load_ext_A(0);
        load_ext_B(0, Bs0);
        if (two) load_ext_B(1, Bs1);
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();

    // ---- four 32 x 32 tiles side by side at a time: the sums to float32 times both constants, the
    // adapter's MFMAs on them, the stores ----
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(g.Y + m0 * g.N, (g.M - m0) * g.N * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i == 2 && two) {
            __syncthreads();
            load_ext_A(1);
            __builtin_amdgcn_s_waitcnt(0);
            __syncthreads();
        }
        f32x4 x[4];
#pragma unroll
        for (int v4 = 0; v4 < 4; ++v4)
            x[v4] = *reinterpret_cast<const f32x4 *>(xs_l + wm * 128 + i * 32 + v4 * 8 + hh_e * 4);
        f32x16 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float w = ws_l[wn * 128 + j * 32 + r32_e];
#pragma unroll
            for (int v = 0; v < 16; ++v) f[j][v] = ((float)acc[i][j][v] * x[v >> 2][v & 3]) * w;
        }
#pragma unroll 1
        for (int e = 0; e < ext_steps; ++e) {
            const int row = two ? 128 * e + wm * 64 + 32 * (i & 1) : wm * 128 + 32 * i;
            const uint8_t *Bst = (e ? Bs1 : Bs0) + wn * 128 * 128;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint32_t o = (uint32_t)(r32_e * 128 + (((2 * s + hh_e) ^ ((r32_e >> 1) & 7)) * 16));
                const bf16x8 fa = *reinterpret_cast<const bf16x8 *>(As0 + o + row * 128);
                const bf16x8 fl = *reinterpret_cast<const bf16x8 *>(As1 + o + row * 128);
                bf16x8 fb[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) fb[j] = *reinterpret_cast<const bf16x8 *>(Bst + o + 32 * j * 128);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb[j], f[j], 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fl, fb[j], f[j], 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n0 + wn * 128 + j * 32 + r32_e >= g.N) continue;
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
                const uint32_t rows = (uint32_t)(i * 32 + (v >> 2) * 8 + (v & 3));
                const uint32_t pk = pack_bf16x2(f[j][v], f[j][v + 1]);
                const uint32_t soff = rows * row_bytes;
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pk, rC, lane_off + j * 64, soff, 0);
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(pk >> 16), rC, lane_off + j * 64, soff + row_bytes, 0);
            }
        }
    }
}

// The splits' sums and the epilogue of a split product.  A wave takes G groups of 16 tokens by 16 weight
// rows: lane (ln, lg) holds token ln and rows 4 lg .. +3, 16 bytes of each partial, which is the output
// layout of v_mfma_f32_16x16x32_bf16 with L2^T's rows as the first operand and s T's as the second, so
// the adapter's RS steps of 32 go straight onto the scaled sums, for each of s T's two halves.  A
// workgroup's four waves lie along the weight rows (256 contiguous bytes per token) and share s T's rows
// through LDS: read by each wave for itself, their 16 rows per load made the whole call 82 instead of
// 75 us at 2048 x 4096 x 4096, r = 64.
// Against float32 partials with the adapter's product in the last split's, which are not exact: 65 x
// 4096 x 4096 with r = 64 31 -> 26 us, 2048 x 4096 x 4096 73 -> 75 us (63 both without an adapter).
template <int G, int RS>
__global__ __launch_bounds__(256) void int8_sum_kernel(Int8Product g) {
    const int lane = threadIdx.x & 63, ln = lane & 15, lg = lane >> 4;
    const int64_t nb = (g.N + 63) / 64;
    const int64_t m0 = (int64_t)(blockIdx.x / (uint32_t)nb) * (16 * G) + ln;
    const int64_t n0 = (int64_t)(blockIdx.x % (uint32_t)nb) * 64 + (threadIdx.x >> 6) * 16, n = n0 + 4 * lg;
    const bool nin = n < g.N;                     // N % 8 == 0: the four rows are inside or outside
    const u32x4 none = {0u, 0u, 0u, 0u};
    u32x4 a[RS ? RS : 1];
#pragma unroll
    for (int s = 0; s < RS; ++s) {
        const int j = 32 * s + 8 * lg;            // r % 8 == 0: a group of 8 is inside or outside
        a[s] = j < g.r && n0 + ln < g.N ? *reinterpret_cast<const u32x4 *>(g.L2T + (n0 + ln) * g.r + j) : none;
    }
    float w[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) w[v] = nin ? g.ws[n + v] : 0.0f;
    const int64_t plane = g.M * g.N / 4;
    constexpr int KU = 8 / G;                     // partials' loads in flight per group
    i32x4 sum[G];
    const i32x4 *p[G];
#pragma unroll
    for (int q = 0; q < G; ++q) {
        sum[q] = i32x4{0, 0, 0, 0};
        const int64_t m = m0 + 16 * q;
        p[q] = reinterpret_cast<const i32x4 *>(g.P + (nin && m < g.M ? m * g.N + n : 0));
    }
    // the tokens' s T rows, shared by the four waves: the first halves, then the second
    constexpr int ROW = RS * 64 + 16;             // bytes, padded: 16 rows' pieces lie on 64 different banks
    constexpr int HALF = 16 * G * ROW;
    __shared__ __align__(16) uint8_t st[RS ? 2 * HALF : 16];
    if (RS > 0) {
        const int64_t mt = m0 - ln;
#pragma unroll
        for (int i = 0; i < (G * RS + 3) / 4; ++i) {
            const int c = (int)threadIdx.x + 256 * i, row = c / (RS ? 4 * RS : 1), j = c % (RS ? 4 * RS : 1) * 8;
            const bool live = j < g.r && mt + row < g.M;
            if (row < 16 * G) {
                *reinterpret_cast<u32x4 *>(st + row * ROW + j * 2) =
                    live ? *reinterpret_cast<const u32x4 *>(g.sT + (mt + row) * g.r + j) : none;
                *reinterpret_cast<u32x4 *>(st + HALF + row * ROW + j * 2) =
                    live ? *reinterpret_cast<const u32x4 *>(g.sTlo + (mt + row) * g.r + j) : none;
            }
        }
    }
    for (int k0 = 0; k0 < g.ksplit; k0 += KU) {
        i32x4 v[G][KU];
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
            for (int q = 0; q < G; ++q)
                if (k0 + u < g.ksplit) v[q][u] = p[q][(k0 + u) * plane];
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
            for (int q = 0; q < G; ++q)
                if (k0 + u < g.ksplit) sum[q] += v[q][u];
    }
    if (RS > 0) __syncthreads();
#pragma unroll
    for (int q = 0; q < G; ++q) {
        const int64_t m = m0 + 16 * q;
        const bool in = nin && m < g.M;
        const float x = m < g.M ? g.xs[m] : 0.0f;
        f32x4 f;
#pragma unroll
        for (int v = 0; v < 4; ++v) f[v] = ((float)sum[q][v] * x) * w[v];
#pragma unroll
        for (int s = 0; s < RS; ++s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bf16x8 b = *reinterpret_cast<const bf16x8 *>(st + h * HALF + (16 * q + ln) * ROW + (32 * s + 8 * lg) * 2);
                f = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[s]), b, f, 0, 0, 0);
            }
        }
        if (in) *reinterpret_cast<uint2 *>(g.Y + m * g.N + n) = uint2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
    }
}

// Two groups of tokens a wave where one would make more than sixteen workgroups a CU: with one and with two,
// 2048 x 4096 x 4096 with r = 64 81.1 and 79.4 us, 1000 x 4096 x 4096 59.4 and 59.9, 300 x 4096 x 11008
// 53.8 and 57.
template <int RS>
void launch_sum(const Int8Product &a, hipStream_t s) {
    const int64_t nb = (a.N + 63) / 64, m16 = (a.M + 15) / 16;
    // a split product has at most 128 tiles: at most 8192 workgroups
    if (m16 * nb > 4096) hipLaunchKernelGGL((int8_sum_kernel<2, RS>), dim3((unsigned)((m16 + 1) / 2 * nb)), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((int8_sum_kernel<1, RS>), dim3((unsigned)(m16 * nb)), dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_int8_gemm(const Int8Product &p, hipStream_t stream) {
    const int64_t tiles = ((p.M + TM - 1) / TM) * ((p.N + TN - 1) / TN);
    const int64_t steps = (p.K + TKB - 1) / TKB;
    Int8Product a = p;
    if (a.ksplit <= 1) {
        a.ksplit = 1;
        a.split_per = (int32_t)steps;
    } else if (!a.P || (int64_t)(a.ksplit - 1) * a.split_per >= steps || (int64_t)a.ksplit * a.split_per < steps) {
        return hipErrorInvalidValue;     // every split non-empty, the partials somewhere to go
    }
    timing_before(stream, 0);
    hipLaunchKernelGGL(int8_gemm_kernel, dim3((unsigned)(tiles * a.ksplit)), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    if (e != hipSuccess || a.ksplit == 1) return e;
    if (a.r == 0) launch_sum<0>(a, stream);
    else if (a.r <= 64) launch_sum<2>(a, stream);
    else launch_sum<4>(a, stream);
    return hipGetLastError();
}

// Reduction steps of 128 codes split as the bf16 products' are (fewer output tiles than half the CUs).
SplitPlan int8_gemm_split(int64_t M, int64_t N, int64_t K) {
    return gemm_split(((M + TM - 1) / TM) * ((N + TN - 1) / TN), (K + TKB - 1) / TKB, 4);
}

}  // namespace nf4k
