// dX of the Int8 QLoRA linear backward where expanding the weight to bf16 first would cost
// more than it saves, as up to about a thousand tokens (gfx950):
//   dX = dY . W' + (dT + dTlo) . L1^T,   W'[n, k] = bf16(ws[n] Wq[n, k]),   reduction over the W rows n
//
// Page: "QLoRA: Efficient Finetuning of Quantized LLMs" study notes (gitcode.csdn.net), section 3.1
// eq. (2) (dequantization, here one constant per row), section 3.5 (the gradient to X runs through the
// BF16 weight), section 4 eq. (3).
//
// Block tile TM x 256 outputs (TM 64 up to 64 tokens, else 128), reduction step 64, 8 waves in 2 x 4,
// MFMA v_mfma_f32_32x32x16_bf16.  dY goes straight from global memory to LDS, 16-byte chunks XOR-swizzled
// by (row / 2).  The weight's 64 x 256 codes of a step come through registers four steps ahead and are
// turned to bf16 on the way to LDS, spread over the MFMA sub-steps: a code costs one conversion of a
// signed byte (v_cvt_f32_i32 with a byte select), one multiplication and half a packed conversion.  The
// W rows are the reduction, so fragments are read with ds_read_b64_tr_b16.  The adapter is r/64 more steps, with dT
// in two bf16 halves: one alone would lose as much of the adapter's term as dX's own rounding.
//
// Bound by no one unit: over a large product the MFMAs are busy 47 % of the CUs' cycles and LDS 59 %
// (counters, 1023 x 22016 x 8192).  Measured, the whole backward with r = 16: 66 us at 333 tokens x 11008 x
// 4096 (this kernel 47), 99 with the weight expanded first.  Four waves of 64 x 128 instead of eight of
// 64 x 64 measured 2 to 6 % slower.
//
// Few output tiles: the reduction is split over up to 16 workgroups per tile, which write float32
// partial tiles that a fixed-order reduction sums (and adds to dX when accumulating).

#include "common.h"
#include "dqtile.h"
#include "int8.h"
#include "launch.h"

namespace nf4k {

namespace {

constexpr int TN = 256;          // output columns per block tile
constexpr int TK = 64;           // W rows per step
// The end of a step: at most VM of the wave's loads still in flight, its LDS operations done, then the
// workgroup barrier.  (__syncthreads would wait for every direct-to-LDS load in flight, those of later
// steps too.)
template <int VM>
__device__ __forceinline__ void step_end() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}
constexpr int ROWB_RED = (TK + 8) * 2;     // adapter step's L1: [256 out][64 red]
// weight step: [64 red][256 out].  A row starts 16 banks after the one before, so that the transposing
// reads of four rows by 32 columns touch each bank once; and the 16-byte pieces of columns 128 .. 255 are
// swapped in pairs, so that 16 lanes writing every second piece of a row do too.
constexpr int ROWB_OUT = (TN + 32) * 2;
constexpr int B_STAGE = (TN * ROWB_RED > TK * ROWB_OUT) ? TN * ROWB_RED : TK * ROWB_OUT;

template <int TM, int NW>
__global__ __launch_bounds__(NW * 64) void int8_bwd_kernel(Int8Bwd g) {
    constexpr int NT = NW * 64;
    constexpr int WR = NT / 16, WQ = TK / WR;         // weight rows per pass of the workgroup, passes per step
    constexpr int WL = 2 * WQ;                        // a thread's weight loads per step: codes and constants
    constexpr int A_STAGE = TM * TK * 2;
    constexpr int WN_WAVES = NW / 2;                  // waves along the output columns, two along the rows
    constexpr int WT_M = TM / 2, WT_N = TN / WN_WAVES;   // wave tile
    constexpr int IM = WT_M / 32, JN = WT_N / 32;
    constexpr int QA = TM / (8 * NW);                       // dY loads (1 KB each) per wave and step
    // each stage its own LDS object: a read of one provably never aliases the loads into another
    __shared__ __align__(16) uint8_t As0[A_STAGE];
    __shared__ __align__(16) uint8_t As1[A_STAGE];
    __shared__ __align__(16) uint8_t As2[A_STAGE];
    __shared__ __align__(16) uint8_t As3[A_STAGE];
    __shared__ __align__(16) uint8_t Bs0[B_STAGE];
    __shared__ __align__(16) uint8_t Bs1[B_STAGE];
    typedef __attribute__((address_space(3))) uint8_t lds_u8;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN_WAVES, wn = wave & (WN_WAVES - 1);
    const int r32 = lane & 31, hh = lane >> 5;

    const int ntm = (int)((g.M + TM - 1) / TM);
    const int ntn = (int)((g.K + TN - 1) / TN);
    const int ntiles = ntm * ntn;
    const int split = (int)(blockIdx.x / (uint32_t)ntiles);
    int tm, tn;
    tile_coords_grouped<4>(ntm, ntn, (int)blockIdx.x - split * ntiles, tm, tn);
    const int64_t m0 = (int64_t)tm * TM;
    const int64_t o0 = (int64_t)tn * TN;
    // this workgroup's steps: kb .. kb + steps - 1
    const int kb = split * g.split_per;
    const int steps = min((int)((g.N + TK - 1) / TK) - kb, g.split_per);
    const int ext_steps = split == g.ksplit - 1 ? (g.r + TK - 1) / TK : 0;

    const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.dY + m0 * g.N, (g.M - m0) * g.N * 2);
    const __amdgpu_buffer_rsrc_t rW = make_rsrc(g.Wq, g.N * g.K);
    const __amdgpu_buffer_rsrc_t rS = make_rsrc(g.ws, g.N * 4);

    // ---- dY: instruction q of a wave writes LDS rows 8u .. 8u+7 (u = QA wave + q); lane l -> row
    // 8u + l/8, physical chunk l%8, which holds logical chunk (l%8) ^ ((row/2)%8) ----
    uint32_t a_voff[QA];
    int a_col[QA];
#pragma unroll
    for (int q = 0; q < QA; ++q) {
        const int row = 8 * (QA * wave + q) + (lane >> 3);
        a_col[q] = ((lane & 7) ^ ((row >> 1) & 7)) * 8;
        a_voff[q] = (uint32_t)((row * g.N + a_col[q]) * 2);
    }
    const int nend = (int)min(g.N, (int64_t)(kb + steps) * TK);     // the split's end; zeros past it
    auto load_A = [&](int step, uint8_t *Ad) {
        const int n0 = (kb + step) * TK, rem = nend - n0;
        lds_u8 *dst = (lds_u8 *)Ad + wave * (QA * 1024);
#pragma unroll
        for (int q = 0; q < QA; ++q) {
            const uint32_t off = a_col[q] < rem ? a_voff[q] + (uint32_t)n0 * 2 : 0xFFFFFFF0u;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(dst + q * 1024), 16, off, 0, 0, 0);
        }
        // what follows stays behind these loads: the waits count on the order
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- W: thread -> rows tid/16 + WR q of the step, columns 16 (tid%16) .. +15: 16 lanes
    // read 256 contiguous bytes of a row ----
    const int w_row = tid >> 4, w_col = (tid & 15) * 16;
    struct WStage {
        u32x4 w[WQ];
        uint32_t s[WQ];
    };
    // The loads go out in step order, so row and offset are kept and moved on (a multiplication and a
    // branch less per step).  Rows past the end and columns past K (all 16 of a thread, K % 64 == 0) read
    // zeros; offsets stay below 2^32: N K < 2^31, and at most 8 steps of 64 K beyond.
    const int w_end = o0 + w_col < g.K ? nend : 0;
    int w_n = kb * TK + w_row;
    uint32_t w_off = (uint32_t)((int64_t)w_n * g.K + o0 + w_col);
    const uint32_t rowq = (uint32_t)(WR * g.K), row64 = (uint32_t)(64 * g.K);
    auto load_W = [&](WStage &st) {
#pragma unroll
        for (int q = 0; q < WQ; ++q) {
            const bool in = w_n + WR * q < w_end;
            st.w[q] = bload16(rW, in ? w_off + q * rowq : 0xFFFFFFF0u);
            st.s[q] = bload4(rS, in ? (uint32_t)(w_n + WR * q) * 4 : 0xFFFFFFF0u);
        }
        w_n += TK;
        w_off += row64;
    };
    // part p (0 .. 2 WQ - 1) of a stage to bf16: eight codes of row p / 2 (rows past the end: constant 0, so zeros)
    auto write_B = [&](const WStage &st, uint8_t *Bst, int p) {
        const int q = p >> 1, h = p & 1;
        const float s = __uint_as_float(st.s[q]);
        uint32_t o[4];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const int32_t u = (int32_t)st.w[q][2 * h + d];
            const float f0 = (float)(int8_t)u * s;
            const float f1 = (float)(int8_t)(u >> 8) * s;
            const float f2 = (float)(int8_t)(u >> 16) * s;
            const float f3 = (float)(u >> 24) * s;
            o[2 * d] = pack_bf16x2(f0, f1);
            o[2 * d + 1] = pack_bf16x2(f2, f3);
        }
        *reinterpret_cast<u32x4 *>(Bst + (w_row + WR * q) * ROWB_OUT + w_col * 2 + 16 * (h ^ (w_col >> 7))) = u32x4{o[0], o[1], o[2], o[3]};
    };

    f32x16 acc[IM][JN];
#pragma unroll
    for (int i = 0; i < IM; ++i)
#pragma unroll
        for (int j = 0; j < JN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // ---- fragments of sub-step s (16 reduction elements): lane (r32, hh) takes elements 16 s + 8 hh ..
    // +7 of its row (A) or column (B) ----
    auto frag_A = [&](const uint8_t *Ast, int s, int i) -> bf16x8 {
        const int row = wm * WT_M + i * 32 + r32;
        return *reinterpret_cast<const bf16x8 *>(Ast + row * 128 + ((2 * s + hh) ^ ((row >> 1) & 7)) * 16);
    };
    // from a [red][out] tile: 16-lane group (hh, half), lane i of it reads row 16 s + 8 hh + i/4 (+4),
    // columns col0 + 4 (i%4) .. +3; after the transpose it holds column col0 + i
    auto frag_B = [&](const uint8_t *Bst, int s, int j) -> bf16x8 {
        const int i16 = lane & 15, half = (lane >> 4) & 1;
        const int col0 = wn * WT_N + j * 32 + half * 16;
        const int rowb = s * 16 + hh * 8 + (i16 >> 2);
        const uint8_t *base = Bst + (col0 + ((4 * (i16 & 3)) ^ (col0 >> 7 << 3))) * 2;
        const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(base + rowb * ROWB_OUT));
        const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(base + (rowb + 4) * ROWB_OUT));
        const v8i16 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf16x8, v);
    };
    auto frag_rowread = [&](const uint8_t *Bst, int s, int j) -> bf16x8 {
        const int row = wn * WT_N + j * 32 + r32;
        return *reinterpret_cast<const bf16x8 *>(Bst + row * ROWB_RED + (s * 16 + hh * 8) * 2);
    };
    struct Frags {
        bf16x8 a[IM], b[JN];
    };
    auto load_frags = [&](const uint8_t *Ast, const uint8_t *Bst, int s, Frags &f) {
#pragma unroll
        for (int i = 0; i < IM; ++i) f.a[i] = frag_A(Ast, s, i);
#pragma unroll
        for (int j = 0; j < JN; ++j) f.b[j] = frag_B(Bst, s, j);
    };
    auto mma = [&](const Frags &f) {
#pragma unroll
        for (int i = 0; i < IM; ++i)
#pragma unroll
            for (int j = 0; j < JN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
    };
    // one sub-step: its MFMAs, the next sub-step's fragment reads, and up to half of the next step's
    // conversion, interleaved
    auto interleave = [&](auto parts) {
        constexpr int NM = IM * JN, ND = IM + 2 * JN, dsw = decltype(parts)::value, valu = 24 * dsw;
#pragma unroll
        for (int k = 0; k < NM; ++k) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                      // 1 MFMA
            __builtin_amdgcn_sched_group_barrier(0x002, (valu + NM - 1) / NM, 0);   // VALU
            __builtin_amdgcn_sched_group_barrier(0x100, (ND + NM - 1) / NM, 0);     // DS reads
            if (k >= NM - dsw) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);   // DS write
        }
    };

    // ---- main loop.  Step s computes stage (Ac, Bc); its next stage's dY landed earlier, and the codes
    // of step s + 1 (registers) become bf16 in Bn during sub-steps 0 to 2.  The barrier sits between
    // sub-steps 2 and 3: by then every wave has its last fragments of the stage in registers and Bn is
    // whole, so the first fragments of the next stage are read under sub-step 3's MFMAs.  After it, dY
    // of step s + 4 starts into the stage's own LDS and the codes of step s + 4 into registers: three
    // steps ahead, since with one each step waited out the loads' latency. ----
    WStage R0, R1, R2, R3;
    Frags f0, f1;
    // Loads issued after dY of step s + 1 that may still be in flight at step s's barrier: step s + 1's
    // codes, then dY and codes of two more steps.
    constexpr int kWaitVm = WL + 2 * (QA + WL);
    auto step_do = [&](int step, uint8_t *Ac, const uint8_t *Bc, const uint8_t *An, uint8_t *Bn, const WStage &conv,
                       WStage &fill) {
        load_frags(Ac, Bc, 1, f1);
        mma(f0);
#pragma unroll
        for (int p = 0; p < WQ; ++p) write_B(conv, Bn, p);
        interleave(IntConst<WQ>());
        __builtin_amdgcn_sched_barrier(0);
        load_frags(Ac, Bc, 2, f0);
        mma(f1);
#pragma unroll
        for (int p = WQ; p < WQ + WQ / 2; ++p) write_B(conv, Bn, p);
        interleave(IntConst<WQ / 2>());
        __builtin_amdgcn_sched_barrier(0);
        load_frags(Ac, Bc, 3, f1);
        mma(f0);
#pragma unroll
        for (int p = WQ + WQ / 2; p < 2 * WQ; ++p) write_B(conv, Bn, p);
        interleave(IntConst<WQ / 2>());
        __builtin_amdgcn_sched_barrier(0);
        step_end<kWaitVm>();
        load_A(step + 4, Ac);
        load_W(fill);
        load_frags(An, Bn, 0, f0);
        mma(f1);
        __builtin_amdgcn_sched_barrier(0);
    };
    load_A(0, As0);
    load_W(R0);
    load_A(1, As1);
    load_W(R1);
    load_A(2, As2);
    load_W(R2);
    load_A(3, As3);
    load_W(R3);
#pragma unroll
    for (int p = 0; p < 2 * WQ; ++p) write_B(R0, Bs0, p);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    load_frags(As0, Bs0, 0, f0);
    // whole groups of four steps: those past the end multiply zeros (leaving in mid-group made the
    // compiler copy registers with loads in flight, and wait for them)
    for (int step = 0; step < steps; step += 4) {
        step_do(step, As0, Bs0, As1, Bs1, R1, R0);
        step_do(step + 1, As1, Bs1, As2, Bs0, R2, R1);
        step_do(step + 2, As2, Bs0, As3, Bs1, R3, R2);
        step_do(step + 3, As3, Bs1, As0, Bs0, R0, R3);
    }
    __builtin_amdgcn_s_waitcnt(0);               // loads past the end still write their zeros
    __syncthreads();

    // ---- adapter: r/64 more steps (zero padded past r), dT's first halves in As0, its second in As1 ----
    if (ext_steps > 0) {
        const __amdgpu_buffer_rsrc_t rAe = make_rsrc(g.dT + m0 * g.r, (g.M - m0) * (int64_t)g.r * 2);
        const __amdgpu_buffer_rsrc_t rAl = make_rsrc(g.dTlo + m0 * g.r, (g.M - m0) * (int64_t)g.r * 2);
        const __amdgpu_buffer_rsrc_t rBe = make_rsrc(g.L1 + o0 * g.r, (g.K - o0) * (int64_t)g.r * 2);
        for (int e = 0; e < ext_steps; ++e) {
#pragma unroll
            for (int q = 0; q < TN / (8 * NW); ++q) {
                const int row = (tid >> 3) + 8 * NW * q, chunk = tid & 7;
                const int jj = e * TK + chunk * 8;
                const uint32_t off = jj < g.r ? (uint32_t)((row * (int64_t)g.r + jj) * 2) : 0xFFFFFFF0u;
                if (row < TM) {
                    const int at = row * 128 + (chunk ^ ((row >> 1) & 7)) * 16;
                    *reinterpret_cast<u32x4 *>(As0 + at) = bload16(rAe, off);
                    *reinterpret_cast<u32x4 *>(As1 + at) = bload16(rAl, off);
                }
                *reinterpret_cast<u32x4 *>(Bs0 + row * ROWB_RED + chunk * 16) = bload16(rBe, off);
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                Frags f;
#pragma unroll
                for (int i = 0; i < IM; ++i) f.a[i] = frag_A(As0, s, i);
#pragma unroll
                for (int j = 0; j < JN; ++j) f.b[j] = frag_rowread(Bs0, s, j);
                mma(f);
#pragma unroll
                for (int i = 0; i < IM; ++i) f.a[i] = frag_A(As1, s, i);
                mma(f);
            }
            __syncthreads();
        }
    }

    // ---- store: lane (r32, hh) of tile (i, j) holds column 32 j + r32 and rows 32 i + 8 (v/4) + 4 hh +
    // v%4; rows past M fall outside the descriptors ----
    const int64_t c0 = o0 + wn * WT_N + r32;
    if (g.ksplit > 1) {
        const __amdgpu_buffer_rsrc_t rP = make_rsrc(g.P + (int64_t)split * g.M * g.K + m0 * g.K, (g.M - m0) * g.K * 4);
        const uint32_t prow = (uint32_t)(g.K * 4);
        const uint32_t poff = (uint32_t)((wm * WT_M + hh * 4) * prow) + (uint32_t)(c0 * 4);
#pragma unroll
        for (int j = 0; j < JN; ++j) {
            if (c0 + j * 32 >= g.K) continue;
#pragma unroll
            for (int i = 0; i < IM; ++i)
#pragma unroll
                for (int v = 0; v < 16; ++v)
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[i][j][v]), rP, poff + j * 128,
                                                          (uint32_t)(i * 32 + (v >> 2) * 8 + (v & 3)) * prow, 0);
        }
        return;
    }
    const __amdgpu_buffer_rsrc_t rC = make_rsrc(g.dX + m0 * g.K, (g.M - m0) * g.K * 2);
    const uint32_t row_bytes = (uint32_t)(g.K * 2);
    const uint32_t lane_off = (uint32_t)((wm * WT_M + hh * 4) * row_bytes) + (uint32_t)(c0 * 2);
#pragma unroll
    for (int j = 0; j < JN; ++j) {
        if (c0 + j * 32 >= g.K) continue;
#pragma unroll
        for (int i = 0; i < IM; ++i) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const uint32_t soff = (uint32_t)(i * 32 + (v >> 2) * 8 + (v & 3)) * row_bytes;
                float f = acc[i][j][v];
                if (g.accumulate)
                    f += bf16_to_f32((uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rC, lane_off + j * 64, soff, 0) & 0xFFFFu);
                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f32_to_bf16(f), rC, lane_off + j * 64, soff, 0);
            }
        }
    }
}

}  // namespace

SplitPlan int8_bwd_split(int64_t M, int64_t N, int64_t K) {
    const int64_t TM = int8_bwd_tile(M);
    return gemm_split(((M + TM - 1) / TM) * ((K + TN - 1) / TN), (N + TK - 1) / TK, 4);
}

hipError_t launch_int8_bwd(const Int8Bwd &p, hipStream_t stream) {
    const int64_t TM = int8_bwd_tile(p.M);
    const int64_t tiles = ((p.M + TM - 1) / TM) * ((p.K + TN - 1) / TN), steps = (p.N + TK - 1) / TK;
    Int8Bwd a = p;
    if (a.ksplit <= 1) {
        a.ksplit = 1;
        a.split_per = (int32_t)steps;
    } else if (!a.P || (int64_t)(a.ksplit - 1) * a.split_per >= steps || (int64_t)a.ksplit * a.split_per < steps) {
        return hipErrorInvalidValue;     // every split non-empty, the partials somewhere to go
    }
    const dim3 grid((unsigned)(tiles * a.ksplit));
    timing_before(stream, 1);
    if (TM == 64) hipLaunchKernelGGL((int8_bwd_kernel<64, 8>), grid, dim3(512), 0, stream, a);
    else hipLaunchKernelGGL((int8_bwd_kernel<128, 8>), grid, dim3(512), 0, stream, a);
    const hipError_t e = hipGetLastError();
    timing_after(stream);
    return e;
}

}  // namespace nf4k
