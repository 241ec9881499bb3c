// dX's product of the loss over the vocabulary (gfx950):  D[t, n] = sum_v P[t, v] W[v, n]  over a piece
// of the vocabulary, P as loss_logits.hip wrote it.
//
// The reduction runs over W's rows, so W's tile is staged as it lies in memory (64 rows of 256 columns) and
// its fragments come from transposing LDS reads (ds_read_b64_tr_b16: each 16-lane group turns 4 rows x 16
// columns).  A row of the stage is 512 bytes; its 64-byte granules are XOR-swizzled by row % 4, so the
// four rows that half a wave reads at once lie in different banks.  P's blocks are copied as they are.
//
// The MFMAs take W's columns as the first operand and the tokens as the second: a lane holds four
// consecutive columns of a token; the results are turned through LDS into rows.
//
// One workgroup a CU; the tiles beyond whole rounds are shared evenly (LossShares; the live rows are counted on the
// device), with float32 partials that loss_fold_kernel sums in a fixed order.
//
// Bound by the MFMAs as the logits are: 4096 x 32000 x 4096 798 us of kernel, 1.35 PFLOP/s (a library product of these
// sizes 1.29); 777 x 50001 x 8192 with 700 labelled 503 to 523 us and the fold 20.

#include "common.h"
#include "dqtile.h"
#include "loss.h"
#include "loss_tile.h"

namespace nf4k {

namespace {

__global__ __launch_bounds__(256, 1) void loss_dx_kernel(LossDxArgs g) {
    // one LDS object per stage: a fragment read of one stage provably never aliases the
    // direct-to-LDS loads in flight into the other
    __shared__ __align__(16) uint8_t S0[2 * LOPB];
    __shared__ __align__(16) uint8_t S1[2 * LOPB];

    const int count = __builtin_amdgcn_readfirstlane(g.r.count[0]);
    const int ntm = (count + LT - 1) / LT, ntn = (int)((g.K + LT - 1) / LT);
    const LossShares sh(ntm * ntn, g.steps);
    // each XCD (blockIdx % 8) takes a contiguous run of tiles, of parts, and of the tails' runs
    const int xcd = (int)blockIdx.x & 7, slot = (int)blockIdx.x >> 3;
    const int rounds = sh.whole / 256, parts = sh.ks * sh.rest;
    const int p0 = parts * xcd / 8, p1 = parts * (xcd + 1) / 8, mine = p0 + slot;
    bool part_left = mine < p1;
    // with runs, parts and runs are 256 together: what an XCD's 32 workgroups have left over
    const bool runs = sh.extra && !part_left;
    const int run = 32 * xcd - p0 + slot - (p1 - p0);
    int64_t at = runs ? sh.begin(run) : 0;
    const int64_t until = runs ? sh.begin(run + 1) : 0;

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;      // along dX's columns, along the tokens
    const int r32 = lane & 31, hh = lane >> 5;

#pragma unroll 1
    for (int round = 0;; ++round) {
        // this turn's tile and its steps
        int tile, kb = 0, steps = g.steps;
        bool split_up = false;
        float *part = nullptr;
        if (round < rounds) {
            tile = sh.whole / 8 * xcd + 32 * round + slot;
        } else if (part_left) {
            const int j = mine / sh.rest, x = mine % sh.rest;
            part_left = false;
            tile = sh.whole + x;
            kb = j * sh.len;
            steps = min(sh.len, g.steps - kb);
            split_up = sh.partial();
            part = g.part + (int64_t)sh.slot_part(j, x) * (LT * LT);
        } else if (at < until) {
            const int x = (int)(at / sh.tail), in = (int)(at - (int64_t)x * sh.tail);
            tile = sh.whole + x;
            kb = sh.ks * sh.len + in;
            steps = (int)min(until - at, (int64_t)(sh.tail - in));
            split_up = true;
            part = g.part + (int64_t)sh.slot_run(run, x) * (LT * LT);
            at += steps;
        } else {
            break;
        }
        int tm, tn;
        loss_place(ntm, ntn, tile, tm, tn);
        const int64_t n0 = (int64_t)tn * LT;

        // W from this turn's first row; rows past V read zeros
        const int64_t v0 = g.v0 + (int64_t)kb * LSTEP;
        const __amdgpu_buffer_rsrc_t rA = make_rsrc(g.W + v0 * g.K, (g.V - v0) * g.K * 2);
        const __amdgpu_buffer_rsrc_t rB = make_rsrc(g.P + ((int64_t)tm * g.steps + kb) * LBLOCK, (int64_t)steps * LBLOCK * 2);

        // W: instruction q of wave w writes stage rows 2u, 2u + 1 (u = 8w + q); lane l takes row 2u + l/32 and
        // physical 16-byte chunk l%32, whose granule (l%32)/4 holds logical granule ((l%32)/4) ^ (row%4)
        uint32_t aoff[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 2 * (8 * wave + q) + (lane >> 5);
            const int col = ((((lane & 31) >> 2) ^ (row & 3)) * 4 + (lane & 3)) * 8;
            aoff[q] = n0 + col < g.K ? (uint32_t)((row * g.K + n0 + col) * 2) : 0x80000000u;
        }
        const uint32_t row4_off = (uint32_t)(4 * g.K * 2);
        const uint32_t step_off = (uint32_t)(LSTEP * g.K * 2);
        // P: instruction q of wave w copies rows 64 w + 8 q ..; past the live rows there is nothing to read
        uint32_t boff[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            boff[q] = tm * LT + 64 * wave + 8 * q + (lane >> 3) < count ? (uint32_t)(wave * 8192 + q * 1024 + lane * 16) : 0x80000000u;
        auto load = [&](int step, uint8_t *st, int part) {
            lds_u8 *da = (lds_u8 *)st + wave * 8192, *db = (lds_u8 *)(st + LOPB) + wave * 8192;
            const uint32_t dead = step < steps ? 0u : 0x80000000u;      // past the descriptor's end
            const int bstep = min(step, steps - 1) * (int)(LBLOCK * 2);    // P's blocks are whole: the last one again
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                if ((q >> 2) != part) continue;
                // rows 2q and 2q + 1 of the wave's 16: q and q + 2 share row % 4
                const uint32_t v = aoff[q & 1] + (uint32_t)(q >> 1) * row4_off + (uint32_t)step * step_off;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void *)(da + q * 1024), 16, v | dead, 0, 0, 0);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rB, (lds_void *)(db + q * 1024), 16, boff[q], bstep, 0, 0);
            }
        };
        // W's fragment of sub-step s, columns wm*128 + 32 i ..: 16-lane group (hh, half) reads rows
        // 16 s + 8 hh + i16/4 (+ 4), columns 16 half + 4 (i16 % 4) .. +3; lane i16 ends with column 16 half + i16
        const int i16 = lane & 15, half = (lane >> 4) & 1, rq = i16 >> 2;
        uint32_t aread[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            aread[i] = (uint32_t)((8 * hh + rq) * 512 + ((wm * 4 + (i ^ rq)) * 64) + half * 32 + (i16 & 3) * 8);
        uint32_t bread[4];
#pragma unroll
        for (int s = 0; s < 4; ++s) bread[s] = (uint32_t)(r32 * 128 + (((2 * s + hh) ^ ((r32 >> 1) & 7)) * 16));
        auto read = [&](const uint8_t *A, int s, LossFrags<4> &f) {
            const uint8_t *B = A + LOPB;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *p = A + aread[i] + s * 16 * 512;
                const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)p);
                const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(p + 4 * 512));
                f.a[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) f.b[j] = *reinterpret_cast<const bf16x8 *>(B + bread[s] + (wn * 128 + 32 * j) * 128);
        };
        f32x16 acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        load(0, S0, 0);
        load(0, S0, 1);
        loss_loop<4, 12, 8, 0>(steps, false, S0, S1, acc, load, read);

        // Lane (r32, hh) of tile (i, j) holds token wn*128 + 32 j + r32 and columns wm*128 + 32 i + 8 (v/4) + 4 hh + v%4.
        // Each wave turns its 128 x 128 values in its own stage of LDS, 64 tokens at a time, into rows of 512 bytes (their
        // 16-byte chunks XOR-swizzled by the row), so that all that follows moves whole lines, two tokens at a time.
        const int lane_e = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
        const int c32 = lane_e & 31, he = lane_e >> 5;
        uint8_t *turn = (wave < 2 ? S0 : S1) + (wave & 1) * LOPB;
        const bool add = !split_up && g.c_old, last = !split_up && g.dX;
        // K is a multiple of 64: what lies past it are whole lanes here
        const int64_t col = n0 + wm * 128 + 4 * c32;
        const bool in = split_up || col < g.K;
        const int64_t colc = in ? col : 0, ld = split_up ? LT : g.K;
        float *dst32 = split_up ? part + wm * 128 + 4 * c32 : g.sum32 + (int64_t)tm * LT * g.K + colc;
#pragma unroll
        for (int jh = 0; jh < 2; ++jh) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        const f32x16 &x = acc[i][2 * jh + j];
                        *reinterpret_cast<f32x4 *>(turn + (32 * j + c32) * 512 + (((8 * i + 2 * v4 + he) ^ c32) * 16)) =
                            f32x4{x[4 * v4], x[4 * v4 + 1], x[4 * v4 + 2], x[4 * v4 + 3]};
                    }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            // lane l: what row l of these 64 needs (dead rows: row 0's, not stored)
            const int r0 = wn * 128 + 64 * jh, live = count - tm * LT - r0;
            const int tl = lane_e < live ? tm * LT + r0 + lane_e : 0;
            const float move = add ? __builtin_amdgcn_exp2f(g.c_old[tl] - g.c[tl]) : 0.0f;
            const float fa = last ? g.r.a[tl] : 0.0f, fb = last ? g.r.b[tl] : 0.0f;
            const int frow = last ? g.r.row[tl] : 0, flab = last ? max(g.r.label[tl], 0) : 0;
            auto of = [&](int v, int u) {      // row 2u's value in the lower half, row 2u + 1's in the upper
                const int a = __builtin_amdgcn_readlane(v, 2 * u), b = __builtin_amdgcn_readlane(v, 2 * u + 1);
                return he ? b : a;
            };
            auto off = [&](float v, int u) { return __int_as_float(of(__float_as_int(v), u)); };
            // eight loads at a time: nothing tells the compiler that the stores between do not change what is read
            constexpr int B = 8;
#pragma unroll 1
            for (int u0 = 0; u0 < 32; u0 += B) {
                if (2 * u0 >= live) break;
                f32x4 x[B], o[B];
                uint2 w[B];
#pragma unroll
                for (int u = 0; u < B; ++u) {
                    const int r = 2 * (u0 + u) + he;
                    const int rc = r < live ? r0 + r : 0;
                    if (add) o[u] = *reinterpret_cast<const f32x4 *>(dst32 + (int64_t)rc * ld);
                    if (last) w[u] = *reinterpret_cast<const uint2 *>(g.W + (int64_t)of(flab, u0 + u) * g.K + colc);
                    x[u] = *reinterpret_cast<const f32x4 *>(turn + r * 512 + ((c32 ^ (r & 31)) * 16));
                }
#pragma unroll
                for (int u = 0; u < B; ++u) {
                    const int r = 2 * (u0 + u) + he;
                    if (add) x[u] += o[u] * off(move, u0 + u);
                    const LossFinal fin{off(fa, u0 + u), off(fb, u0 + u)};
                    const int row = of(frow, u0 + u);
                    if (r >= live || !in) continue;
                    if (last) *reinterpret_cast<uint2 *>(g.dX + (int64_t)row * g.K + col) = fin.value(x[u], w[u]);
                    else *reinterpret_cast<f32x4 *>(dst32 + (int64_t)(r0 + r) * ld) = x[u];
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        __syncthreads();       // the stages are free
    }
}

// Workgroup: FR rows of a tile with partials; the last one: the losses' mean
constexpr int FR = 8;
__global__ __launch_bounds__(256) void loss_fold_kernel(LossDxArgs g) {
    const int count = g.r.count[0];
    const int ntm = (count + LT - 1) / LT, ntn = (int)((g.K + LT - 1) / LT);
    const LossShares sh(ntm * ntn, g.steps);
    if (blockIdx.x == gridDim.x - 1) {
        if (g.mean) loss_write_mean(g.r.sums, (int)((g.M + kLossJoinRows - 1) / kLossJoinRows), count, g.mean);
        return;
    }
    const int x = (int)blockIdx.x / (LT / FR), r0 = (int)blockIdx.x % (LT / FR) * FR;
    if (x >= sh.rest || !sh.partial()) return;
    int tm, tn;
    loss_place(ntm, ntn, sh.whole + x, tm, tn);
    if (tm * LT + r0 >= count) return;
    // the tile's parts and the runs of its tail, in the order of its steps
    const int e0 = sh.extra ? sh.run_of((int64_t)x * sh.tail) : 0;
    const int np = sh.ks, n = np + (sh.extra ? sh.run_of((int64_t)(x + 1) * sh.tail - 1) - e0 + 1 : 0);
    auto of = [&](int i) { return i < np ? sh.slot_part(i, x) : sh.slot_run(e0 + i - np, x); };
    // two columns' worth of 16 bytes a thread, four partials of both at a time
    constexpr int N = FR * (LT / 4) / 256;
    const int c = threadIdx.x % (LT / 4) * 4, k = tn * LT + c;
    int row[N];
    const float *p[N];
    f32x4 x4[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int tl = r0 + i * (256 / (LT / 4)) + (int)threadIdx.x / (LT / 4);
        row[i] = tm * LT + tl;
        p[i] = g.part + tl * LT + c;
        x4[i] = f32x4{0, 0, 0, 0};
    }
    // what the last step takes, on its way beside the partials (a label out of the vocabulary: a and b are NaN)
    uint2 w[N];
    LossFinal fin[N];
    int token[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!g.dX || row[i] >= count || k >= g.K) continue;
        w[i] = *reinterpret_cast<const uint2 *>(g.W + (int64_t)max(g.r.label[row[i]], 0) * g.K + k);
        fin[i] = LossFinal{g.r.a[row[i]], g.r.b[row[i]]};
        token[i] = g.r.row[row[i]];
    }
    for (int s0 = 0; s0 < n; s0 += 4) {
        f32x4 v[N][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t o = s0 + u < n ? (int64_t)of(s0 + u) * (LT * LT) : 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (s0 + u < n && row[i] < count) v[i][u] = *reinterpret_cast<const f32x4 *>(p[i] + o);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (s0 + u < n) x4[i] += v[i][u];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (row[i] >= count || k >= g.K) continue;
        const int t = row[i];
        f32x4 *sum = g.sum32 ? reinterpret_cast<f32x4 *>(g.sum32 + (int64_t)t * g.K + k) : nullptr;
        if (g.c_old) x4[i] += *sum * __builtin_amdgcn_exp2f(g.c_old[t] - g.c[t]);
        if (!g.dX) {
            *sum = x4[i];
            continue;
        }
        *reinterpret_cast<uint2 *>(g.dX + (int64_t)token[i] * g.K + k) = fin[i].value(x4[i], w[i]);
    }
}

}  // namespace

hipError_t launch_loss_dx(const LossDxArgs &a, hipStream_t stream) {
    hipLaunchKernelGGL(loss_dx_kernel, dim3(256), dim3(256), 0, stream, a);      // a workgroup on each CU
    return hipGetLastError();
}

hipError_t launch_loss_fold(const LossDxArgs &a, hipStream_t stream) {
    // fewer than 256 tiles have partials, and no more than there are
    const int64_t tiles = (int64_t)(a.Mp / LT) * ((a.K + LT - 1) / LT);
    hipLaunchKernelGGL(loss_fold_kernel, dim3((uint32_t)((tiles < 255 ? tiles : 255) * (LT / FR) + 1)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nf4k
