// What stands around the two products of the loss over the vocabulary (gfx950): the live rows, the sums over
// the vocabulary's tiles, the losses, and dX from its partials.  With d = ln sum_{v != y} e^z_v - z_y (the
// log odds against the label y):
//   loss = ln(1 + e^d) = max(d, 0) + ln(1 + e^-|d|),   1 - p_y = 1 / (1 + e^-d)
//   dX = g (sum_{v != y} p_v W_v - (1 - p_y) W_y) = g (1 - p_y) (sum_{v != y} e^z_v W_v / sum_{v != y} e^z_v - W_y)
// The e^z_v of the last form are bf16 above and below the line; in d they are not rounded.
// Nothing here subtracts two large numbers: a label that is nearly certain keeps a loss and a gradient of full
// precision.
//
// All of it is latency: 4 us for the list of live rows, 6 to 13 for the join (125 tiles of 4096 rows with the
// gradient 9, 512 of 511 rows without it 9, a piece of 128 tiles of 8192 rows with it 13).

#include "common.h"
#include "loss.h"

namespace nf4k {

namespace {

constexpr int PREP = 1024;
constexpr int PREP_REST = 128;       // workgroups that clear the rows without a label, a wave a row

// Workgroup 0: the live rows, in order.  The others: loss and dX of the rest set to zero.
__global__ __launch_bounds__(PREP) void loss_prep_kernel(const int64_t *__restrict__ labels, int64_t M, int64_t V, int64_t K,
                                                         LossRows r, float *__restrict__ loss, uint16_t *__restrict__ dX) {
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int lane = tid & 63;
        for (int64_t m = (int64_t)(blockIdx.x - 1) * (PREP / 64) + (tid >> 6); m < M; m += (int64_t)(gridDim.x - 1) * (PREP / 64)) {
            if (labels[m] >= 0) continue;
            if (lane == 0) loss[m] = 0.0f;
            if (dX)
                for (int64_t k = lane * 8; k < K; k += 64 * 8) *reinterpret_cast<u32x4 *>(dX + m * K + k) = u32x4{0, 0, 0, 0};
        }
        return;
    }
    // runs of 64 labels, a wave each: how many are live, where each run's rows begin, then the rows themselves; 1024
    // runs at a time
    __shared__ int begin[PREP], waves[PREP / 64];
    const int lane = tid & 63, wave = tid >> 6;
    auto label = [&](int64_t m) { return m < M ? labels[m] : (int64_t)-1; };
    int base = 0;
    for (int64_t b = 0; b < M; b += (int64_t)PREP * 64) {
        const int runs = (int)min((M - b + 63) / 64, (int64_t)PREP);
        for (int run = wave; run < runs; run += PREP / 64) {
            const uint64_t live = __builtin_amdgcn_ballot_w64(label(b + 64 * run + lane) >= 0);
            if (lane == 0) begin[run] = __popcll(live);
        }
        __syncthreads();
        // exclusive sums of the runs' counts: within a wave, then over the waves
        const int n = tid < runs ? begin[tid] : 0;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(sum, d);
            if (lane >= d) sum += v;
        }
        if (lane == 63) waves[wave] = sum;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < PREP / 64; ++w) {
            before += w < wave ? waves[w] : 0;
            all += waves[w];
        }
        begin[tid] = base + before + sum - n;
        __syncthreads();
        for (int run = wave; run < runs; run += PREP / 64) {
            const int64_t m = b + 64 * run + lane, l = label(m);
            const uint64_t live = __builtin_amdgcn_ballot_w64(l >= 0);
            if (l < 0) continue;
            const int at = begin[run] + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(live >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)live, 0u));
            r.row[at] = (int32_t)m;
            r.label[at] = l < V ? (int32_t)l : -1;
        }
        base += all;
        __syncthreads();
    }
    if (tid == 0) r.count[0] = base;
}

// JR rows a workgroup and 256 / JR threads over the tiles of a row.  NARROW: tiles of one step, never cut, and tables by
// row ([row][tile]); otherwise tiles of four steps, cut ones among them, and tables by tile ([tile][Mp]).
template <int JR, bool NARROW>
__global__ __launch_bounds__(256) void loss_join_kernel(LossJoin g) {
    constexpr int JS = 256 / JR, BLOCKS = NARROW ? 1 : 4;
    constexpr int W0 = NARROW ? 1 : JR, NWR = NARROW ? 4 / JR : 4;      // first lane step of a row; waves that share one
    __shared__ float pc[4][JR], ps[4][JR], pp[4][JR];
    __shared__ double sl[JR];
    const int count = g.r.count[0];
    const int tid = threadIdx.x, lr = NARROW ? tid / JS : tid % JR, slice = NARROW ? tid % JS : tid / JR;
    const int wave = tid >> 6, w0 = NARROW ? lr * NWR : 0;
    const int row = blockIdx.x * JR + lr;
    const bool live = row < count;
    // the workgroup's sum of losses, by thread 0
    auto finish = [&](double s) {
        if (!NARROW || !g.tickets) {
            if (tid) return;
            g.r.sums[blockIdx.x] = s;
            if (gridDim.x == 1) g.mean[0] = count ? (float)(s / count) : 0.0f;
            return;
        }
        if (wave) return;
        int ended = 0;
        if (tid == 0) {
            __hip_atomic_store(&g.r.sums[blockIdx.x], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            ended = __hip_atomic_fetch_add(&g.r.count[1], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) + 1;
        }
        if (__builtin_amdgcn_readfirstlane(ended) != (int)gridDim.x) return;
        // the workgroup that ends last: the sums in a fixed order
        double all = 0.0;
        for (int i = tid; i < (int)gridDim.x; i += 64) all += __hip_atomic_load(&g.r.sums[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) all += __shfl_xor(all, d);
        if (tid == 0) g.mean[0] = count ? (float)(all / count) : 0.0f;
    };
    if ((int)blockIdx.x * JR >= count) {
        if (g.last) finish(0.0);
        return;
    }
    const float NEG = -__builtin_inff();
    const float c_old = g.c_in && live ? g.c_in[row] : NEG;
    // The new reference: the largest there is; eight tiles' loads at a time.  A tile with nothing but the label has a sum of
    // zero and a reference that says nothing.
    float c = c_old, sum = 0.0f, sum_p = 0.0f, low = -NEG;
    // entries of this row's tiles: ntile, and the second halves of the tiles that are cut
    const LossTiles tiles((count + LT - 1) / LT, g.ntile);
    const int cut = NARROW ? g.ntile : tiles.first_cut(row / LT), entries = 2 * g.ntile - cut;
    auto at = [&](int t) { return NARROW ? (int64_t)row * g.ntile + t : (int64_t)(t < g.ntile ? t : t + cut) * g.Mp + row; };
    // what the row's own results take, on its way already
    int m = 0, label = -1;
    float zl = 0.0f, weight = 0.0f;
    if (g.last && live && slice == 0) {
        m = g.r.row[row];
        label = g.r.label[row];
        zl = g.r.zl[row];
        weight = g.dloss ? g.dloss[m] : 1.0f / (float)count;
    }
    if (live)
        for (int t0 = slice; t0 < entries; t0 += JS * 8) {
            float f[8], s[8], sp[8], most = c;
            bool has[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int t = t0 + u * JS;
                has[u] = t < entries;
                f[u] = has[u] ? g.tref[at(t)] : NEG;
                s[u] = has[u] ? g.tsum[at(t)] : 0.0f;
                sp[u] = g.grad && has[u] ? g.tp[at(t)] : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                has[u] = has[u] && s[u] != 0.0f;
                most = fmaxf(most, has[u] ? f[u] : NEG);
                low = fminf(low, has[u] ? f[u] : -NEG);
            }
            // c = most also before the first tile, where there is nothing to move (and both may be -inf)
            const float move = most == c ? 1.0f : __builtin_amdgcn_exp2f(c - most);
            sum *= move;
            sum_p *= move;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (!has[u]) continue;
                const float to = __builtin_amdgcn_exp2f(f[u] - most);
                sum += s[u] * to;
                sum_p += sp[u] * to;
            }
            c = most;
        }
    float top = c;
#pragma unroll
    for (int d = W0; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    pc[wave][lr] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NWR; ++w) top = fmaxf(top, pc[w0 + w][lr]);
    const float move = sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(c - top);
    sum = sum == 0.0f ? 0.0f : sum * move;
    sum_p = sum == 0.0f ? 0.0f : sum_p * move;
#pragma unroll
    for (int d = W0; d < 64; d <<= 1) {
        sum += __shfl_xor(sum, d);
        sum_p += __shfl_xor(sum_p, d);
    }
    ps[wave][lr] = sum;
    pp[wave][lr] = sum_p;
    __syncthreads();
    // Tiles with a reference below the row's: p is brought to it (rare, and only this workgroup's rows).  Row `row` of
    // P's blocks: 128 bytes for each 64 vocabulary rows, so 512 for a whole tile.
    if (g.P && __syncthreads_or(live && !(low >= top))) {
        for (int t = slice; live && t < entries; t += JS) {
            const int tile = t < g.ntile ? t : t - g.ntile + cut;
            // blocks this entry stands for: all of its tile's, or the half's
            const int b0 = t < g.ntile ? 0 : BLOCKS / 2, b1 = t < g.ntile && tile >= cut ? BLOCKS / 2 : BLOCKS;
            const float from = g.tref[at(t)];
            if (from == top || g.tsum[at(t)] == 0.0f) continue;
            const float f = __builtin_amdgcn_exp2f(from - top);
            for (int b = b0; b < b1; ++b) {
                const int64_t block = ((int64_t)(row / LT) * g.ntile + tile) * BLOCKS + b;
                u32x4 *p = reinterpret_cast<u32x4 *>(g.P + (block * g.prows + row % LT) * LSTEP);
                for (int i = 0; i < 8; ++i) {
                    u32x4 v = p[i];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = pack_bf16x2(bf16_to_f32(v[k] & 0xFFFFu) * f, __uint_as_float(v[k] & 0xFFFF0000u) * f);
                    p[i] = v;
                }
            }
        }
    }
    if (slice == 0) {
        double value = 0.0;
        if (live) {
            const float moved = g.c_in ? __builtin_amdgcn_exp2f(c_old - top) : 0.0f;
            float S = g.c_in ? g.r.S[row] * moved : 0.0f, Sp = g.c_in && g.grad ? g.r.a[row] * moved : 0.0f;
#pragma unroll
            for (int w = 0; w < NWR; ++w) {
                S += ps[w0 + w][lr];
                Sp += pp[w0 + w][lr];
            }
            g.r.S[row] = S;
            if (g.grad && !g.last) g.r.a[row] = Sp;
            g.c_out[row] = top > NEG ? top : 0.0f;
            if (g.last) {
                // ln S + (c - zl) ln 2; a label out of the vocabulary has no logit, and one that is not finite gives NaN (as it
                // stands, d would be infinite: a loss of 0 or infinity)
                if (label < 0 || !(fabsf(zl) < __builtin_inff())) zl = __builtin_nanf("");
                const float d = (log2f(S) + (top - zl)) * kLn2;
                const float loss = fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d)));
                g.loss[m] = loss;
                value = (double)loss;
                if (g.grad) {
                    // The sum of P as it was rounded, not S: see loss_logits.hip.  (p_v's own factor, 1 / (S + 2^(zl - top)), leaves
                    // float32 where the label lies 2^128 above the reference.)
                    g.r.a[row] = Sp == 0.0f ? 0.0f : 1.0f / Sp;
                    g.r.b[row] = weight / (1.0f + expf(-d));
                }
            }
        }
        sl[lr] = value;
    }
    if (!g.last) return;
    __syncthreads();
    double s = 0.0;
    if (tid == 0)
        for (int i = 0; i < JR; ++i) s += sl[i];
    finish(s);
}

__global__ __launch_bounds__(256) void loss_mean_kernel(LossRows r, int64_t M, float *mean) {
    loss_write_mean(r.sums, (int)((M + kLossJoinRows - 1) / kLossJoinRows), r.count[0], mean);
}

}  // namespace

hipError_t launch_loss_prep(const int64_t *labels, int64_t M, int64_t V, int64_t K, const LossRows &r, float *loss,
                            uint16_t *dX, hipStream_t stream) {
    const int64_t rest = (M + PREP / 64 - 1) / (PREP / 64);
    hipLaunchKernelGGL(loss_prep_kernel, dim3(1 + (uint32_t)(rest < PREP_REST ? rest : PREP_REST)), dim3(PREP), 0, stream,
                       labels, M, V, K, r, loss, dX);
    return hipGetLastError();
}

hipError_t launch_loss_join(const LossJoin &a, bool narrow, hipStream_t stream) {
    if (narrow) {
        const uint32_t grid = (uint32_t)((a.M + kLossJoinRowsNarrow - 1) / kLossJoinRowsNarrow);
        hipLaunchKernelGGL((loss_join_kernel<kLossJoinRowsNarrow, true>), dim3(grid), dim3(256), 0, stream, a);
    } else {
        const uint32_t grid = (uint32_t)((a.M + kLossJoinRows - 1) / kLossJoinRows);
        hipLaunchKernelGGL((loss_join_kernel<kLossJoinRows, false>), dim3(grid), dim3(256), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_loss_mean(const LossRows &r, int64_t M, float *mean, hipStream_t stream) {
    hipLaunchKernelGGL(loss_mean_kernel, dim3(1), dim3(256), 0, stream, r, M, mean);
    return hipGetLastError();
}

}  // namespace nf4k
