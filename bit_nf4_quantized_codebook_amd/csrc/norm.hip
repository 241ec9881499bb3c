// Norm glue between two blocks of a decoder layer (gfx950), not a step of the method:
//   n = w_post B / rms(B);  R' = alpha R + beta gate n;  H = w_pre R' / rms(R')
// with rms(x) = sqrt(mean(x^2) + eps), and the backward of it.  float32 arithmetic throughout; H is
// taken from R' as computed, before R' is rounded to its type.
//
// Both directions are bound by HBM: a workgroup holds one row in registers (each thread 8-element
// pieces), so every element is read and written once, and the row's sums cross waves through LDS.
// Backward: a workgroup takes a run of rows and keeps the sums for dw_pre, dw_post and dgate of its
// columns in registers; at the end of the run (or of a gate row) it writes them as float32 partials,
// which a second launch sums in a fixed order.
//
// Measured (bytes read and written once, against a large copy's 5.2 TB/s): forward 39 us at 4096 x 4096 with
// a float32 residual (201 MB, 5.1 TB/s); backward 52 us at 4096 x 4096 bf16 (201 MB; 44 the rows, 6 the sum)
// and 35 us at 1001 x 8192 float32 (148 MB).  Above 8192 columns a thread holds four pieces and no row ahead:
// 2048 x 16384 116 us in bf16 (403 MB, 3.5 TB/s).

#include "common.h"
#include "int8.h"
#include "launch.h"

namespace nf4k {

namespace {

typedef float f32v4 __attribute__((ext_vector_type(4)));

// The forward reads the residual past the caches (43.2 -> 39.2 us at 4096 x 4096 float32); in the
// backward that cost 1.5 to 6 us a call, and its loads stay ordinary.
template <bool F32>
__device__ __forceinline__ void load_res(const void *x, int64_t e, float f[8]) {
    Raw8<F32> r;
    r.template load<true>(x, e);
    r.floats(f);
}
// The large outputs are stored past the caches (nontemporal): they are written whole and far larger
// than an L2, and a launch's end otherwise waits for their write-back (forward, 4096 x 4096 float32
// residual: 46.2 -> 42.5 us a call; backward, 1001 x 8192: 37.9 -> 35.1 us).
template <bool F32>
__device__ __forceinline__ void store_res(void *x, int64_t e, const float f[8]) {
    if (F32) {
        f32v4 *p = reinterpret_cast<f32v4 *>(reinterpret_cast<float *>(x) + e);
        __builtin_nontemporal_store(f32v4{f[0], f[1], f[2], f[3]}, p);
        __builtin_nontemporal_store(f32v4{f[4], f[5], f[6], f[7]}, p + 1);
    } else {
        __builtin_nontemporal_store(pack8_bf16(f), reinterpret_cast<u32x4 *>(reinterpret_cast<uint16_t *>(x) + e));
    }
}
// partial sums: read again by the next launch
__device__ __forceinline__ void store_sum(float *p, const float f[8]) {
    reinterpret_cast<f32v4 *>(p)[0] = f32v4{f[0], f[1], f[2], f[3]};
    reinterpret_cast<f32v4 *>(p)[1] = f32v4{f[4], f[5], f[6], f[7]};
}
__device__ __forceinline__ u32x4 load_p(const uint16_t *x, int64_t e) { return *reinterpret_cast<const u32x4 *>(x + e); }
__device__ __forceinline__ void load_b16(const uint16_t *x, int64_t e, float f[8]) { unpack8_bf16(load_p(x, e), f); }

// Sums of NV values over the workgroup; every thread gets them.  `slot` alternates between calls: a
// wave may write the next sums while another still reads these, but not the ones after.
template <int NT, int NV>
__device__ __forceinline__ void block_sum(float (&v)[NV], float (*red)[3][NT / 64], int slot) {
    constexpr int NW = NT / 64;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = wave_sum(v[i]);
    if (NW == 1) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) red[slot][i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) s += red[slot][i][w];
        v[i] = s;
    }
}

template <int NT, int V, bool F32>
__global__ __launch_bounds__(NT) void norm_fwd_kernel(NormArgs g) {
    __shared__ float red[2][3][NT / 64];
    __shared__ uint32_t redm[NT / 64];
    const int tid = threadIdx.x;
    const int64_t m = g.m0 + blockIdx.x, row = m * g.C;
    const float inv_c = 1.0f / (float)g.C;
    float r[V][8], b[V][8];
    bool in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * NT + tid) * 8;
        in[v] = c < g.C;
#pragma unroll
        for (int k = 0; k < 8; ++k) r[v][k] = b[v][k] = 0.0f;
        if (in[v]) {
            load_res<F32>(g.R, row + c, r[v]);
            if (g.B) load_b16(g.B, row + c, b[v]);
        }
    }
    if (g.B) {
        float ib = 1.0f;
        if (g.w_post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int k = 0; k < 8; ++k) s[0] = __builtin_fmaf(b[v][k], b[v][k], s[0]);
            block_sum<NT, 1>(s, red, 0);
            ib = 1.0f / sqrtf(s[0] * inv_c + g.eps);
        }
        const int64_t grow = g.gate ? (m / g.gate_tokens) * g.C : 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * NT + tid) * 8;
            if (!in[v]) continue;
            float w[8], gt[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = gt[k] = 1.0f;
            if (g.w_post) load_b16(g.w_post, c, w);
            if (g.gate) load_b16(g.gate, grow + c, gt);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                r[v][k] = __builtin_fmaf(g.beta * gt[k], b[v][k] * ib * w[k], g.alpha * r[v][k]);
            store_res<F32>(g.R_out, row + c, r[v]);
        }
    }
    if (!g.w_pre) return;
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[0] = __builtin_fmaf(r[v][k], r[v][k], s[0]);
    block_sum<NT, 1>(s, red, 1);
    const float ir = 1.0f / sqrtf(s[0] * inv_c + g.eps);
    uint32_t amax = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * NT + tid) * 8;
        if (!in[v]) continue;
        float w[8];
        load_b16(g.w_pre, c, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[v][k] = r[v][k] * ir * w[k];
        const u32x4 h = pack8_bf16(r[v]);
        __builtin_nontemporal_store(h, reinterpret_cast<u32x4 *>(g.H + row + c));
        unpack8_bf16(h, r[v]);
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = max(amax, __float_as_uint(r[v][k]) & 0x7FFFFFFFu);
    }
    if (!g.Hq) return;
    amax = wave_max(amax);
    if (NT > 64) {
        if ((tid & 63) == 0) redm[tid >> 6] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) amax = max(amax, redm[w]);
    }
    const RowCode rc = row_code<false>(amax);
    if (tid == 0) g.Hs[m] = rc.scale;
    by_mode(rc, [&](auto mode) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * NT + tid) * 8;
            const uint2 o = codes8<decltype(mode)::value>(r[v], rc);
            if (in[v]) *reinterpret_cast<uint2 *>(g.Hq + row + c) = o;
        }
    });
}

// How the backward's rows are cut into runs, one workgroup each.  Without a gate (or with one row of
// it for all tokens) a run is `per` rows.  Gate rows of at least `per` tokens are cut into `cpg` runs
// each, so that a run has one gate row and its sum is a partial like the others'.  Shorter ones go
// `gpc` to a run, which writes their dgate itself.
struct NormRuns {
    int64_t T;          // tokens of a gate row (M without a gate)
    int64_t per;        // rows of a run
    int64_t cpg, gpc;   // runs per gate row (0: gate rows per run instead), gate rows per run
    int64_t n;          // runs
};

// The weights and the gate row stay in registers over a run, except with four pieces per thread: the
// row takes the registers, the weights are read again (from L2) for each row, and the sums for dw_pre
// and dw_post lie in LDS, every thread's own.
template <int NT, int V, bool F32>
__global__ __launch_bounds__(NT) void norm_bwd_kernel(NormArgs g, NormRuns q) {
    constexpr bool HOLD = V < 4;
    __shared__ float red[4][3][NT / 64];
    __shared__ f32v4 lsum[2][HOLD ? 1 : V * 2][HOLD ? 1 : NT];     // dw_pre's and dw_post's sums
    const int tid = threadIdx.x;
    const int64_t run = blockIdx.x;
    const float inv_c = 1.0f / (float)g.C;
    int64_t m0, m1;
    if (q.cpg) {
        const int64_t grp = run / q.cpg, j = run % q.cpg;
        m0 = grp * q.T + j * q.per;
        m1 = min(min(m0 + q.per, (grp + 1) * q.T), g.M);
    } else {
        m0 = run * q.per;
        m1 = min(m0 + q.per, g.M);
    }
    const u32x4 none = {0u, 0u, 0u, 0u}, ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    bool in[V];
    u32x4 hpre[HOLD ? V : 1], hpost[HOLD ? V : 1], hgate[HOLD ? V : 1];
    float a_pre[HOLD ? V : 1][8], a_post[HOLD ? V : 1][8], a_gate[V][8];
    // sum[which][v] += d
    auto add = [&](int which, int v, const float d[8]) {
        if (HOLD) {
            float *a = which ? a_post[HOLD ? v : 0] : a_pre[HOLD ? v : 0];
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] += d[k];
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32v4 &a = lsum[which][HOLD ? 0 : 2 * v + h][HOLD ? 0 : tid];
                a += f32v4{d[4 * h], d[4 * h + 1], d[4 * h + 2], d[4 * h + 3]};
            }
        }
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * NT + tid) * 8;
        in[v] = c < g.C;
        if (HOLD) {
            hpre[v] = in[v] && g.w_pre ? load_p(g.w_pre, c) : none;
            hpost[v] = in[v] && g.w_post ? load_p(g.w_post, c) : none;
            hgate[v] = ones;
#pragma unroll
            for (int k = 0; k < 8; ++k) a_pre[HOLD ? v : 0][k] = a_post[HOLD ? v : 0][k] = 0.0f;
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h) lsum[h & 1][HOLD ? 0 : 2 * v + (h >> 1)][HOLD ? 0 : tid] = f32v4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) a_gate[v][k] = 0.0f;
    }
    int64_t grow = 0, next_gate = m0;         // the gate row, and the token at which it changes
    auto pre = [&](int v, float f[8]) {
        if (HOLD) unpack8_bf16(hpre[v], f);
        else unpack8_bf16(g.w_pre && in[v] ? load_p(g.w_pre, (v * NT + tid) * 8) : none, f);
    };
    auto post = [&](int v, float f[8]) {
        if (HOLD) unpack8_bf16(hpost[v], f);
        else unpack8_bf16(g.w_post ? load_p(g.w_post, (v * NT + tid) * 8) : none, f);
    };
    auto gate = [&](int v, float f[8]) {
        if (HOLD) unpack8_bf16(hgate[v], f);
        else unpack8_bf16(g.gate ? load_p(g.gate, grow * g.C + (v * NT + tid) * 8) : ones, f);
    };
    // A row's four operands, loaded one row ahead where the registers allow it: the row's two sums over
    // the workgroup then run under the next row's loads.
    struct Row {
        Raw8<F32> r[V], t[V];
        u32x4 dh[V], b[V];
    };
    auto load = [&](int64_t m, Row &x) {
        const int64_t row = m * g.C;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t e = row + (v * NT + tid) * 8;
            x.r[v].zero();
            x.t[v].zero();
            x.dh[v] = x.b[v] = none;
            if (!in[v]) continue;
            if (g.dH) {
                x.r[v].load(g.R, e);
                x.dh[v] = load_p(g.dH, e);
            }
            if (g.dR_out) x.t[v].load(g.dR_out, e);
            if (g.B) x.b[v] = load_p(g.B, e);
        }
    };
    constexpr bool AHEAD = V < 4;
    Row cur, nxt;
    if (AHEAD && m0 < m1) load(m0, cur);
    for (int64_t m = m0; m < m1; ++m) {
        const int64_t row = m * g.C;
        if (AHEAD) load(m + 1 < m1 ? m + 1 : m, nxt);
        else load(m, cur);
        if (g.gate && m == next_gate) {
            grow = m / q.T;
            next_gate = (grow + 1) * q.T;
            if (HOLD) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (in[v]) hgate[v] = load_p(g.gate, grow * g.C + (v * NT + tid) * 8);
            }
        }
        float r[V][8], t[V][8];
        u32x4 dh[V], b[V];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            cur.r[v].floats(r[v]);
            cur.t[v].floats(t[v]);
            dh[v] = cur.dh[v];
            b[v] = cur.b[v];
            float w[8], d[8], x[8];
            pre(v, w);
            unpack8_bf16(dh[v], d);
            unpack8_bf16(b[v], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                s[0] = __builtin_fmaf(r[v][k], r[v][k], s[0]);
                s[1] = __builtin_fmaf(w[k] * d[k], r[v][k], s[1]);
                s[2] = __builtin_fmaf(x[k], x[k], s[2]);
            }
        }
        const int par = (int)((m - m0) & 1) * 2;
        block_sum<NT, 3>(s, red, par);
        const float ir = 1.0f / sqrtf(s[0] * inv_c + g.eps);
        const float ib = g.w_post ? 1.0f / sqrtf(s[2] * inv_c + g.eps) : 1.0f;
        // t = ir (w dH - xh mean(w dH xh)): no power of ir by itself, which would overflow where eps and
        // the row are tiny (and, times a sum of zero, give NaN)
        const float k1 = ir * (s[1] * inv_c);
        float s2[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!in[v]) continue;
            float w[8], d[8], x[8], o[8];
            pre(v, w);
            unpack8_bf16(dh[v], d);
            unpack8_bf16(b[v], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float xh = r[v][k] * ir;
                o[k] = d[k] * xh;
                t[v][k] += ir * (w[k] * d[k] - k1 * xh);
            }
            add(0, v, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o[k] = g.alpha * t[v][k];
            }
            store_res<F32>(g.dR, row + (v * NT + tid) * 8, o);
            if (!g.B) continue;
            gate(v, o);
            post(v, w);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float bh = x[k] * ib;
                a_gate[v][k] = __builtin_fmaf(t[v][k], g.w_post ? bh * w[k] : bh, a_gate[v][k]);
                t[v][k] *= g.beta * o[k];                                    // u
                o[k] = t[v][k] * bh;
                s2[0] = __builtin_fmaf(w[k] * t[v][k], x[k], s2[0]);
            }
            if (g.w_post) add(1, v, o);
        }
        if (g.dB) {
            float k2 = 0.0f;
            if (g.w_post) {
                block_sum<NT, 1>(s2, red, par + 1);
                k2 = ib * (s2[0] * inv_c);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!in[v]) continue;
                if (g.w_post) {
                    float w[8], x[8];
                    post(v, w);
                    unpack8_bf16(b[v], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) t[v][k] = ib * (w[k] * t[v][k] - k2 * (x[k] * ib));
                }
                __builtin_nontemporal_store(pack8_bf16(t[v]), reinterpret_cast<u32x4 *>(g.dB + row + (v * NT + tid) * 8));
            }
        }
        if (AHEAD) cur = nxt;
        if (!q.cpg && g.dgate && (m + 1 == next_gate || m + 1 == g.M)) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!in[v]) continue;
                float o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    o[k] = g.beta * a_gate[v][k];
                    a_gate[v][k] = 0.0f;
                }
                *reinterpret_cast<u32x4 *>(g.dgate + grow * g.C + (v * NT + tid) * 8) = pack8_bf16(o);
            }
        }
    }
    // partials: [3][runs][C]
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * NT + tid) * 8;
        if (!in[v]) continue;
        if (HOLD) {
            if (g.dw_pre) store_sum(g.P + run * g.C + c, a_pre[HOLD ? v : 0]);
            if (g.dw_post) store_sum(g.P + (q.n + run) * g.C + c, a_post[HOLD ? v : 0]);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (g.dw_pre) reinterpret_cast<f32v4 *>(g.P + run * g.C + c)[h] = lsum[0][HOLD ? 0 : 2 * v + h][HOLD ? 0 : tid];
                if (g.dw_post)
                    reinterpret_cast<f32v4 *>(g.P + (q.n + run) * g.C + c)[h] = lsum[1][HOLD ? 0 : 2 * v + h][HOLD ? 0 : tid];
            }
        }
        if (g.dgate && q.cpg) store_sum(g.P + (2 * q.n + run) * g.C + c, a_gate[v]);
    }
}

// Fixed-order sums of the partials: workgroup (x, y) takes 64 columns of output y (dw_pre, dw_post,
// then the gate rows).  Sixteen threads cover the columns, four each; the sixteen groups of them
// take every sixteenth run, and their sums are added in order.
__global__ __launch_bounds__(256) void norm_sum_kernel(NormArgs g, NormRuns q, int first_gate) {
    __shared__ f32v4 part[16][16];
    const int tid = threadIdx.x, lc = tid & 15, sl = tid >> 4;
    const int64_t c = (int64_t)blockIdx.x * 64 + lc * 4;
    const int y = blockIdx.y;
    const float *P = g.P;
    uint16_t *out;
    int64_t n = q.n;
    float sc = 1.0f;
    if (y >= first_gate) {
        const int64_t grp = y - first_gate;
        P += (2 * q.n + grp * q.cpg) * g.C;
        n = q.cpg;
        out = g.dgate + grp * g.C;
        sc = g.beta;
    } else if (y == 0 && g.dw_pre) {
        out = g.dw_pre;
    } else {
        P += q.n * g.C;
        out = g.dw_post;
    }
    f32v4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < g.C)
        for (int64_t i = sl; i < n; i += 16 * 8) {       // eight loads in flight, added in order
            f32v4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + 16 * u < n) v[u] = *reinterpret_cast<const f32v4 *>(P + (i + 16 * u) * g.C + c);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i + 16 * u < n) acc += v[u];
        }
    part[sl][lc] = acc;
    __syncthreads();
    if (sl == 0 && c < g.C) {
#pragma unroll
        for (int i = 1; i < 16; ++i) acc += part[i][lc];
        *reinterpret_cast<uint2 *>(out + c) = uint2{pack_bf16x2(sc * acc.x, sc * acc.y), pack_bf16x2(sc * acc.z, sc * acc.w)};
    }
}

// Runs aimed at: what the CUs hold at once in bf16 (eight waves with two or more pieces per thread, sixteen
// with one), but no fewer than eight rows each beyond the first 256, so that the partials stay a small
// part of the traffic.  Two things pass that count and cost a second round of workgroups:
//   - the float32 kernels with one piece take 130 to 136 registers, so that a CU holds twelve of their
//     waves: 8192 x 2048 74 us, against 51 in bf16 (302 and 201 MB);
//   - norm_runs cuts each gate row by itself: at 4096 x 4096 bf16, 512 tokens per gate row give 512 runs and
//     52 us, 500 give 567 and 71 us, 10 give 820 and 70 us.
int64_t norm_target(int64_t M, int64_t C) {
    const int64_t per_cu = C <= 512 ? 16 : (C <= 1024 ? 8 : (C <= 2048 ? 4 : (C <= 4096 ? 2 : 1)));
    const int64_t most = M / 8 > 256 ? M / 8 : 256;
    const int64_t runs = 256 * per_cu < most ? 256 * per_cu : most;
    return runs < M ? runs : M;
}

NormRuns norm_runs(int64_t M, int64_t C, int64_t gate_tokens) {
    NormRuns q;
    q.T = gate_tokens > 0 && gate_tokens < M ? gate_tokens : M;
    const int64_t runs = norm_target(M, C);
    q.per = (M + runs - 1) / runs;
    const int64_t groups = (M + q.T - 1) / q.T;
    if (q.T >= q.per) {
        q.cpg = (q.T + q.per - 1) / q.per;
        q.per = (q.T + q.cpg - 1) / q.cpg;
        q.gpc = 0;
        q.n = groups * q.cpg;
    } else {
        q.cpg = 0;
        q.gpc = q.per / q.T;
        q.per = q.gpc * q.T;
        q.n = (groups + q.gpc - 1) / q.gpc;
    }
    return q;
}

template <bool F32>
void fwd_any(const NormArgs &a, int64_t rows, hipStream_t s) {
    const dim3 gd((unsigned)rows);
    if (a.C <= 512) hipLaunchKernelGGL((norm_fwd_kernel<64, 1, F32>), gd, dim3(64), 0, s, a);
    else if (a.C <= 1024) hipLaunchKernelGGL((norm_fwd_kernel<128, 1, F32>), gd, dim3(128), 0, s, a);
    else if (a.C <= 2048) hipLaunchKernelGGL((norm_fwd_kernel<256, 1, F32>), gd, dim3(256), 0, s, a);
    else if (a.C <= 4096) hipLaunchKernelGGL((norm_fwd_kernel<256, 2, F32>), gd, dim3(256), 0, s, a);
    else if (a.C <= 8192) hipLaunchKernelGGL((norm_fwd_kernel<512, 2, F32>), gd, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<1024, 2, F32>), gd, dim3(1024), 0, s, a);
}
template <bool F32>
void bwd_any(const NormArgs &a, const NormRuns &q, hipStream_t s) {
    const dim3 gd((unsigned)q.n);
    if (a.C <= 512) hipLaunchKernelGGL((norm_bwd_kernel<64, 1, F32>), gd, dim3(64), 0, s, a, q);
    else if (a.C <= 1024) hipLaunchKernelGGL((norm_bwd_kernel<128, 1, F32>), gd, dim3(128), 0, s, a, q);
    else if (a.C <= 2048) hipLaunchKernelGGL((norm_bwd_kernel<256, 1, F32>), gd, dim3(256), 0, s, a, q);
    else if (a.C <= 4096) hipLaunchKernelGGL((norm_bwd_kernel<256, 2, F32>), gd, dim3(256), 0, s, a, q);
    else if (a.C <= 8192) hipLaunchKernelGGL((norm_bwd_kernel<512, 2, F32>), gd, dim3(512), 0, s, a, q);
    else hipLaunchKernelGGL((norm_bwd_kernel<512, 4, F32>), gd, dim3(512), 0, s, a, q);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs &a, hipStream_t stream) {
    NormArgs p = a;
    for (p.m0 = 0; p.m0 < a.M; p.m0 += kMaxRowGrid) {
        const int64_t rows = a.M - p.m0 < kMaxRowGrid ? a.M - p.m0 : kMaxRowGrid;
        if (a.f32) fwd_any<true>(p, rows, stream);
        else fwd_any<false>(p, rows, stream);
    }
    return hipGetLastError();
}

// Runs, whatever the gate: ceil(M / T) ceil(T / per) with T >= per is at most 2 M / per + 2.
size_t norm_bwd_ws(int64_t M, int64_t C) {
    return (size_t)(2 * norm_target(M, C) + 2) * 3 * C * 4;
}

hipError_t launch_norm_bwd(const NormArgs &a, hipStream_t stream) {
    const NormRuns q = norm_runs(a.M, a.C, a.gate ? a.gate_tokens : 0);
    if ((size_t)q.n * 3 * a.C * 4 > norm_bwd_ws(a.M, a.C)) return hipErrorInvalidValue;
    if (a.f32) bwd_any<true>(a, q, stream);
    else bwd_any<false>(a, q, stream);
    const int first_gate = (a.dw_pre ? 1 : 0) + (a.dw_post ? 1 : 0);
    const int64_t gates = a.dgate && q.cpg ? (a.M + q.T - 1) / q.T : 0;
    if (first_gate + gates > 0)
        hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.C + 63) / 64), (unsigned)(first_gate + gates)), dim3(256), 0,
                           stream, a, q, first_gate);
    return hipGetLastError();
}

}  // namespace nf4k
