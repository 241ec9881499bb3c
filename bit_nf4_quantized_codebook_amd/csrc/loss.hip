// What stands around the two products of the loss over the vocabulary (gfx950): the live rows, the sums over
// the vocabulary's tiles, the losses, and dX from its partials.  With d = ln sum_{v != y} e^z_v - z_y (the
// log odds against the label y):
//   loss = ln(1 + e^d) = max(d, 0) + ln(1 + e^-|d|),   1 - p_y = 1 / (1 + e^-d)
//   dX = g (sum_{v != y} p_v W_v - (1 - p_y) W_y)
// Nothing here subtracts two large numbers: a label that is nearly certain keeps a loss and a gradient of full
// precision.

#include "common.h"
#include "loss.h"

namespace nf4k {

namespace {

constexpr int PREP = 1024;

// Workgroup 0: the live rows, in order.  The others: loss and dX of the rest set to zero.
__global__ __launch_bounds__(PREP) void loss_prep_kernel(const int64_t *__restrict__ labels, int64_t M, int64_t V, int64_t K,
                                                         LossRows r, float *__restrict__ loss, uint16_t *__restrict__ dX) {
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        for (int64_t m = blockIdx.x - 1; m < M; m += gridDim.x - 1) {
            if (labels[m] >= 0) continue;
            if (tid == 0) loss[m] = 0.0f;
            if (dX)
                for (int64_t k = tid * 8; k < K; k += PREP * 8) *reinterpret_cast<u32x4 *>(dX + m * K + k) = u32x4{0, 0, 0, 0};
        }
        return;
    }
    __shared__ int scan[PREP];
    const int64_t per = (M + PREP - 1) / PREP, m0 = tid * per, m1 = min(m0 + per, M);
    int n = 0;
    for (int64_t m = m0; m < m1; ++m) n += labels[m] >= 0;
    scan[tid] = n;
    __syncthreads();
    for (int d = 1; d < PREP; d <<= 1) {
        const int v = tid >= d ? scan[tid - d] : 0;
        __syncthreads();
        scan[tid] += v;
        __syncthreads();
    }
    if (tid == PREP - 1) {
        r.count[0] = scan[tid];
        r.count[1] = 0;
    }
    int at = scan[tid] - n;
    for (int64_t m = m0; m < m1; ++m) {
        const int64_t l = labels[m];
        if (l < 0) continue;
        r.row[at] = (int32_t)m;
        r.label[at] = l < V ? (int32_t)l : -1;
        r.zl[at] = __builtin_nanf("");      // a label in the vocabulary writes its logit over it
        ++at;
    }
}

constexpr int JR = 32, JS = 8;      // rows of a workgroup, and threads over the tiles of a row

__global__ __launch_bounds__(JR * JS) void loss_join_kernel(LossJoin g) {
    __shared__ float part[JS][JR];
    __shared__ double total[JR * JS];
    __shared__ bool final_wg;
    const int count = g.r.count[0];
    const int tid = threadIdx.x, lr = tid % JR, slice = tid / JR;
    const int row = blockIdx.x * JR + lr;
    const bool live = row < count;
    const int nwg = (count + JR - 1) / JR;
    if ((int)blockIdx.x >= nwg && !(g.last && blockIdx.x == 0)) return;

    // the new reference: the old one unless a tile went past it
    const float NEG = -__builtin_inff();
    const float c_old = g.c_in && live ? g.c_in[row] : NEG;
    float c = c_old;
    if (live)
        for (int t = slice; t < g.ntile; t += JS) c = fmaxf(c, g.tref[(int64_t)t * g.Mp + row]);
    part[slice][lr] = c;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < JS; ++s) c = fmaxf(c, part[s][lr]);
    __syncthreads();
    float sum = 0.0f;
    if (live)
        for (int t = slice; t < g.ntile; t += JS) {
            const int64_t o = (int64_t)t * g.Mp + row;
            sum += g.tsum[o] * __builtin_amdgcn_exp2f(g.tref[o] - c);
        }
    part[slice][lr] = sum;
    __syncthreads();
    if (slice == 0 && live) {
        float S = g.c_in ? g.r.S[row] * __builtin_amdgcn_exp2f(c_old - c) : 0.0f;
#pragma unroll
        for (int s = 0; s < JS; ++s) S += part[s][lr];
        g.r.S[row] = S;
        g.c_out[row] = c;
        if (g.last) {
            const float zl = g.r.zl[row];
            // ln S + (c - zl) ln 2
            const float d = (log2f(S) + (c - zl)) * kLn2;
            const int32_t m = g.r.row[row];
            g.loss[m] = fmaxf(d, 0.0f) + log1pf(expf(-fabsf(d)));
            if (g.grad) {
                const float w = g.dloss ? g.dloss[m] : 1.0f / (float)count;
                g.r.a[row] = w / (S + __builtin_amdgcn_exp2f(zl - c));
                g.r.b[row] = w / (1.0f + expf(-d));
            }
        }
    }
    if (!g.last) return;
    // the workgroup that ends last sums the losses, in a fixed order
    __threadfence();
    __syncthreads();
    if (tid == 0) final_wg = atomicAdd(&g.r.count[1], 1) + 1 == (nwg > 0 ? nwg : 1);
    __syncthreads();
    if (!final_wg) return;
    __threadfence();
    double s = 0.0;
    for (int i = tid; i < count; i += JR * JS)
        s += (double)__hip_atomic_load(&g.loss[g.r.row[i]], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    total[tid] = s;
    __syncthreads();
    for (int d = JR * JS / 2; d > 0; d >>= 1) {
        if (tid < d) total[tid] += total[tid + d];
        __syncthreads();
    }
    if (tid == 0) g.mean[0] = count ? (float)(total[0] / count) : 0.0f;
}

// One workgroup for 256 rows and one tile of the vocabulary: four blocks of P.
__global__ __launch_bounds__(256) void loss_rescale_kernel(uint16_t *__restrict__ P, const float *__restrict__ tref,
                                                           const float *__restrict__ c, const int32_t *__restrict__ cnt,
                                                           int32_t Mp, int32_t ntile) {
    __shared__ float f[LT];
    const int count = cnt[0], tid = threadIdx.x;
    const int tm = blockIdx.x / ntile, t = blockIdx.x % ntile;
    if (tm * LT >= count) return;
    const int row = tm * LT + tid;
    const float from = row < count ? tref[(int64_t)t * Mp + row] : 0.0f, to = row < count ? c[row] : 0.0f;
    f[tid] = __builtin_amdgcn_exp2f(from - to);
    if (!__syncthreads_or(!(from == to))) return;
    uint16_t *base = P + ((int64_t)tm * ntile + t) * 4 * LBLOCK;
    for (int i = tid; i < 4 * LBLOCK / 8; i += 256) {
        const float s = f[(i >> 3) & (LT - 1)];     // 8 chunks a row, 256 rows a block
        u32x4 v = reinterpret_cast<u32x4 *>(base)[i];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[k] = pack_bf16x2(bf16_to_f32(v[k] & 0xFFFFu) * s, __uint_as_float(v[k] & 0xFFFF0000u) * s);
        reinterpret_cast<u32x4 *>(base)[i] = v;
    }
}

__global__ __launch_bounds__(256) void loss_fold_kernel(LossFold g) {
    const int count = g.r.count[0];
    const int ntm = (count + LT - 1) / LT, ntn = (int)((g.K + LT - 1) / LT), tiles = ntm * ntn;
    const LossSplit sp = loss_split(tiles, g.steps);
    const int k8 = (int)(g.K >> 3);
    const int64_t n = (int64_t)count * k8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int row = (int)(i / k8), k = (int)(i % k8) * 8;
        const float *p = g.part + ((int64_t)(row / LT) * ntn + k / LT) * (LT * LT) + (row % LT) * LT + k % LT;
        f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
        if (g.c_old) {
            const float s = __builtin_amdgcn_exp2f(g.c_old[row] - g.c[row]);
            const f32x4 *o = reinterpret_cast<const f32x4 *>(g.sum32 + (int64_t)row * g.K + k);
            lo = o[0] * s;
            hi = o[1] * s;
        }
        for (int s = 0; s < sp.ks; ++s) {
            const f32x4 *q = reinterpret_cast<const f32x4 *>(p + (int64_t)s * tiles * (LT * LT));
            lo += q[0];
            hi += q[1];
        }
        if (!g.dX) {
            f32x4 *o = reinterpret_cast<f32x4 *>(g.sum32 + (int64_t)row * g.K + k);
            o[0] = lo;
            o[1] = hi;
            continue;
        }
        const float a = g.r.a[row], b = g.r.b[row];
        const int32_t lab = g.r.label[row];
        const u32x4 w = *reinterpret_cast<const u32x4 *>(g.W + (int64_t)(lab < 0 ? 0 : lab) * g.K + k);
        u32x4 out;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = j < 2 ? lo[2 * j] : hi[2 * j - 4], y = j < 2 ? lo[2 * j + 1] : hi[2 * j - 3];
            out[j] = pack_bf16x2(a * x - b * bf16_to_f32(w[j] & 0xFFFFu), a * y - b * __uint_as_float(w[j] & 0xFFFF0000u));
        }
        *reinterpret_cast<u32x4 *>(g.dX + (int64_t)g.r.row[row] * g.K + k) = out;
    }
}

}  // namespace

hipError_t launch_loss_prep(const int64_t *labels, int64_t M, int64_t V, int64_t K, const LossRows &r, float *loss,
                            uint16_t *dX, hipStream_t stream) {
    const uint32_t rest = (uint32_t)(M < 2048 ? M : 2048);
    hipLaunchKernelGGL(loss_prep_kernel, dim3(1 + rest), dim3(PREP), 0, stream, labels, M, V, K, r, loss, dX);
    return hipGetLastError();
}

hipError_t launch_loss_join(const LossJoin &a, hipStream_t stream) {
    hipLaunchKernelGGL(loss_join_kernel, dim3((uint32_t)((a.M + JR - 1) / JR)), dim3(JR * JS), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_loss_rescale(uint16_t *P, const float *tref, const float *c, const int32_t *count, int32_t Mp,
                               int32_t ntile, hipStream_t stream) {
    hipLaunchKernelGGL(loss_rescale_kernel, dim3((uint32_t)(Mp / LT) * (uint32_t)ntile), dim3(256), 0, stream, P, tref, c,
                       count, Mp, ntile);
    return hipGetLastError();
}

hipError_t launch_loss_fold(const LossFold &a, hipStream_t stream) {
    const int64_t blocks = ((int64_t)a.Mp * (a.K >> 3) + 255) / 256;
    hipLaunchKernelGGL(loss_fold_kernel, dim3((uint32_t)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nf4k
