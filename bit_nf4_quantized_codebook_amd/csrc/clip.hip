// The global norm of a list of gradient tensors, and all of them scaled to a largest norm (gfx950):
//   norm = sqrt(sum over all tensors of g^2);   out = norm > max_norm ? g (max_norm / norm) : g
//
// Two passes over the gradients, both streams.  The list is cut into chunks of CHUNK elements, numbered
// through; a workgroup takes a contiguous run of chunks and finds its first tensor by bisection.  Squares
// are summed in float64: nothing overflows or vanishes, whatever the gradients' size, and the VALU has the time
// (the stream leaves room for some 60 operations an element).  Each workgroup leaves one partial sum; the
// second pass sums them again in every workgroup, in a fixed order, which is cheaper than a launch between.
//
// The list itself (pointers, sizes) comes in kernel arguments, LIST entries a launch, and is written to the
// workspace for the two passes.

#include "common.h"
#include "clip.h"

namespace nf4k {

namespace {

constexpr int CHUNK = 8192;      // elements; a workgroup's threads take 32 each
constexpr int NT = 256;

struct ClipBatch {
    ClipEntry e[kClipList];
    int32_t first, n;
};

__global__ __launch_bounds__(64) void clip_list_kernel(ClipBatch b, ClipEntry *list) {
    for (int i = threadIdx.x; i < b.n; i += 64) list[b.first + i] = b.e[i];
}

// the tensor that holds chunk c
__device__ __forceinline__ int find(const ClipEntry *list, int n, int64_t c) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list[mid].chunk <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// f(element index, value) over a chunk of a tensor
template <class T, class F>
__device__ __forceinline__ void each(const void *base, int64_t i0, int64_t i1, F f) {
    for (int64_t i = i0 + threadIdx.x; i < i1; i += NT) f(i, reinterpret_cast<const T *>(base)[i]);
}

__device__ __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float value(float x) { return x; }

__global__ __launch_bounds__(NT) void clip_norm_kernel(const ClipEntry *__restrict__ list, int n, int64_t chunks,
                                                       double *__restrict__ part) {
    __shared__ double sh[NT];
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double s = 0.0;
    if (c0 < c1) {
        int t = find(list, n, c0);
        for (int64_t c = c0; c < c1; ++c) {
            while (t + 1 < n && list[t + 1].chunk <= c) ++t;
            const ClipEntry e = list[t];
            const int64_t i0 = (c - e.chunk) * CHUNK, i1 = min(i0 + CHUNK, e.numel);
            auto add = [&](int64_t, auto x) {
                const double v = (double)value(x);
                s = __builtin_fma(v, v, s);
            };
            if (e.f32) each<float>(e.g, i0, i1, add);
            else each<uint16_t>(e.g, i0, i1, add);
        }
    }
    sh[threadIdx.x] = s;
    __syncthreads();
    for (int d = NT / 2; d > 0; d >>= 1) {
        if ((int)threadIdx.x < d) sh[threadIdx.x] += sh[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) part[blockIdx.x] = sh[0];
}

__global__ __launch_bounds__(NT) void clip_scale_kernel(const ClipEntry *__restrict__ list, int n, int64_t chunks,
                                                        const double *__restrict__ part, int nparts, float max_norm,
                                                        float *__restrict__ norm_out) {
    __shared__ double sh[NT];
    double s = 0.0;
    for (int i = threadIdx.x; i < nparts; i += NT) s += part[i];
    sh[threadIdx.x] = s;
    __syncthreads();
    for (int d = NT / 2; d > 0; d >>= 1) {
        if ((int)threadIdx.x < d) sh[threadIdx.x] += sh[threadIdx.x + d];
        __syncthreads();
    }
    const double norm = __builtin_sqrt(sh[0]);
    if (blockIdx.x == 0 && threadIdx.x == 0) norm_out[0] = (float)norm;
    // a norm that is not finite, as the caller sees it in float32, leaves the gradients as they are
    const bool clip = norm > (double)max_norm && (float)norm < __builtin_inff();
    // the factor stays in float64: it may be far below float32's range where the products are not
    const double f = clip ? (double)max_norm / norm : 1.0;
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    if (c0 >= c1) return;
    int t = find(list, n, c0);
    for (int64_t c = c0; c < c1; ++c) {
        while (t + 1 < n && list[t + 1].chunk <= c) ++t;
        const ClipEntry e = list[t];
        if (!clip && e.out == e.g) continue;
        const int64_t i0 = (c - e.chunk) * CHUNK, i1 = min(i0 + CHUNK, e.numel);
        if (e.f32) each<float>(e.g, i0, i1, [&](int64_t i, float x) { reinterpret_cast<float *>(e.out)[i] = clip ? (float)((double)x * f) : x; });
        else
            each<uint16_t>(e.g, i0, i1, [&](int64_t i, uint16_t x) {
                reinterpret_cast<uint16_t *>(e.out)[i] = clip ? (uint16_t)f32_to_bf16((float)((double)bf16_to_f32(x) * f)) : x;
            });
    }
}

}  // namespace

int64_t clip_chunks(int64_t numel) { return (numel + CHUNK - 1) / CHUNK; }

hipError_t launch_clip(ClipEntry (*get)(const void *, int32_t), const void *ctx, int32_t n, float max_norm, float *norm,
                       ClipEntry *list, double *part, hipStream_t stream) {
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; i += kClipList) {
        ClipBatch b{};
        b.first = i;
        b.n = n - i < kClipList ? n - i : kClipList;
        for (int k = 0; k < b.n; ++k) {
            b.e[k] = get(ctx, i + k);
            b.e[k].chunk = chunks;
            chunks += clip_chunks(b.e[k].numel);
        }
        hipLaunchKernelGGL(clip_list_kernel, dim3(1), dim3(64), 0, stream, b, list);
        const hipError_t rc = hipGetLastError();
        if (rc != hipSuccess) return rc;
    }
    const int grid = (int)(chunks < kClipParts ? (chunks > 0 ? chunks : 1) : kClipParts);
    hipLaunchKernelGGL(clip_norm_kernel, dim3(grid), dim3(NT), 0, stream, list, n, chunks, part);
    hipError_t rc = hipGetLastError();
    if (rc != hipSuccess) return rc;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(grid), dim3(NT), 0, stream, list, n, chunks, part, grid, max_norm, norm);
    return hipGetLastError();
}

}  // namespace nf4k
