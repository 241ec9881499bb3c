// The global norm of a list of gradient tensors, and all of them scaled to a largest norm (gfx950):
//   norm = sqrt(sum over all tensors of g^2);   out = norm > max_norm ? g (max_norm / norm) : g
//
// Two passes over the gradients, both streams.  The list is cut into chunks of CHUNK elements, numbered
// through; a workgroup takes a contiguous run of chunks and looks for its first tensor.  Squares
// are summed in float64: nothing overflows or vanishes, whatever the gradients' size, and the VALU has the time
// (the stream leaves room for some 60 operations an element).  Each workgroup leaves one partial sum; the
// second pass sums them again in every workgroup, in a fixed order, which is cheaper than a launch between.
//
// The second pass walks backwards, since what the first read last still lies in the memory-side cache, and both its loads
// and its stores are nontemporal, so as not to drive the rest out.
//
// Bound by HBM: 224 adapter pairs of the 7B width in bf16 (320 MB) take 160 us, where reading them twice and writing
// them once at a copy's 5.0 TB/s takes 192; 217 us with plain loads and stores and 8192 elements a chunk, 167 walking
// forwards, 185 with nontemporal loads in the first pass too.  61 mixed pairs of odd sizes 29.5 us: 33
// with the first tensor found by bisection and each chunk's entry read again.  One pair takes 8 us of kernels, 11 as a
// call.
//
// The list (pointers, sizes, first chunks) is a table in device memory that the caller keeps with the gradients: made from 448
// tensors by the Python binding it costs 1.0 ms of the host, six calls' time.

#include "common.h"
#include "clip.h"

namespace nf4k {

namespace {

constexpr int CHUNK = kClipChunk;      // a workgroup's threads take 16 elements each
constexpr int NT = 256;

__device__ __forceinline__ int64_t first(const ClipEntry &e) { return e.chunk >> 1; }

// The tensor that holds chunk c: the last one that begins at or before it (tensors without elements have no chunk).  The
// whole workgroup looks, each thread at one of NT places: a load's latency for 256 tensors, two for 65536.
__device__ __forceinline__ int find(const ClipEntry *list, int n, int64_t c) {
    int lo = 0;
    while (n > 1) {
        const int step = (n + NT - 1) / NT, i = (int)threadIdx.x * step;
        const int k = __syncthreads_count(i < n && first(list[lo + i]) <= c) - 1;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

__device__ __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float rounded(float x, float) { return x; }
__device__ __forceinline__ uint16_t rounded(float x, uint16_t) { return (uint16_t)f32_to_bf16(x); }

// A chunk's elements as 16-byte vectors: VEC of them to a vector, PER vectors to a thread, whose loads are all
// issued before the first is used.
template <class T>
struct Vec {
    static constexpr int VEC = 16 / (int)sizeof(T), PER = CHUNK / NT / VEC;
    typedef T type __attribute__((ext_vector_type(VEC)));
};

// first elements of a chunk before its address is a multiple of 16 bytes
template <class T>
__device__ __forceinline__ int head(const T *p) {
    return (int)(((16 - ((uintptr_t)p & 15u)) & 15u) / sizeof(T));
}

template <class T>
__device__ __forceinline__ double squares(const T *p, int n) {
    typedef typename Vec<T>::type V;
    constexpr int VEC = Vec<T>::VEC, PER = Vec<T>::PER;
    const int tid = threadIdx.x;
    double s = 0.0;
    auto add = [&](T x) {
        const double v = (double)value(x);
        s = __builtin_fma(v, v, s);
    };
    const int h = min(head(p), n), nv = (n - h) / VEC;
    const V *q = reinterpret_cast<const V *>(p + h);
    V v[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) v[u] = u * NT + tid < nv ? q[u * NT + tid] : (V)(T)0;
    if (tid < h) add(p[tid]);
    const int rest = h + nv * VEC + tid;
    if (rest < n) add(p[rest]);
#pragma unroll
    for (int u = 0; u < PER; ++u)
#pragma unroll
        for (int k = 0; k < VEC; ++k) add(v[u][k]);
    return s;
}

template <class T>
__device__ __forceinline__ void scale(const T *p, T *o, int n, bool clip, double f) {
    typedef typename Vec<T>::type V;
    constexpr int VEC = Vec<T>::VEC, PER = Vec<T>::PER;
    const int tid = threadIdx.x;
    auto to = [&](T x) { return clip ? rounded((float)((double)value(x) * f), x) : x; };
    int h = 0, nv = 0;
    // where the two addresses differ modulo 16 bytes, element by element
    if ((((uintptr_t)p ^ (uintptr_t)o) & 15u) == 0) {
        h = min(head(p), n);
        nv = (n - h) / VEC;
        const V *q = reinterpret_cast<const V *>(p + h);
        V *w = reinterpret_cast<V *>(o + h);
        V v[PER];
#pragma unroll
        for (int u = 0; u < PER; ++u)
            if (u * NT + tid < nv) v[u] = __builtin_nontemporal_load(&q[u * NT + tid]);
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            if (u * NT + tid >= nv) continue;
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[u][k] = to(v[u][k]);
            __builtin_nontemporal_store(v[u], &w[u * NT + tid]);
        }
        if (tid < h) o[tid] = to(p[tid]);
    }
    for (int i = h + nv * VEC + tid; i < n; i += NT) o[i] = to(p[i]);
}

// the workgroup's sum, in every thread
__device__ __forceinline__ double over_block(double s) {
    __shared__ double sh[NT / 64];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

__global__ __launch_bounds__(NT) void clip_norm_kernel(const ClipEntry *__restrict__ list, int n, int64_t chunks,
                                                       double *__restrict__ part) {
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    double s = 0.0;
    if (c0 < c1) {
        int t = find(list, n, c0);
        ClipEntry e = list[t];
        auto next = [&]() { return t + 1 < n ? first(list[t + 1]) : chunks; };
        int64_t end = next();
        for (int64_t c = c0; c < c1; ++c) {
            while (c >= end) {
                e = list[++t];
                end = next();
            }
            const int64_t i0 = (c - first(e)) * CHUNK, i1 = min(i0 + CHUNK, e.numel);
            if (e.chunk & 1) s += squares(reinterpret_cast<const float *>(e.g) + i0, (int)(i1 - i0));
            else s += squares(reinterpret_cast<const uint16_t *>(e.g) + i0, (int)(i1 - i0));
        }
    }
    s = over_block(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(NT) void clip_scale_kernel(const ClipEntry *__restrict__ list, int n, int64_t chunks,
                                                        const double *__restrict__ part, int nparts, float max_norm,
                                                        float *__restrict__ norm_out) {
    const int64_t c0 = chunks * blockIdx.x / gridDim.x, c1 = chunks * (blockIdx.x + 1) / gridDim.x;
    // the partials and the workgroup's tensor are on their way together
    double p[kClipParts / NT], s = 0.0;
#pragma unroll
    for (int i = 0; i < kClipParts / NT; ++i) p[i] = i * NT + (int)threadIdx.x < nparts ? part[i * NT + threadIdx.x] : 0.0;
    int t = c0 < c1 ? find(list, n, c1 - 1) : 0;
#pragma unroll
    for (int i = 0; i < kClipParts / NT; ++i) s += p[i];
    const double norm = __builtin_sqrt(over_block(s));
    if (blockIdx.x == 0 && threadIdx.x == 0) norm_out[0] = (float)norm;
    // a norm that is not finite, as the caller sees it in float32, leaves the gradients as they are
    const bool clip = norm > (double)max_norm && (float)norm < __builtin_inff();
    // the factor stays in float64: it may be far below float32's range where the products are not
    const double f = clip ? (double)max_norm / norm : 1.0;
    if (c0 >= c1) return;
    ClipEntry e = list[t];
    for (int64_t c = c1 - 1; c >= c0; --c) {
        while (first(e) > c) e = list[--t];
        if (!clip && e.out == e.g) continue;
        const int64_t i0 = (c - first(e)) * CHUNK, i1 = min(i0 + CHUNK, e.numel);
        if (e.chunk & 1) scale(reinterpret_cast<const float *>(e.g) + i0, reinterpret_cast<float *>(e.out) + i0, (int)(i1 - i0), clip, f);
        else scale(reinterpret_cast<const uint16_t *>(e.g) + i0, reinterpret_cast<uint16_t *>(e.out) + i0, (int)(i1 - i0), clip, f);
    }
}

}  // namespace

hipError_t launch_clip(const ClipEntry *table, int32_t n, int64_t chunks, float max_norm, float *norm, double *part,
                       hipStream_t stream) {
    const int grid = (int)(chunks < kClipParts ? (chunks > 0 ? chunks : 1) : kClipParts);
    hipLaunchKernelGGL(clip_norm_kernel, dim3(grid), dim3(NT), 0, stream, table, n, chunks, part);
    const hipError_t rc = hipGetLastError();
    if (rc != hipSuccess) return rc;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(grid), dim3(NT), 0, stream, table, n, chunks, part, grid, max_norm, norm);
    return hipGetLastError();
}

}  // namespace nf4k
