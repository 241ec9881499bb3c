// Gradient clipping over a list of tensors: its table and launcher (clip.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4k {

struct ClipEntry {
    const void *g;
    void *out;           // may be g
    int64_t numel;
    int64_t chunk;       // chunks of the tensors before it, times two; + 1: float32
};
constexpr int kClipChunk = 4096;     // elements
constexpr int kClipParts = 2048;     // workgroups of a pass at most, eight on each CU (224 pairs: 160 us, 173 with 1024, 163 with 4096)

// table: device [n]; part: device [kClipParts]
hipError_t launch_clip(const ClipEntry *table, int32_t n, int64_t chunks, float max_norm, float *norm, double *part,
                       hipStream_t stream);

}  // namespace nf4k
