// Gradient clipping over a list of tensors: launcher (clip.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4k {

struct ClipEntry {
    const void *g;
    void *out;           // may be g
    int64_t numel;
    int64_t chunk;       // chunks of the tensors before it
    int32_t f32, pad;
};
constexpr int kClipList = 96;        // entries of a launch that writes the list: 3840 bytes of arguments
constexpr int kClipParts = 2048;     // workgroups of a pass at most

int64_t clip_chunks(int64_t numel);
// get(i): entry i of the caller's list (its chunk field is filled here); list: device [n]; part: device
// [kClipParts]
hipError_t launch_clip(ClipEntry (*get)(const void *, int32_t), const void *ctx, int32_t n, float max_norm, float *norm,
                       ClipEntry *list, double *part, hipStream_t stream);

}  // namespace nf4k
