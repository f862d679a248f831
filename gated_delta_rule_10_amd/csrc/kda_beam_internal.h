// Internal launch interface of the beam-search entry points (include/kda_beam.h)
// between their C-ABI layer (kda_beam_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_beam.h"

namespace kda {

struct SelectArgs {
    const void *logits;
    int64_t stride;
    const float *scores;
    const uint8_t *done;  // or nullptr
    int32_t done_token, N, W, V, K;
    kda_dtype_t dtype;
    float *out_scores;
    int32_t *out_parent, *out_token;
    void *ws;
};

struct ReorderArgs {
    char *states;
    int64_t layer_stride, slot_bytes;
    const int32_t *slots, *parent;
    int32_t *slots_out;
    int32_t layers, nslots, N, W;
};

hipError_t launch_beam_select(const SelectArgs &a, hipStream_t stream);
hipError_t launch_state_reorder(const ReorderArgs &a, hipStream_t stream);

// Workspace bytes of a selection on the current device.
size_t beam_select_workspace(int32_t N, int32_t W, int32_t V);

}  // namespace kda
