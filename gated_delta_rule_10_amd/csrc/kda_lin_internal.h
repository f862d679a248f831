// Internal launch interface of the linear-attention entry points
// (include/kda_lin.h) between their C-ABI layer (kda_lin_api.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_lin.h"

namespace kda {

struct LinArgs {
    const void *q, *k, *v;      // rows of qs / ks / vs elements, in_dtype
    const float *g;             // log decay
    int64_t qs, ks, vs, gs;     // token strides in elements
    const int32_t *cu;          // [N + 1] (prompts only)
    const float *s0;            // initial states or nullptr (prompts only)
    float *sT;                  // final states or nullptr; the cache of single tokens
    const int32_t *slots;       // of the states, [N], or nullptr
    void *o;                    // [T, H, V] out_dtype
    void *ws;
    int32_t N, T, H, Hk, K, V, nslots;
    float scale;
    kda_dtype_t in_dtype, out_dtype;
};

// Threads of a workgroup of single tokens.
constexpr int kLinDecodeThreads = 1024;

hipError_t launch_lin_chunk(const LinArgs &a, hipStream_t stream);
hipError_t launch_lin_decode(const LinArgs &a, hipStream_t stream);  // N sequences of one token

// Workspace bytes of a prompt call on the current device.
size_t lin_chunk_workspace(int32_t N, int32_t T, int32_t H, int32_t K, int32_t V, kda_dtype_t in_dtype);

}  // namespace kda
