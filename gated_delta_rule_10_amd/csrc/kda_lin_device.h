// Device pieces shared by the linear-attention kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_device.h"
#include "kda_lin_internal.h"

namespace kda {

// Log decays below this count as this where they are summed: e^-110 is 0 in fp32, and sums of
// them stay finite, so that differences of sums across a -infinity are not NaN. (A NaN stays one.)
constexpr float kLowestDecay = -110.f;
__device__ __forceinline__ float log_decay(float g) { return g < kLowestDecay ? kLowestDecay : g; }

// Slot of sequence n's state, -1 if it holds nothing.
__device__ __forceinline__ int slot_of(const LinArgs &a, int n) {
    if (!a.slots) return n;
    const int s = ld_meta(a.slots, n);
    return s >= 0 && s < a.nslots ? s : -1;
}

// What a chunk's tokens keep, in LDS. With G the inclusive sums of log2 e^g over the chunk: G in two
// fp32 parts (so that differences, which may be small between large sums, are right to fp32), e^G,
// and e^(G of the last token - G).
struct Decays {
    const float *hi, *lo, *grown, *left;
};

// fp32 to an output element: bf16 to nearest even, a NaN stays one
__device__ __forceinline__ void store_out(float *p, float x) { *p = x; }
__device__ __forceinline__ void store_out(bf16_t *p, float x) {
    *reinterpret_cast<__bf16 *>(p) = static_cast<__bf16>(x);
}

}  // namespace kda
