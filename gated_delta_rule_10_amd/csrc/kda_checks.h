// Host-side checks and small helpers that the C-ABI layers of kda_attn.h,
// kda_lin.h and kda_beam.h share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <cstring>

#include "kda.h"

namespace kda {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool given(const void *p) { return p && aligned16(p); }
inline bool head_dim_ok(int32_t d) { return d == 64 || d == 128; }
inline bool dtype_valid(kda_dtype_t d) { return d == KDA_F32 || d == KDA_BF16; }
inline bool dtype_pair_ok(kda_dtype_t in, kda_dtype_t out) { return in == KDA_BF16 || out == KDA_F32; }

// whether two arrays (a null pointer is none) share bytes
inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

// token strides of q, k and v
inline bool stride_ok(int64_t stride, int64_t heads, int32_t d) {
    return stride >= heads * d && stride % 8 == 0 && stride <= (int64_t(1) << 24);
}

// A call's end: its launch status and, with KDA_DEBUG_SYNC=1 (read once per process), that of
// its work on `stream`.
inline hipError_t finish(hipError_t e, hipStream_t stream) {
    static const bool wait = [] {
        const char *x = std::getenv("KDA_DEBUG_SYNC");
        return x && std::strcmp(x, "1") == 0;
    }();
    if (e == hipSuccess && wait) e = hipStreamSynchronize(stream);
    if (e == hipSuccess && wait) e = hipGetLastError();
    return e;
}

}  // namespace kda
