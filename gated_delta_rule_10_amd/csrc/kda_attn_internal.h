// Internal launch interface of the attention entry points (include/kda_attn.h)
// between their C-ABI layer (kda_attn_api.cpp) and the HIP kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_attn.h"
#include "kda_internal.h"

namespace kda {

// Where a kernel finds keys and values: a paged cache, or the packed tokens of
// the call itself.
struct AttnArgs {
    const void *q;  // [T] rows of q_stride, H heads of K elements, in_dtype
    const void *k;  // packed: as q with Hk heads; cache: [pages, Hk, page, K]
    const void *v;
    const uint8_t *kexp, *vexp;  // E4M3 cache: [pages, Hk, page]
    int64_t qs, ks, vs;          // token strides in elements (ks, vs: packed only)
    const int32_t *cu;           // [N + 1]
    const int32_t *lens;         // [N] cache only
    const int32_t *table;        // [N, max_pages] cache only
    const uint64_t *mask;        // [T] or nullptr, cache only
    void *o;                     // [T, H, V]
    void *ws;                    // cache only
    int32_t N, T, H, Hk, G, K, V;
    int32_t page_shift, max_pages, num_pages;
    float c;                     // scale * log2(e): weights are 2^(c q.k - m)
    kda_dtype_t in_dtype, out_dtype;
    kda_kv_dtype_t kv_dtype;
    int32_t W;                   // workgroups that share the call's work (cache only)
    int32_t whole;               // cache only: no (sequence, kv head, row tile) is shared among workgroups
};

struct KvArgs {
    void *k, *v;                 // tokens: [T] rows of ks / vs elements
    void *kc, *vc;               // [pages, Hk, page, K | V]
    uint8_t *kexp, *vexp;
    int64_t ks, vs;
    const int32_t *cu, *lens, *table;
    int32_t N, T, Hk, K, V;
    int32_t page_shift, max_pages, num_pages;
    kda_dtype_t dtype;           // of k, v
    kda_kv_dtype_t kv_dtype;
};

// Compute units of the current device (cached per device).
int compute_units();

// Each launcher enqueues its kernel(s) on `stream` and returns the launch status.
hipError_t launch_attn_prompt(const AttnArgs &a, hipStream_t stream);
hipError_t launch_attn_cache(const AttnArgs &a, hipStream_t stream);
hipError_t launch_kv_write(const KvArgs &a, hipStream_t stream);
hipError_t launch_kv_read(const KvArgs &a, hipStream_t stream);

// Workgroups and workspace bytes of the cache attention on the current device, for page tables
// that reach max_tokens.
int32_t attn_cache_workgroups();
size_t attn_cache_workspace(int32_t N, int32_t T, int32_t H, int32_t Hk, int32_t V, int32_t max_tokens, kda_dtype_t in_dtype);

}  // namespace kda
