// C-ABI layer of the attention entry points (include/kda_attn.h): host-side
// argument validation, kernel selection and error mapping, as kda_api.cpp does
// for kda.h. Reads no device memory, allocates nothing and never synchronises.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "kda_attn.h"
#include "kda_attn_internal.h"
#include "kda_checks.h"

using namespace kda;

namespace {

bool kv_dtype_valid(kda_kv_dtype_t d) { return d == KDA_KV_F32 || d == KDA_KV_BF16 || d == KDA_KV_E4M3; }

bool kv_pair_ok(kda_dtype_t in, kda_kv_dtype_t kv) { return (in == KDA_F32) == (kv == KDA_KV_F32); }

// Sizes shared by all entry points. d_k and d_v are checked separately (KDA_ERR_UNSUPPORTED).
bool sizes_ok(int32_t N, int32_t T, int32_t H, int32_t Hk) {
    if (N < 1 || T < 0 || H < 1 || Hk < 1 || H % Hk != 0) return false;
    if (static_cast<int64_t>(T) * H >= INT32_MAX - 1023) return false;  // rows (token, head) are int32 on the device
    return static_cast<int64_t>(N) * H * 16 <= INT32_MAX;  // grids, with one tile more per sequence and head
}

// A launch has to stay below 2^32 threads. Prompts: tiles of 256 rows and 512 threads (fp32: 16 and
// 256), one more tile per sequence and kv head. Cache attention: the join's 512 threads per 16 rows
// of tiles of up to 128. Cache writes and reads: 4 threads to a row, 64 rows to a workgroup.
bool below(int64_t x, int bits) { return x < int64_t(1) << bits; }
bool prompt_ok(int64_t N, int64_t T, int64_t H, int64_t Hk, kda_dtype_t in) {
    return in == KDA_F32 ? below(T * H + 16 * N * Hk, 28) : below(T * H + 256 * N * Hk, 31);
}
bool cache_ok(int64_t N, int64_t T, int64_t H, int64_t Hk) { return below(T * H + 128 * N * Hk, 27); }
bool kv_ok(int64_t T, int64_t Hk) { return below(T * Hk + 64, 30); }

// The cache of a call over N sequences of Hk kv heads, without its type pair.
kda_status_t check_cache(const kda_kv_cache_t *c, int32_t N) {
    if (!c || !kv_dtype_valid(c->dtype)) return KDA_ERR_INVALID_ARG;
    const void *req[] = {c->k, c->v, c->page_table, c->lens};
    for (const void *p : req)
        if (!given(p)) return KDA_ERR_INVALID_ARG;
    if (c->dtype == KDA_KV_E4M3) {
        if (!given(c->k_exp) || !given(c->v_exp)) return KDA_ERR_INVALID_ARG;
    } else if (c->k_exp || c->v_exp) {
        return KDA_ERR_INVALID_ARG;
    }
    if (c->num_pages < 1 || c->max_pages < 1) return KDA_ERR_INVALID_ARG;
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return KDA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c->max_pages) * c->page_size >= INT32_MAX - 1023) return KDA_ERR_INVALID_ARG;
    if (static_cast<int64_t>(N) * c->max_pages > INT32_MAX) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// scale in the log2 domain has to be finite too
constexpr double kLog2e = 1.4426950408889634;
bool scale_ok(float s) { return std::isfinite(static_cast<float>(s * kLog2e)); }

int32_t log2_of(int32_t x) {
    int32_t s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

kda_status_t kv_call(bool write, void *k, void *v, const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t Hk,
                     int32_t d_k, int32_t d_v, int64_t k_stride, int64_t v_stride, kda_dtype_t dtype,
                     const kda_kv_cache_t *cache, hipStream_t stream) {
    if (!sizes_ok(N, T_total, Hk, Hk) || !kv_ok(T_total, Hk) || !dtype_valid(dtype) || !given(cu_seqlens)) return KDA_ERR_INVALID_ARG;
    const kda_status_t cs = check_cache(cache, N);
    if (cs != KDA_OK) return cs;
    if (T_total > 0 && (!given(k) || !given(v))) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v)) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(k_stride, Hk, d_k) || !stride_ok(v_stride, Hk, d_v)) return KDA_ERR_INVALID_ARG;
    // written from F32 to an F32 cache and from BF16 to the others; read into F32 from any
    if (write ? !kv_pair_ok(dtype, cache->dtype) : dtype == KDA_BF16 && cache->dtype == KDA_KV_F32)
        return KDA_ERR_UNSUPPORTED;
    if (T_total == 0) return KDA_OK;
    kda::KvArgs a{};
    a.k = k; a.v = v; a.kc = cache->k; a.vc = cache->v; a.kexp = cache->k_exp; a.vexp = cache->v_exp;
    a.ks = k_stride; a.vs = v_stride; a.cu = cu_seqlens; a.lens = cache->lens; a.table = cache->page_table;
    a.N = N; a.T = T_total; a.Hk = Hk; a.K = d_k; a.V = d_v;
    a.page_shift = log2_of(cache->page_size); a.max_pages = cache->max_pages; a.num_pages = cache->num_pages;
    a.dtype = dtype; a.kv_dtype = cache->dtype;
    const hipError_t e = write ? kda::launch_kv_write(a, stream) : kda::launch_kv_read(a, stream);
    return finish(e, stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // namespace

namespace kda {

// threads that race on a device's first query store the same value
int compute_units() {
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1) n = 256;
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace kda

extern "C" {

kda_status_t kda_attn_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int32_t N,
                          int32_t T_total, int32_t H, int32_t Hk, int32_t d_k, int32_t d_v, int64_t q_stride,
                          int64_t k_stride, int64_t v_stride, kda_dtype_t in_dtype, kda_dtype_t out_dtype,
                          float scale, void *o, hipStream_t stream) {
    if (!sizes_ok(N, T_total, H, Hk) || !dtype_valid(in_dtype) || !dtype_valid(out_dtype)) return KDA_ERR_INVALID_ARG;
    if (!prompt_ok(N, T_total, H, Hk, in_dtype)) return KDA_ERR_INVALID_ARG;
    if (!given(cu_seqlens) || !scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    if (T_total > 0 && (!given(q) || !given(k) || !given(v) || !given(o))) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v) || !dtype_pair_ok(in_dtype, out_dtype)) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(q_stride, H, d_k) || !stride_ok(k_stride, Hk, d_k) || !stride_ok(v_stride, Hk, d_v))
        return KDA_ERR_INVALID_ARG;
    if (T_total == 0) return KDA_OK;
    kda::AttnArgs a{};
    a.q = q; a.k = k; a.v = v; a.qs = q_stride; a.ks = k_stride; a.vs = v_stride;
    a.cu = cu_seqlens; a.o = o; a.N = N; a.T = T_total; a.H = H; a.Hk = Hk; a.G = H / Hk; a.K = d_k; a.V = d_v;
    a.c = static_cast<float>(scale * kLog2e);
    a.in_dtype = in_dtype; a.out_dtype = out_dtype;
    return finish(kda::launch_attn_prompt(a, stream), stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status_t kda_kv_write(const void *k, const void *v, const int32_t *cu_seqlens, int32_t N, int32_t T_total,
                          int32_t Hk, int32_t d_k, int32_t d_v, int64_t k_stride, int64_t v_stride,
                          kda_dtype_t in_dtype, const kda_kv_cache_t *cache, hipStream_t stream) {
    return kv_call(true, const_cast<void *>(k), const_cast<void *>(v), cu_seqlens, N, T_total, Hk, d_k, d_v, k_stride,
                   v_stride, in_dtype, cache, stream);
}

kda_status_t kda_kv_read(void *k, void *v, const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t Hk,
                         int32_t d_k, int32_t d_v, kda_dtype_t out_dtype, const kda_kv_cache_t *cache,
                         hipStream_t stream) {
    return kv_call(false, k, v, cu_seqlens, N, T_total, Hk, d_k, d_v, static_cast<int64_t>(Hk) * d_k,
                   static_cast<int64_t>(Hk) * d_v, out_dtype, cache, stream);
}

size_t kda_attn_cache_fwd_workspace_size(int32_t N, int32_t T_total, int32_t H, int32_t Hk, int32_t d_k, int32_t d_v,
                                         int32_t max_tokens, kda_dtype_t in_dtype) {
    if (!sizes_ok(N, T_total, H, Hk) || !cache_ok(N, T_total, H, Hk) || !head_dim_ok(d_k) || !head_dim_ok(d_v) || !dtype_valid(in_dtype)) return 0;
    if (T_total == 0 || max_tokens < 1) return 0;
    return kda::attn_cache_workspace(N, T_total, H, Hk, d_v, max_tokens, in_dtype);
}

kda_status_t kda_attn_cache_fwd(const void *q, const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t H,
                                int32_t Hk, int32_t d_k, int32_t d_v, int64_t q_stride, kda_dtype_t in_dtype,
                                kda_dtype_t out_dtype, float scale, const kda_kv_cache_t *cache,
                                const uint64_t *tree_mask, void *o, void *workspace, size_t workspace_bytes,
                                hipStream_t stream) {
    if (!sizes_ok(N, T_total, H, Hk) || !dtype_valid(in_dtype) || !dtype_valid(out_dtype)) return KDA_ERR_INVALID_ARG;
    if (!cache_ok(N, T_total, H, Hk)) return KDA_ERR_INVALID_ARG;
    if (!given(cu_seqlens) || !scale_ok(scale)) return KDA_ERR_INVALID_ARG;
    const kda_status_t cs = check_cache(cache, N);
    if (cs != KDA_OK) return cs;
    if (T_total > 0 && (!given(q) || !given(o))) return KDA_ERR_INVALID_ARG;
    if (!aligned16(tree_mask) || !aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v) || !dtype_pair_ok(in_dtype, out_dtype) || !kv_pair_ok(in_dtype, cache->dtype))
        return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(q_stride, H, d_k)) return KDA_ERR_INVALID_ARG;
    if (T_total == 0) return KDA_OK;
    const size_t need =
        kda::attn_cache_workspace(N, T_total, H, Hk, d_v, cache->max_pages * cache->page_size, in_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    kda::AttnArgs a{};
    a.q = q; a.k = cache->k; a.v = cache->v; a.kexp = cache->k_exp; a.vexp = cache->v_exp; a.qs = q_stride;
    a.cu = cu_seqlens; a.lens = cache->lens; a.table = cache->page_table; a.mask = tree_mask; a.o = o; a.ws = workspace;
    a.N = N; a.T = T_total; a.H = H; a.Hk = Hk; a.G = H / Hk; a.K = d_k; a.V = d_v;
    a.page_shift = log2_of(cache->page_size); a.max_pages = cache->max_pages; a.num_pages = cache->num_pages;
    a.c = static_cast<float>(scale * kLog2e);
    a.in_dtype = in_dtype; a.out_dtype = out_dtype; a.kv_dtype = cache->dtype;
    return finish(kda::launch_attn_cache(a, stream), stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
