/*
 * kda_attn.h -- C ABI of libkda: softmax attention for the full-attention
 * layers that stand between KDA layers, on AMD Instinct MI355X (gfx950).
 *
 * A hybrid stack interleaves KDA layers with full softmax attention (3:1 in
 * the Kimi Linear article, "Kimi Linear爆发背后的秘密：重新定义长上下文推理效率",
 * xugj520.cn). These entry points are the two steps of such a layer with grouped
 * query heads of 64 or 128 channels, on the packed variable-length layout of
 * kda.h, and the paged key/value cache between them. (The article's own full
 * layers are MLA, whose expanded keys are wider and whose cache is a latent:
 * neither is here.)
 *
 *     kda_attn_fwd        causal attention inside each packed sequence (prompt)
 *     kda_kv_write        new keys and values into the paged cache
 *     kda_kv_read         the same tokens back out of it
 *     kda_attn_cache_fwd  attention of new tokens over the cache: one token
 *                         per sequence, several, or a tree of drafted tokens
 *
 * For a row (token i, query head h) with kv head g = h / (H / Hk):
 *
 *     w_j = exp(scale q_i . k_j - max),   o_i = sum_j w_j v_j / sum_j w_j
 *
 * over the tokens j that the row sees. A row that sees no token is 0. A token
 * that a row does not see has no influence on it, whatever its k and v hold
 * (infinities and NaN included).
 *
 * Conventions: those of kda.h. Pointers are device memory on the current HIP
 * device, 16-byte aligned, owned by the caller; the library allocates nothing
 * and never synchronises; all work is enqueued on `stream` and can be captured
 * in a HIP graph; arguments are checked on the host before anything is
 * enqueued. Status codes, types, kda_status_string and KDA_DEBUG_SYNC are
 * kda.h's; the texts name the limits of kda.h. Here KDA_ERR_UNSUPPORTED is also
 * a page size or a pair of input and cache types that there is no kernel for,
 * and KDA_ERR_WORKSPACE a workspace smaller than
 * kda_attn_cache_fwd_workspace_size().
 *  - H is the number of query heads, Hk the number of key/value heads; H is a
 *    multiple of Hk, and query head h uses kv head h / (H / Hk).
 *  - d_k and d_v are 64 or 128, each on its own.
 *  - q, k and v may be parts of wider rows (a fused projection): element
 *    (t, h, i) is at t * stride + h * d + i, with the token stride in elements,
 *    at least heads * d, at most 2^24 and a multiple of 8. Outputs are dense.
 *  - cu_seqlens [N + 1] int32: sequence n has rows [cu_seqlens[n],
 *    cu_seqlens[n + 1]) of the packed token axis. Rows from cu_seqlens[N] on
 *    are neither read nor written.
 *  - Device-side contents that break the rules below never cause an access
 *    outside the given arrays: offsets are clamped to [0, T], cached lengths
 *    to the page table's reach, and a page outside [0, num_pages) holds
 *    nothing (not written, read as zeros, seen by no row).
 *  - Arithmetic: fp32 scores, softmax statistics and accumulation. With bf16
 *    inputs the weights w_j are rounded to bf16 (by at most 2^-8 of each) before
 *    the product with v; over a cache with up to 16 rows (mean new tokens of a
 *    sequence times H / Hk) they keep 16 bits. E4M3 codes are multiplied as
 *    exact bf16 numbers, but below bf16's least normal one (2^-126) and above
 *    its largest (infinity). Results do not depend on timing: no atomics.
 *  - Range: outputs are summed before they are divided, with weights of up to
 *    2^8, so finite values of v have to stay below 2^120 / (tokens that a row
 *    sees) in magnitude; larger ones may give infinities or NaN. Down to 2^-100
 *    they keep the accuracy above; below it, the smallest weights are lost. An
 *    infinity in v is one in the rows that see it, but may be NaN where its
 *    weight is below 2^-126.
 *  - cu_seqlens, lens, page_table and tree_mask must not change while a call
 *    that reads them runs.
 */
#ifndef KDA_ATTN_H_
#define KDA_ATTN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What a cache holds. */
typedef enum {
    KDA_KV_F32 = 0,  /* fp32, as given (F32 inputs) */
    KDA_KV_BF16 = 1, /* bf16, as given (BF16 inputs) */
    KDA_KV_E4M3 = 2  /* 8-bit floats (4 exponent bits, 3 of mantissa, largest 448, no infinity) with
                        one power-of-two scale per token and head (BF16 inputs) */
} kda_kv_dtype_t;

/*
 * A paged key/value cache, and which of its pages a batch of N sequences uses.
 * Position p of sequence n lies in page page_table[n][p / page_size], at
 * offset p % page_size of it.
 */
typedef struct {
    void *k; /* [num_pages, Hk, page_size, d_k] kv_dtype */
    void *v; /* [num_pages, Hk, page_size, d_v] kv_dtype */
    /* E4M3 only (NULL otherwise): [num_pages, Hk, page_size], the scale of a
     * token and head as a biased exponent: value = code * 2^(byte - 127). */
    uint8_t *k_exp;
    uint8_t *v_exp;
    const int32_t *page_table; /* [N, max_pages] */
    const int32_t *lens;       /* [N] tokens of each sequence in the cache, the new ones of the call included */
    int32_t num_pages;
    int32_t page_size; /* 16, 32, 64, 128 or 256 */
    int32_t max_pages; /* row length of page_table */
    kda_kv_dtype_t dtype;
} kda_kv_cache_t;

/*
 * Causal attention inside each of N packed sequences: token i sees the tokens
 * of its sequence up to and including itself.
 *
 *   q  [T_total, H, d_k]   k  [T_total, Hk, d_k]   v  [T_total, Hk, d_v]   in_dtype
 *   o  [T_total, H, d_v]   out_dtype output (dense)
 *
 * Sizes: N >= 1, H >= 1, T_total >= 0, 16 N H < 2^31, and, as a launch holds less
 * than 2^32 threads, T_total H + 256 N Hk < 2^31 (F32 inputs: T_total H + 16 N Hk <
 * 2^28); T_total H < 2^31 - 1024.
 * dtype pairs: (F32, F32), (BF16, BF16), (BF16, F32).
 * `scale` is finite (1 / sqrt(d_k) is customary).
 */
kda_status_t kda_attn_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int32_t N,
                          int32_t T_total, int32_t H, int32_t Hk, int32_t d_k, int32_t d_v, int64_t q_stride,
                          int64_t k_stride, int64_t v_stride, kda_dtype_t in_dtype, kda_dtype_t out_dtype,
                          float scale, void *o, hipStream_t stream);

/*
 * Write T_total packed new tokens into the cache: of sequence n's L =
 * cu_seqlens[n + 1] - cu_seqlens[n] new tokens, token i goes to position
 * lens[n] - L + i (one with a negative position is not written).
 *
 * F32 and BF16 caches hold k and v as given. An E4M3 cache holds, per token
 * and head, the least e >= -127 with max |x| <= 448 * 2^e over the row's finite
 * elements, and x * 2^-e rounded to the nearest code (ties to even): exact but
 * for that one rounding. An infinity or NaN becomes a NaN. Pages may be shared
 * by sequences, but a place that the call writes must be one position of one
 * sequence.
 * Sizes, here and for kda_kv_read: N >= 1, Hk >= 1, T_total >= 0, 16 N Hk < 2^31,
 * T_total Hk < 2^30 - 64.
 */
kda_status_t kda_kv_write(const void *k, const void *v, const int32_t *cu_seqlens, int32_t N, int32_t T_total,
                          int32_t Hk, int32_t d_k, int32_t d_v, int64_t k_stride, int64_t v_stride,
                          kda_dtype_t in_dtype, const kda_kv_cache_t *cache, hipStream_t stream);

/*
 * Read the last cu_seqlens[n + 1] - cu_seqlens[n] cached tokens of every
 * sequence (the positions that kda_kv_write fills for the same arguments) into
 * dense k [T_total, Hk, d_k] and v [T_total, Hk, d_v] of out_dtype (F32 from
 * any cache, BF16 from BF16 and E4M3). Positions that hold nothing read as
 * zeros. A code's value rounds to out_dtype: exact, but below bf16's least
 * normal number and above its largest (which becomes infinity).
 */
kda_status_t kda_kv_read(void *k, void *v, const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t Hk,
                         int32_t d_k, int32_t d_v, kda_dtype_t out_dtype, const kda_kv_cache_t *cache,
                         hipStream_t stream);

/*
 * Attention of T_total packed new tokens over the cache, which holds their own
 * keys and values already (kda_kv_write first). Sequence n's L new tokens are
 * the last L of its lens[n] cached ones. Each sees every token before the
 * first new one, and of the new ones:
 *   tree_mask NULL: those up to and including itself;
 *   tree_mask [T_total] uint64: new token b of its sequence where bit b is set.
 *     Set a token's own bit for it to see itself. Tokens from the 65th on are
 *     seen by none of a sequence's new tokens.
 *
 *   q  [T_total, H, d_k]  in_dtype    o  [T_total, H, d_v]  out_dtype output (dense)
 *
 * dtype pairs as for kda_attn_fwd; F32 inputs with an F32 cache, BF16 inputs
 * with a BF16 or E4M3 one. Sizes: N >= 1, H >= 1, T_total >= 0, 16 N H < 2^31,
 * T_total H + 128 N Hk < 2^27, N max_pages < 2^31, max_pages page_size < 2^31 - 1024.
 * Meant for single tokens and drafts: chunks of a prompt are right here too, but
 * without the prompt kernel's overlap. The form is chosen for the whole call, from
 * the mean number of new tokens.
 * workspace: kda_attn_cache_fwd_workspace_size bytes of device scratch, whatever
 * they hold (NULL if that is 0). Calls that may overlap must not share one.
 */
kda_status_t kda_attn_cache_fwd(const void *q, const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t H,
                                int32_t Hk, int32_t d_k, int32_t d_v, int64_t q_stride, kda_dtype_t in_dtype,
                                kda_dtype_t out_dtype, float scale, const kda_kv_cache_t *cache,
                                const uint64_t *tree_mask, void *o, void *workspace, size_t workspace_bytes,
                                hipStream_t stream);

/*
 * Bytes of device workspace kda_attn_cache_fwd needs on the current device for
 * these sizes and page tables that reach max_tokens = max_pages * page_size
 * cached tokens; 0 means the call may pass workspace = NULL (or the sizes are
 * invalid). It grows with N, and is otherwise bounded by the device's compute
 * units, not by the cached lengths.
 */
size_t kda_attn_cache_fwd_workspace_size(int32_t N, int32_t T_total, int32_t H, int32_t Hk, int32_t d_k,
                                         int32_t d_v, int32_t max_tokens, kda_dtype_t in_dtype);

#ifdef __cplusplus
}
#endif

#endif /* KDA_ATTN_H_ */
