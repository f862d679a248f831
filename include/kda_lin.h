/*
 * kda_lin.h -- C ABI of libkda: linear attention with one decay per head, on
 * AMD Instinct MI355X (gfx950).
 *
 * The layers of this kind that stand where KDA layers stand in other hybrid
 * stacks forget by one factor per head instead of one per key channel, and write
 * without the delta rule's correction. Per (sequence, value head), with a
 * d_k x d_v fp32 state S (row i = key channel i, column j = value channel j):
 *
 *     S_t = e^(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t
 *
 * Two entry points, as for KDA:
 *
 *     kda_lin_chunk_fwd    packed variable-length prompts, chunkwise
 *     kda_lin_decode_step  one token per sequence, the state cache in place
 *
 * Forward only, like kda.h. The states have the layout of kda.h's, so one cache
 * and one set of slots serve both kinds of layer (and kda_beam.h's reordering).
 *
 * Conventions: those of kda.h. Pointers are device memory on the current HIP
 * device, 16-byte aligned, owned by the caller; the library allocates nothing
 * and never synchronises; all work is enqueued on `stream` and can be captured
 * in a HIP graph; arguments are checked on the host before anything is
 * enqueued. Status codes, types, kda_status_string and KDA_DEBUG_SYNC are
 * kda.h's.
 *  - H is the number of value heads (of v, log_decay, o and the states), Hk the
 *    number of key/query heads; H is a multiple of Hk, and value head h uses
 *    key head h / (H / Hk).
 *  - d_k and d_v are 64 or 128, each on its own.
 *  - q, k and v may be parts of wider rows (a fused projection): element
 *    (t, h, i) is at t * stride + h * d + i, with the token stride in elements,
 *    at least heads * d, at most 2^24 and a multiple of 8. Outputs are dense.
 *  - log_decay is fp32: g of token t and head h at t * decay_stride + h. A
 *    decay_stride of 0 gives every token of a head the same g ([H]); otherwise
 *    it is at least H and at most 2^24. g <= 0; -infinity forgets a finite
 *    state whole (a token that starts anew). g below -110 counts as -110 where it is
 *    summed, and e^-110 is 0 in fp32.
 *  - Device-side contents that break the rules below never cause an access
 *    outside the given arrays: offsets are clamped to [0, T], and a slot outside
 *    [0, num_slots) holds nothing: its sequence starts from zeros and its state
 *    is not written (padding).
 *  - Arithmetic: the state, decays and sums are fp32 (sums of g in fp64). fp32
 *    inputs are multiplied in fp32. With bf16 inputs q, k and v are exact, the
 *    decayed values go into the state with 24 bits, so that states are right to
 *    fp32, and the decayed scores and the state that q reads are rounded for the
 *    outputs to the sum of two bf16 numbers (by at most 2^-16 of each term),
 *    whatever the outputs' type. Single tokens are fp32 throughout.
 *    Results do not depend on timing: no atomics. They may differ in the last bits
 *    between batches, which decide where long sequences are cut into segments.
 *  - Range: products and states have to stay below 2^120 in magnitude. An
 *    infinity or NaN in a token's q reaches that token's output only. In its k, v
 *    or g it may reach the outputs of its head from that token on and the state,
 *    and does as long as it has not decayed to 0 (how far it goes then depends on
 *    where the sequence is cut); never an earlier token, another head or another
 *    sequence.
 */
#ifndef KDA_LIN_H_
#define KDA_LIN_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention over N packed sequences. Sequence n has rows
 * [cu_seqlens[n], cu_seqlens[n + 1]) of the packed token axis; rows before
 * cu_seqlens[0] and from cu_seqlens[N] on are neither read nor written.
 *
 *   q, k        [T_total, Hk, d_k]  in_dtype    v [T_total, H, d_v] in_dtype
 *   log_decay   [T_total, H] or [H] fp32
 *   cu_seqlens  [N + 1] int32
 *   state_slots NULL: initial_state and final_state are [N, H, d_k, d_v] fp32.
 *               [N] int32: they are caches [num_slots, H, d_k, d_v], and
 *               sequence n uses slot state_slots[n] of both. Slots of different
 *               sequences must differ.
 *   initial_state  NULL for zeros
 *   final_state    output, NULL if not wanted; may be the same pointer as
 *                  initial_state, else shares no memory with it. A sequence
 *                  without tokens leaves final_state = initial_state (or 0).
 *   o           [T_total, H, d_v]   out_dtype output (dense), shares no memory
 *               with the inputs
 *
 * Sizes: N >= 1, H >= 1, 0 <= T_total < 2^31 - 1024, T_total H < 2^31 - 1024,
 * N H < 2^22; num_slots >= 1 with state_slots. `scale` is finite and multiplies
 * o only. dtype pairs: (F32, F32), (BF16, BF16), (BF16, F32).
 * workspace: kda_lin_chunk_fwd_workspace_size bytes of device scratch, whatever
 * they hold (NULL if that is 0). Calls that may overlap must not share one.
 */
kda_status_t kda_lin_chunk_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                               const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t H, int32_t Hk,
                               int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               int64_t decay_stride, kda_dtype_t in_dtype, kda_dtype_t out_dtype, float scale,
                               const float *initial_state, float *final_state, const int32_t *state_slots,
                               int32_t num_slots, void *o, void *workspace, size_t workspace_bytes,
                               hipStream_t stream);

/*
 * Bytes of device workspace kda_lin_chunk_fwd needs on the current device for
 * these sizes; 0 means the call may pass workspace = NULL (or the sizes are
 * invalid).
 */
size_t kda_lin_chunk_fwd_workspace_size(int32_t N, int32_t T_total, int32_t H, int32_t d_k, int32_t d_v,
                                        kda_dtype_t in_dtype);

/*
 * One token for each of B sequences, updating the fp32 state cache in place.
 *
 *   q, k        [B, Hk, d_k]  in_dtype     v [B, H, d_v] in_dtype
 *   log_decay   [B, H] or [H] fp32
 *   state_cache [num_slots, H, d_k, d_v] fp32
 *   slot_idx    [B] int32 of distinct slots, or NULL for slot b = b (then
 *               B <= num_slots)
 *   o           [B, H, d_v]   out_dtype output (dense)
 *
 * Sizes: B >= 1, H >= 1, num_slots >= 1, B H < 2^22. All arithmetic is fp32.
 */
kda_status_t kda_lin_decode_step(const void *q, const void *k, const void *v, const float *log_decay,
                                 float *state_cache, const int32_t *slot_idx, void *o, int32_t B, int32_t H,
                                 int32_t Hk, int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, int64_t decay_stride, int32_t num_slots, kda_dtype_t in_dtype,
                                 kda_dtype_t out_dtype, float scale, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LIN_H_ */
