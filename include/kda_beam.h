/*
 * kda_beam.h -- C ABI of libkda: beam search over the recurrent states of KDA
 * and linear-attention layers, on AMD Instinct MI355X (gfx950).
 *
 * A step of a beam search has the single-token forms of kda.h or kda_lin.h run
 * with one state slot per beam, then chooses the next beams from all beams'
 * logits, and lets each chosen beam go on from its parent's state:
 *
 *     kda_beam_select    the K best (beam, token) pairs of every request
 *     kda_state_reorder  states and slots after the chosen parents
 *
 * Conventions: those of kda.h (device pointers, 16-byte aligned, the caller's;
 * no allocation, no synchronisation, all work on `stream`, capturable; arguments
 * checked on the host).
 */
#ifndef KDA_BEAM_H_
#define KDA_BEAM_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * For each of N requests with W beams, the K candidates of the largest
 *
 *     c(w, x) = scores[n][w] + logits[n][w][x] - ln sum_y e^logits[n][w][y]
 *
 * over beams w and tokens x of a vocabulary of V, in falling order; of equal ones
 * the lowest (w, x) first. A beam with done[n][w] != 0 has ended: its one
 * candidate is (w, done_token) with c = scores[n][w], and its logits are not read.
 * What is -infinity (in fp32) or NaN is no candidate: masked tokens (logits of
 * -infinity; a token at a finite mask, such as the type's lowest value, is a
 * candidate like any other), the tokens of a beam whose logits hold a NaN or
 * +infinity, and a beam whose score is -infinity (one that holds nothing, as all
 * but one of the first step's).
 * Where fewer than K candidates are left, the other places get score -infinity,
 * parent -1 and token -1.
 *
 *   logits      [N, W, V]  dtype (F32 or BF16); row n W + w at (n W + w) * stride
 *               elements, V <= stride <= 2^31
 *   scores      [N, W]     fp32, finite or -infinity
 *   done        [N, W]     uint8, or NULL (none has ended)
 *   out_scores  [N, K]     fp32: c, rounded once
 *   out_parent  [N, K]     int32: w
 *   out_token   [N, K]     int32: x
 *
 * Sums and comparisons: e^logit is right to 2^-23 of itself, sums of them and c
 * are fp64 (of two terms fp32), so that a row's logarithm is right to 2^-22,
 * which decides between candidates of different beams; those of one beam are
 * compared by their logits.
 * Sizes: N >= 1, 1 <= W <= 64, V >= 1, 1 <= K <= 64, W V < 2^31, N W < 2^20,
 * 0 <= done_token < V if done is given. Outputs share no memory with scores, done
 * or each other, but out_scores may be scores itself where K = W.
 * workspace: kda_beam_select_workspace_size bytes of device scratch, whatever
 * they hold. Calls that may overlap must not share one.
 */
kda_status_t kda_beam_select(const void *logits, int64_t stride, const float *scores, const uint8_t *done,
                             int32_t done_token, int32_t N, int32_t W, int32_t V, int32_t K, kda_dtype_t dtype,
                             float *out_scores, int32_t *out_parent, int32_t *out_token, void *workspace,
                             size_t workspace_bytes, hipStream_t stream);

/* Bytes of device workspace kda_beam_select needs on the current device (0 if the sizes are invalid). */
size_t kda_beam_select_workspace_size(int32_t N, int32_t W, int32_t V, int32_t K);

/*
 * States after a choice. Beam j of request n goes on from beam parent[n][j] of
 * it. The first beam (lowest j) that goes on from a parent keeps the parent's
 * slot; the other beams take the slots of the beams that none goes on from, in
 * rising order of both, and the parent's state is copied there. So a state is
 * only moved where a parent has several children, and no slot is both read and
 * written. A parent outside [0, W) is none: the beam takes a slot with whatever
 * it holds. So does a beam but the first that goes on from a parent whose slot
 * holds nothing (below): there is no state to copy, and the slot's own is another
 * beam's that has ended. Such a beam's state has to be written anew (a prompt
 * without an initial state, or a first token whose g is -infinity over finite
 * values) before it is read; kda_beam_select chooses no beam whose score is
 * -infinity, which is what a beam that holds nothing should have.
 *
 *   states      of every layer [num_slots] rows of slot_bytes (a state cache
 *               [num_slots, H, d_k, d_v], or any other per-sequence state),
 *               layer l at l * layer_stride bytes; updated in place
 *   slots       [N, W] int32: the beams' slots before. Distinct; a slot outside
 *               [0, num_slots) holds nothing and is not read or written.
 *   parent      [N, W] int32
 *   slots_out   [N, W] int32 output: their slots afterwards, a permutation of
 *               each request's. Shares no memory with slots or parent.
 *
 * Sizes: N >= 1, 1 <= W <= 64, N W < 2^20, layers >= 1, num_slots >= 1,
 * slot_bytes a multiple of 16 from 16 to 2^36, layer_stride a multiple of 16
 * and, with several layers, at least num_slots * slot_bytes; N layers < 2^22.
 */
kda_status_t kda_state_reorder(void *states, int64_t layer_stride, int32_t layers, int32_t num_slots,
                               int64_t slot_bytes, const int32_t *slots, const int32_t *parent, int32_t *slots_out,
                               int32_t N, int32_t W, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_BEAM_H_ */
