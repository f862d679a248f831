// C-ABI layer of the beam-search entry points (include/kda_beam.h): host-side
// argument validation and error mapping. Reads no device memory, allocates
// nothing and never synchronises.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "kda_beam.h"
#include "kda_beam_internal.h"
#include "kda_checks.h"

using namespace kda;

namespace {

bool beams_ok(int32_t N, int32_t W) {
    return N >= 1 && W >= 1 && W <= 64 && static_cast<int64_t>(N) * W < 1 << 20;
}
bool select_ok(int32_t N, int32_t W, int32_t V, int32_t K) {
    return beams_ok(N, W) && V >= 1 && K >= 1 && K <= 64 && static_cast<int64_t>(W) * V <= INT32_MAX;
}

}  // namespace

extern "C" {

size_t kda_beam_select_workspace_size(int32_t N, int32_t W, int32_t V, int32_t K) {
    return select_ok(N, W, V, K) ? beam_select_workspace(N, W, V) : 0;
}

kda_status_t kda_beam_select(const void *logits, int64_t stride, const float *scores, const uint8_t *done,
                             int32_t done_token, int32_t N, int32_t W, int32_t V, int32_t K, kda_dtype_t dtype,
                             float *out_scores, int32_t *out_parent, int32_t *out_token, void *workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    if (!select_ok(N, W, V, K) || !dtype_valid(dtype) || stride < V || stride > int64_t(1) << 31) return KDA_ERR_INVALID_ARG;
    const void *all[] = {logits, scores, out_scores, out_parent, out_token};
    for (const void *p : all)
        if (!given(p)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(done) || (done && (done_token < 0 || done_token >= V)) || !aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < beam_select_workspace(N, W, V)) return KDA_ERR_WORKSPACE;
    // A request's new scores may only take the place of its own: other requests' scores and beams that have ended are
    // still read while outputs are written.
    const size_t beams = static_cast<size_t>(N) * W, outs = static_cast<size_t>(N) * K * 4;
    const void *out[] = {out_scores, out_parent, out_token};
    for (int i = 0; i < 3; ++i) {
        const bool in_place = i == 0 && out_scores == scores && K == W;
        if ((!in_place && overlap(out[i], outs, scores, beams * 4)) || overlap(out[i], outs, done, beams)) return KDA_ERR_INVALID_ARG;
        if (overlap(out[i], outs, out[(i + 1) % 3], outs)) return KDA_ERR_INVALID_ARG;
    }
    SelectArgs a{};
    a.logits = logits; a.stride = stride; a.scores = scores; a.done = done; a.done_token = done_token;
    a.N = N; a.W = W; a.V = V; a.K = K; a.dtype = dtype;
    a.out_scores = out_scores; a.out_parent = out_parent; a.out_token = out_token; a.ws = workspace;
    return finish(launch_beam_select(a, stream), stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status_t kda_state_reorder(void *states, int64_t layer_stride, int32_t layers, int32_t num_slots,
                               int64_t slot_bytes, const int32_t *slots, const int32_t *parent, int32_t *slots_out,
                               int32_t N, int32_t W, hipStream_t stream) {
    if (!beams_ok(N, W) || layers < 1 || num_slots < 1 || static_cast<int64_t>(N) * layers >= 1 << 22) return KDA_ERR_INVALID_ARG;
    if (!given(states) || !given(slots) || !given(parent) || !given(slots_out)) return KDA_ERR_INVALID_ARG;
    const size_t beams = static_cast<size_t>(N) * W * sizeof(int32_t);  // every workgroup reads its request's
    if (overlap(slots_out, beams, slots, beams) || overlap(slots_out, beams, parent, beams)) return KDA_ERR_INVALID_ARG;
    if (slot_bytes < 16 || slot_bytes % 16 != 0 || slot_bytes > int64_t(1) << 36) return KDA_ERR_INVALID_ARG;
    if (layers > 1 && (layer_stride % 16 != 0 || layer_stride / slot_bytes < num_slots)) return KDA_ERR_INVALID_ARG;
    ReorderArgs a{};
    a.states = static_cast<char *>(states); a.layer_stride = layer_stride; a.slot_bytes = slot_bytes;
    a.slots = slots; a.parent = parent; a.slots_out = slots_out; a.layers = layers; a.nslots = num_slots; a.N = N; a.W = W;
    return finish(launch_state_reorder(a, stream), stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
