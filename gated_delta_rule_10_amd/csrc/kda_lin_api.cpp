// C-ABI layer of the linear-attention entry points (include/kda_lin.h):
// host-side argument validation and error mapping, as kda_api.cpp does for
// kda.h. Reads no device memory, allocates nothing and never synchronises.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kda_checks.h"
#include "kda_lin.h"
#include "kda_lin_internal.h"

using namespace kda;

namespace {

// Launches stay below 2^32 threads: single tokens N H workgroups of kLinDecodeThreads, prompts N H of up to
// 512 and a bounded number more for segments of long sequences.
static_assert(((int64_t(1) << 22) - 1) * kLinDecodeThreads < int64_t(1) << 32, "a launch's threads");
bool sizes_ok(int32_t N, int32_t T, int32_t H) {
    return N >= 1 && T >= 0 && T < INT32_MAX - 1023 && H >= 1 && static_cast<int64_t>(T) * H < INT32_MAX - 1023 &&
           static_cast<int64_t>(N) * H < int64_t(1) << 22;
}

// The decays' token stride: 0 for one value per head.
bool decay_ok(int64_t stride, int32_t H) { return stride == 0 || (stride >= H && stride <= (int64_t(1) << 24)); }

}  // namespace

extern "C" {

size_t kda_lin_chunk_fwd_workspace_size(int32_t N, int32_t T_total, int32_t H, int32_t d_k, int32_t d_v,
                                        kda_dtype_t in_dtype) {
    if (!sizes_ok(N, T_total, H) || !head_dim_ok(d_k) || !head_dim_ok(d_v) || !dtype_valid(in_dtype)) return 0;
    return lin_chunk_workspace(N, T_total, H, d_k, d_v, in_dtype);
}

kda_status_t kda_lin_chunk_fwd(const void *q, const void *k, const void *v, const float *log_decay,
                               const int32_t *cu_seqlens, int32_t N, int32_t T_total, int32_t H, int32_t Hk,
                               int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                               int64_t decay_stride, kda_dtype_t in_dtype, kda_dtype_t out_dtype, float scale,
                               const float *initial_state, float *final_state, const int32_t *state_slots,
                               int32_t num_slots, void *o, void *workspace, size_t workspace_bytes,
                               hipStream_t stream) {
    if (!sizes_ok(N, T_total, H) || Hk < 1 || H % Hk != 0) return KDA_ERR_INVALID_ARG;
    if (!dtype_valid(in_dtype) || !dtype_valid(out_dtype) || !given(cu_seqlens) || !std::isfinite(scale))
        return KDA_ERR_INVALID_ARG;
    const void *tokens[] = {q, k, v, log_decay, o};
    for (const void *p : tokens)
        if (T_total > 0 ? !given(p) : !aligned16(p)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(initial_state) || !aligned16(final_state) || !aligned16(state_slots) || !aligned16(workspace))
        return KDA_ERR_INVALID_ARG;
    if (state_slots && num_slots < 1) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v) || !dtype_pair_ok(in_dtype, out_dtype)) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(q_stride, Hk, d_k) || !stride_ok(k_stride, Hk, d_k) || !stride_ok(v_stride, H, d_v) ||
        !decay_ok(decay_stride, H))
        return KDA_ERR_INVALID_ARG;
    const size_t states = static_cast<size_t>(state_slots ? num_slots : N) * H * d_k * d_v * sizeof(float);
    if (initial_state != final_state && overlap(initial_state, states, final_state, states)) return KDA_ERR_INVALID_ARG;
    const size_t need = lin_chunk_workspace(N, T_total, H, d_k, d_v, in_dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
    LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.gs = decay_stride;
    a.cu = cu_seqlens; a.s0 = initial_state; a.sT = final_state; a.slots = state_slots; a.o = o; a.ws = workspace;
    a.N = N; a.T = T_total; a.H = H; a.Hk = Hk; a.K = d_k; a.V = d_v; a.nslots = state_slots ? num_slots : N;
    a.scale = scale; a.in_dtype = in_dtype; a.out_dtype = out_dtype;
    return finish(launch_lin_chunk(a, stream), stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

kda_status_t kda_lin_decode_step(const void *q, const void *k, const void *v, const float *log_decay,
                                 float *state_cache, const int32_t *slot_idx, void *o, int32_t B, int32_t H,
                                 int32_t Hk, int32_t d_k, int32_t d_v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, int64_t decay_stride, int32_t num_slots, kda_dtype_t in_dtype,
                                 kda_dtype_t out_dtype, float scale, hipStream_t stream) {
    if (!sizes_ok(B, B, H) || Hk < 1 || H % Hk != 0 || num_slots < 1) return KDA_ERR_INVALID_ARG;
    if (!dtype_valid(in_dtype) || !dtype_valid(out_dtype) || !std::isfinite(scale)) return KDA_ERR_INVALID_ARG;
    const void *all[] = {q, k, v, log_decay, state_cache, o};
    for (const void *p : all)
        if (!given(p)) return KDA_ERR_INVALID_ARG;
    if (!aligned16(slot_idx) || (!slot_idx && B > num_slots)) return KDA_ERR_INVALID_ARG;
    if (!head_dim_ok(d_k) || !head_dim_ok(d_v) || !dtype_pair_ok(in_dtype, out_dtype)) return KDA_ERR_UNSUPPORTED;
    if (!stride_ok(q_stride, Hk, d_k) || !stride_ok(k_stride, Hk, d_k) || !stride_ok(v_stride, H, d_v) ||
        !decay_ok(decay_stride, H))
        return KDA_ERR_INVALID_ARG;
    LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.qs = q_stride; a.ks = k_stride; a.vs = v_stride; a.gs = decay_stride;
    a.sT = state_cache; a.slots = slot_idx; a.o = o; a.N = B; a.T = B; a.H = H; a.Hk = Hk; a.K = d_k; a.V = d_v;
    a.nslots = num_slots; a.scale = scale; a.in_dtype = in_dtype; a.out_dtype = out_dtype;
    return finish(launch_lin_decode(a, stream), stream) == hipSuccess ? KDA_OK : KDA_ERR_HIP;
}

}  // extern "C"
