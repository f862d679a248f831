// Causal attention inside packed sequences (kda_attn_fwd).
//
// A workgroup takes one tile of R rows of a (sequence, kv head), row r being
// token r / G and query head r % G, and streams the keys and values up to the
// tile's last token.
#include "kda_attn_stream.h"

namespace kda {
namespace {

template <int K, int V, int RT, typename TC>
__global__ __launch_bounds__(64 * kWaves) void attn_prompt_kernel(AttnArgs a, int slots) {
    using S = Stream<K, V, RT, TC>;
    constexpr int R = S::R;
    __shared__ __align__(16) char lds[S::kLds];
    __shared__ float stat[2][kWaves][R];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    char *lk = lds + w * (S::KB + S::VB), *lv = lk + S::KB;

    const int kvh = blockIdx.x % a.Hk;
    const int64_t slot = slots - 1 - static_cast<int>(blockIdx.x / a.Hk);  // the longest first
    const int n = seq_of_slot(a.cu, a.N, a.T, a.G, R, slot);
    int start, count;
    seq_rows(a.cu, n, a.T, start, count);
    const int64_t first = (slot - static_cast<int64_t>(start) * a.G / R - n) * R;
    if (first < 0 || first >= static_cast<int64_t>(count) * a.G) return;
    const int r0 = static_cast<int>(first);
    const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(count) * a.G - r0));
    const int open = r0 / a.G + 1, last = (r0 + rows - 1) / a.G + 1;

    S st;
    st.reset();
    st.load_q(a, start, kvh, r0, rows, lane);
    const bool here[2] = {true, true};
    const uint32_t none[2] = {0, 0};
    if (w * kStepWave < last) st.load_packed(a, start, kvh, w * kStepWave, lane);
    for (int p0 = w * kStepWave; p0 < last; p0 += kStep) {
        const bool masked = p0 + kStepWave > open;
        uint32_t sees[RT];
        if (masked) st.visible(sees, a, start, r0, rows, p0, 0, count, here, lane);
        const bool odd = st.stage(lk, lv, masked, p0, count, here, lane);
        if (p0 + kStep < last) st.load_packed(a, start, kvh, p0 + kStep, lane);
        __builtin_amdgcn_wave_barrier();
        st.step(lk, lv, a.c, masked, sees, odd, none, none, lane);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    st.join(lds, stat, w, lane, rows, [&](int row, int ch, float, f32x4 x, float l) {
        store_out(a, start, kvh, r0 + row, ch, x, l);
    });
}

template <int K, int V, int RT, typename TC>
hipError_t launch_rt(const AttnArgs &a, hipStream_t st) {
    const int64_t slots = static_cast<int64_t>(a.T) * a.G / (16 * RT) + a.N;
    hipLaunchKernelGGL((attn_prompt_kernel<K, V, RT, TC>), dim3(static_cast<unsigned>(slots * a.Hk)), dim3(64 * kWaves), 0, st,
                       a, static_cast<int>(slots));
    return hipGetLastError();
}

template <int K, int V> hipError_t launch_dims(const AttnArgs &a, hipStream_t st) {
    if (a.in_dtype == KDA_F32) return launch_rt<K, V, 2, float>(a, st);
    return launch_rt<K, V, 4, bf16_t>(a, st);
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace kda
