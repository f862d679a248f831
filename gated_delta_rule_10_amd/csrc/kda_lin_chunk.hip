// Linear attention with one decay per head over packed prompts (kda_lin_chunk_fwd).
//
// Token by token, as the definition says: a workgroup holds the state of one
// (sequence, value head) in registers, each thread V / 256 part of a column.
#include "kda_lin_device.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int clamp_to(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

template <int K, int V, typename TIn, typename TOut>
__global__ __launch_bounds__(kThreads) void lin_tokens_kernel(LinArgs a) {
    constexpr int P = kThreads / V, R = K / P;  // threads to a column, rows of each
    __shared__ float qs[K], ks[K], part[P][V];
    const int tid = threadIdx.x, col = tid % V, p = tid / V;
    const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H, hk = h / (a.H / a.Hk);
    const int start = clamp_to(a.cu[n], 0, a.T), end = clamp_to(a.cu[n + 1], start, a.T), slot = slot_of(a, n);
    const int64_t base = (static_cast<int64_t>(slot) * a.H + h) * (K * V) + col;
    float S[R];
#pragma unroll
    for (int i = 0; i < R; ++i) S[i] = a.s0 && slot >= 0 ? a.s0[base + (p * R + i) * V] : 0.f;
    for (int t = start; t < end; ++t) {
        __syncthreads();
        if (tid < K) {
            qs[tid] = io<TIn>::load(static_cast<const TIn *>(a.q) + t * a.qs + hk * K + tid);
            ks[tid] = io<TIn>::load(static_cast<const TIn *>(a.k) + t * a.ks + hk * K + tid);
        }
        const float v = io<TIn>::load(static_cast<const TIn *>(a.v) + t * a.vs + h * V + col), d = __expf(log_decay_of(a, t, h));
        __syncthreads();
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            S[i] = fmaf(ks[p * R + i], v, d * S[i]);
            o = fmaf(qs[p * R + i], S[i], o);
        }
        part[p][col] = o;
        __syncthreads();
        if (p == 0) {
            for (int i = 1; i < P; ++i) o += part[i][col];
            store_out(static_cast<TOut *>(a.o) + (static_cast<int64_t>(t) * a.H + h) * V + col, a.scale * o);
        }
    }
    if (a.sT && slot >= 0)
#pragma unroll
        for (int i = 0; i < R; ++i) a.sT[base + (p * R + i) * V] = S[i];
}

template <int K, int V> hipError_t launch_dims(const LinArgs &a, hipStream_t st) {
    const dim3 grid(a.N * a.H), block(kThreads);
    if (a.in_dtype == KDA_F32)
        hipLaunchKernelGGL((lin_tokens_kernel<K, V, float, float>), grid, block, 0, st, a);
    else if (a.out_dtype == KDA_BF16)
        hipLaunchKernelGGL((lin_tokens_kernel<K, V, bf16_t, bf16_t>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((lin_tokens_kernel<K, V, bf16_t, float>), grid, block, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_chunk(const LinArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

size_t lin_chunk_workspace(int32_t, int32_t, int32_t, int32_t, int32_t, kda_dtype_t) { return 0; }

}  // namespace kda
