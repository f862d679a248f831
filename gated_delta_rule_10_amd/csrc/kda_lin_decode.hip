// Linear attention with one decay per head, one token per sequence
// (kda_lin_decode_step): S = e^g S + k v^T in place, o = scale S^T q.
//
// Bound by the state, read and written once. A workgroup of 16 waves takes a
// (sequence, head): a wave's load covers rows of V columns, 16 bytes a lane, and
// 4 loads of a lane the state. Unlike the delta rule, a row's update needs
// nothing but the row, so each piece is written back as soon as it has arrived,
// and only the output waits for the sum over the rows. 64 sequences of 32 heads of
// 128 x 128 are 272 MB: 48.6 us, 5.6 TB/s, as against 46 at the rate at which a large tensor
// is scaled in place (5.9). (8 waves: 49.3, or 50.9 for half of the columns each; 4 waves
// 50.4; 200 sequences 148, 154, 156 and 155.) One sequence takes 4.5 us on the card (halves: 4.1), and
// 12 with the call.
#include "kda_lin_device.h"

namespace kda {
namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = kLinDecodeThreads / 64;

// Nontemporal: a state is touched once per step, and the caches of a model's layers exceed the
// Infinity Cache (measured for the same access in kda_decode.hip).
template <int K, int V, typename TIn, typename TOut>
__global__ __launch_bounds__(64 * kWaves) void lin_decode_kernel(LinArgs a) {
    constexpr int LPR = V / 4, RPI = 64 / LPR, ITERS = K / (kWaves * RPI);
    static_assert(ITERS * kWaves * RPI == K && K <= 64 * kWaves, "rows are covered by the waves' loads");
    __shared__ float2 kq[K];
    __shared__ f4 red[kWaves][LPR];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int c4 = lane % LPR, rsub = lane / LPR;
    const int bh = blockIdx.x, col0 = 4 * c4;
    const int b = bh / a.H, h = bh - b * a.H, hk = h / (a.H / a.Hk);
    float ki = 0.f, qi = 0.f;
    if (tid < K) {
        ki = io<TIn>::load(static_cast<const TIn *>(a.k) + b * a.ks + hk * K + tid);
        qi = io<TIn>::load(static_cast<const TIn *>(a.q) + b * a.qs + hk * K + tid);
    }
    const float4 v = io<TIn>::load4(static_cast<const TIn *>(a.v) + b * a.vs + h * V + col0);
    const float g = log_decay(a.g[b * a.gs + h]);
    const int slot = slot_of(a, b);
    float *S = a.sT + (static_cast<int64_t>(slot) * a.H + h) * (K * V) + col0;
    f4 s[ITERS];
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int row = (i * kWaves + w) * RPI + rsub;
        s[i] = slot >= 0 ? __builtin_nontemporal_load(reinterpret_cast<const f4 *>(S + row * V)) : f4{0.f, 0.f, 0.f, 0.f};
    }
    if (tid < K) kq[tid] = make_float2(ki, qi);
    const float d = __expf(g);
    const f4 vv = {v.x, v.y, v.z, v.w};
    __syncthreads();
    f4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < ITERS; ++i) {
        const int row = (i * kWaves + w) * RPI + rsub;
        const float2 x = kq[row];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(x.x, vv[j], d * s[i][j]);
            o[j] = fmaf(x.y, s[i][j], o[j]);
        }
        if (slot >= 0) __builtin_nontemporal_store(s[i], reinterpret_cast<f4 *>(S + row * V));
    }
#pragma unroll
    for (int m = LPR; m < 64; m <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] += __shfl_xor(o[j], m);
    if (rsub == 0) red[w][c4] = o;
    __syncthreads();
    if (tid < LPR) {
        o = red[0][tid];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) o += red[i][tid];
        TOut *out = static_cast<TOut *>(a.o) + static_cast<int64_t>(bh) * V + col0;
#pragma unroll
        for (int j = 0; j < 4; ++j) store_out(out + j, a.scale * o[j]);
    }
}

template <int K, int V> hipError_t launch_dims(const LinArgs &a, hipStream_t st) {
    const dim3 grid(a.N * a.H), block(64 * kWaves);
    if (a.in_dtype == KDA_F32)
        hipLaunchKernelGGL((lin_decode_kernel<K, V, float, float>), grid, block, 0, st, a);
    else if (a.out_dtype == KDA_BF16)
        hipLaunchKernelGGL((lin_decode_kernel<K, V, bf16_t, bf16_t>), grid, block, 0, st, a);
    else
        hipLaunchKernelGGL((lin_decode_kernel<K, V, bf16_t, float>), grid, block, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_decode(const LinArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace kda
