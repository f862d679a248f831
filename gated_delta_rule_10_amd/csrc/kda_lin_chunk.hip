// Linear attention with one decay per head over packed prompts (kda_lin_chunk_fwd).
//
// A workgroup walks a segment of a sequence for one value head, chunk by chunk,
// with the state in registers (kda_lin_bf16.h). A sequence is one segment where
// there are enough sequences and heads to fill the card; otherwise it is cut, and
// two more launches come before: one walks all segments but each sequence's last
// from a state of zeros (the first from the initial state) to their ends, without
// outputs, and one joins these, a segment's state being the one before it times
// e^(its sum of g), plus its own. They read k and v a second time, and are worth
// it where a few sequences would leave the card empty.
#include "kda_attn_internal.h"
#include "kda_lin_bf16.h"
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

constexpr double kLog2e = 1.4426950408889634;

// A segmented call's workspace: the states at the segments' starts (as the registers of a workgroup
// hold them, see fragment()), and the sums of log2 e^g over them.
struct Segments {
    float *state;
    double *sum;
};

template <typename W, typename TOut, int K, int V>
__global__ __launch_bounds__(W::NT, W::kWavesPerSimd) void lin_segments_kernel(LinArgs a, Segments ws, int R) {
    using T = typename W::T;
    constexpr int C = W::C;
    constexpr bool OUT = W::OUT;
    __shared__ __align__(16) char lds[W::kLds];
    __shared__ __align__(16) float table[2][4][C];
    __shared__ int strange[2];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int place = blockIdx.x / a.H, h = blockIdx.x - place * a.H, hk = h / (a.H / a.Hk);
    const int n = seq_of_slot(a.cu, a.N, a.T, 1, R, place, lane);
    int start, count;
    seq_rows(a.cu, n, a.T, start, count);
    const int seg = place - (start / R + n), segs = max(1, (count + R - 1) / R);
    if (seg < 0 || seg >= segs || (!OUT && seg == segs - 1)) return;
    const int t0 = start + seg * R, tokens = min(R, count - seg * R), chunks = (tokens + C - 1) / C;
    const int slot = slot_of(a, n);
    const int64_t held = (static_cast<int64_t>(slot) * a.H + h) * (K * V);
    const int64_t piece = static_cast<int64_t>(place) * a.H + h;

    W s;
    s.clear();
    if (OUT && segs > 1) {
        s.get(ws.state + piece * (K * V), w, lane);
    } else if (seg == 0 && a.s0 && slot >= 0) {
#pragma unroll
        for (int m = 0; m < W::M; ++m)
#pragma unroll
            for (int r = 0; r < W::kRegs; ++r) s.S[m][r] = a.s0[held + W::element(m, r, w, lane)];
    }
    if (!OUT && seg == 0) s.put(ws.state + piece * (K * V), w, lane);

    const T *qp = static_cast<const T *>(a.q) + t0 * a.qs + hk * K, *kp = static_cast<const T *>(a.k) + t0 * a.ks + hk * K;
    const T *vp = static_cast<const T *>(a.v) + t0 * a.vs + h * V;
    TOut *op = static_cast<TOut *>(a.o) + (static_cast<int64_t>(t0) * a.H + h) * V;
    double sum = 0.0;  // of the segment's decays so far
    auto decay = [&](int c) { return lane < min(C, tokens - c * C) ? log_decay_of(a, t0 + c * C + lane, h) : 0.f; };
    auto tabulate = [&](float g, int b, int rows) {
        double x = static_cast<double>(g) * kLog2e;
#pragma unroll
        for (int d = 1; d < C; d <<= 1) {
            const double y = __shfl_up(x, d);
            x += lane >= d ? y : 0.0;
        }
        const double all = __shfl(x, C - 1);
        sum += all;
        if (lane < C) {
            const float hi = static_cast<float>(x);
            table[b][0][lane] = hi;
            table[b][1][lane] = static_cast<float>(x - static_cast<double>(hi));
            table[b][2][lane] = __builtin_amdgcn_exp2f(hi);
            table[b][3][lane] = lane < rows ? __builtin_amdgcn_exp2f(static_cast<float>(all - x)) : 0.f;
        }
        if (lane == 0) strange[b] = 0;
    };
    float g = 0.f;
    if (w == W::NW - 1 && chunks > 0) {
        tabulate(decay(0), 0, tokens);
        g = chunks > 1 ? decay(1) : 0.f;
    }
    if (chunks > 0) s.load(qp, kp, vp, a, min(C, tokens), tid);
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1, rows = min(C, tokens - c * C);
        __syncthreads();  // all have read the chunk before
        if (s.to_lds(lds, tid)) strange[b] = 1;
        auto next = [&] {
            qp += C * a.qs, kp += C * a.ks, vp += C * a.vs;
            if (c + 1 < chunks) s.load(qp, kp, vp, a, min(C, tokens - (c + 1) * C), tid);
        };
        __syncthreads();
        if (w == W::NW - 1 && c + 1 < chunks) {
            tabulate(g, b ^ 1, tokens - (c + 1) * C);
            if (c + 2 < chunks) g = decay(c + 2);
        }
        const Decays d = {table[b][0], table[b][1], table[b][2], table[b][3]};
        s.template chunk<TOut>(op, static_cast<int64_t>(a.H) * V, a.scale, lds, d, strange[b], rows, w, lane, next);
        op += static_cast<int64_t>(C) * a.H * V;
    }
    if (OUT) {
        if (seg == segs - 1 && a.sT && slot >= 0)
#pragma unroll
            for (int m = 0; m < W::M; ++m)
#pragma unroll
                for (int r = 0; r < W::kRegs; ++r) a.sT[held + W::element(m, r, w, lane)] = s.S[m][r];
    } else {
        s.put(ws.state + (piece + a.H) * (K * V), w, lane);  // the next segment's
        if (tid == W::NT - 1) ws.sum[piece] = sum;
    }
}

// The states at the starts of each sequence's segments from the third on: that of the one before,
// decayed over it, added to what it wrote itself. Four elements of the state to a thread.
template <int KV> __global__ __launch_bounds__(256) void lin_join_kernel(LinArgs a, Segments ws, int R) {
    constexpr int PER = KV / 4 / 256;
    const int e = (blockIdx.x % PER) * 256 + threadIdx.x, nh = blockIdx.x / PER, n = nh / a.H, h = nh - n * a.H;
    int start, count;
    seq_rows(a.cu, n, a.T, start, count);
    const int segs = (count + R - 1) / R;
    const int64_t piece = (static_cast<int64_t>(start / R) + n) * a.H + h;
    if (segs < 3) return;
    f32x4 *p = reinterpret_cast<f32x4 *>(ws.state + piece * KV) + e;
    const int64_t step = static_cast<int64_t>(a.H) * (KV / 4);
    f32x4 x = p[step];
    for (int g = 2; g < segs; ++g) {
        const float d = __builtin_amdgcn_exp2f(static_cast<float>(ws.sum[piece + static_cast<int64_t>(g - 1) * a.H]));
        const f32x4 own = p[g * step];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaf(d, x[i], own[i]);
        p[g * step] = x;
    }
}

// Tokens to a segment, and an upper bound of the segments: sequence n's begin at place
// cu[n] / R + n, so a place finds its sequence from cu alone.
struct Plan {
    int R;
    int64_t places;
    bool cut;
};
constexpr int kLeastChunks = 8;
Plan plan_of(int32_t N, int32_t T, int32_t H) {
    const int64_t chunks = static_cast<int64_t>(T) / 64 + N, groups = 2 * compute_units();
    const int64_t L = max(static_cast<int64_t>(kLeastChunks), (chunks * H + groups - 1) / groups);
    if (64 * L >= T) return {(T + 63) / 64 * 64 + 64, N, false};
    return {static_cast<int>(64 * L), T / (64 * L) + N, true};
}

template <int K, int V, typename TOut> hipError_t launch_bf16(const LinArgs &a, hipStream_t st) {
    const Plan p = plan_of(a.N, a.T, a.H);
    Segments ws{};
    if (p.cut) {
        ws.sum = static_cast<double *>(a.ws);
        ws.state = reinterpret_cast<float *>(static_cast<char *>(a.ws) + (p.places * a.H * 8 + 255) / 256 * 256);
    }
    const dim3 grid(static_cast<unsigned>(p.places * a.H)), block(LinBf16<K, V, 0>::NT);
    if (p.cut) {
        hipLaunchKernelGGL((lin_segments_kernel<LinBf16<K, V, 0>, float, K, V>), grid, block, 0, st, a, ws, p.R);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((lin_join_kernel<K * V>), dim3(a.N * a.H * (K * V / 1024)), dim3(256), 0, st, a, ws, p.R);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((lin_segments_kernel<LinBf16<K, V, sizeof(TOut) / 2>, TOut, K, V>), grid, block, 0, st, a, ws, p.R);
    return hipGetLastError();
}

template <int K, int V> hipError_t launch_dims(const LinArgs &a, hipStream_t st) {
    const dim3 grid(a.N * a.H), block(kThreads);
    if (a.in_dtype == KDA_F32)
        hipLaunchKernelGGL((lin_tokens_kernel<K, V, float, float>), grid, block, 0, st, a);
    else if (a.out_dtype == KDA_BF16)
        return launch_bf16<K, V, bf16_t>(a, st);
    else
        return launch_bf16<K, V, float>(a, st);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_chunk(const LinArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

size_t lin_chunk_workspace(int32_t N, int32_t T, int32_t H, int32_t K, int32_t V, kda_dtype_t in_dtype) {
    if (in_dtype != KDA_BF16) return 0;
    const Plan p = plan_of(N, T, H);
    if (!p.cut) return 0;
    return (static_cast<size_t>(p.places) * H * 8 + 255) / 256 * 256 + static_cast<size_t>(p.places) * H * K * V * 4;
}

}  // namespace kda
