// Attention of new tokens over the paged cache (kda_attn_cache_fwd).
//
// The cache is what the call has to read, so it is read once: a workgroup
// takes all rows of a (sequence, kv head), the new tokens times the query heads
// of the group, in tiles of R rows, over a run of steps of 128 cached tokens.
//
// Split. Sequences differ in length and only the device knows it, so the steps
// of all (sequence, kv head, row tile)s are laid on one line and each of W
// workgroups takes an equal piece of it. A (sequence, kv head, row tile) that
// one workgroup covers is finished there; otherwise each piece leaves its
// maximum, sum and unnormalised output in the workspace, and a second kernel
// joins them in the order of the line, so results do not depend on timing.
#include "kda_attn_stream.h"

namespace kda {
namespace {

// Sequence n's place on the line.
struct Seq {
    int start, count;  // its new tokens
    int ctx, end;      // tokens before them (may be below 0), cached tokens within the page table
    int tiles, steps;  // row tiles; steps per row tile
    __device__ __forceinline__ int64_t units(int Hk) const { return static_cast<int64_t>(Hk) * tiles * steps; }
};

__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int n, int R) {
    Seq s;
    seq_rows(a.cu, n, a.T, s.start, s.count);
    const int len = max(ld_meta(a.lens, n), 0);
    s.ctx = len - s.count;
    s.end = min(len, a.max_pages << a.page_shift);
    s.tiles = static_cast<int>((static_cast<int64_t>(s.count) * a.G + R - 1) / R);
    s.steps = max((s.end + kStep - 1) / kStep, 1);  // at least one, which writes the rows
    return s;
}

// A workgroup takes at least kMinSteps steps where the line is short, so that a
// short cache is not cut into pieces that cost more to join than to read.
constexpr int kMinSteps = 2;
__device__ __forceinline__ int64_t line_workgroups(int64_t U, int W) {
    const int64_t w = (U + kMinSteps - 1) / kMinSteps;
    return w < W ? max(w, static_cast<int64_t>(1)) : W;
}
__device__ __forceinline__ int64_t line_begin(int64_t w, int64_t U, int64_t W) { return w * U / W; }
__device__ __forceinline__ int64_t line_owner(int64_t u, int64_t U, int64_t W) { return ((u + 1) * W - 1) / U; }

__device__ __forceinline__ int64_t wave_scan(int64_t x, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int lo = __shfl_up(static_cast<int>(x & 0xFFFFFFFFll), d), hi = __shfl_up(static_cast<int>(x >> 32), d);
        if (lane >= d) x += (static_cast<int64_t>(hi) << 32) | static_cast<uint32_t>(lo);
    }
    return x;
}

// Workspace: prefix of the line [N + 1] int64, then 2 W partial tiles. A
// workgroup has at most two pieces that are not whole, its first and its last.
__host__ __device__ inline size_t part_floats(int R, int V) { return static_cast<size_t>(R) * (V + 2); }
__host__ __device__ inline size_t prefix_bytes(int N) { return (static_cast<size_t>(N) + 1) * 8 + 255 & ~static_cast<size_t>(255); }

// Total of the line, and the sequence that holds unit u with the units before it. Workgroup-uniform.
// Every thread of the workgroup calls it. prefix: written if not nullptr.
template <int R> struct Line {
    int64_t total;
    __device__ __forceinline__ void scan(const AttnArgs &a, int tid, int64_t (&sh)[kWaves], int64_t *prefix) {
        const int lane = tid & 63, w = tid >> 6;
        int64_t base = 0;
        for (int n0 = 0; n0 < a.N; n0 += 64 * kWaves) {
            const int n = n0 + tid;
            const int64_t mine = n < a.N ? seq_of(a, min(n, a.N - 1), R).units(a.Hk) : 0;
            const int64_t inc = wave_scan(mine, lane);
            if (lane == 63) sh[w] = inc;
            __syncthreads();
            int64_t before = base, all = 0;
#pragma unroll
            for (int u = 0; u < kWaves; ++u) {
                if (u < w) before += sh[u];
                all += sh[u];
            }
            if (prefix && n < a.N) prefix[n] = before + inc - mine;
            base += all;
            __syncthreads();
        }
        total = base;
        if (prefix && tid == 0) prefix[a.N] = base;
    }
    // the sequence that holds unit u < total, and the line before it
    __device__ __forceinline__ void find(const AttnArgs &a, int64_t u, int tid, int64_t (&sh)[kWaves], int &n_of,
                                         int64_t &before_of, int &sh_n, int64_t &sh_before) const {
        const int lane = tid & 63, w = tid >> 6;
        int64_t base = 0;
        for (int n0 = 0; n0 < a.N; n0 += 64 * kWaves) {
            const int n = n0 + tid;
            const int64_t mine = n < a.N ? seq_of(a, min(n, a.N - 1), R).units(a.Hk) : 0;
            const int64_t inc = wave_scan(mine, lane);
            if (lane == 63) sh[w] = inc;
            __syncthreads();
            int64_t before = base, all = 0;
#pragma unroll
            for (int x = 0; x < kWaves; ++x) {
                if (x < w) before += sh[x];
                all += sh[x];
            }
            before += inc - mine;
            if (before <= u && u < before + mine) {
                sh_n = n;
                sh_before = before;
            }
            base += all;
            __syncthreads();
            if (u < base) break;
        }
        n_of = __builtin_amdgcn_readfirstlane(sh_n);
        before_of = sh_before;
    }
};

template <int K, int V, int RT, typename TC>
__global__ __launch_bounds__(64 * kWaves) void attn_cache_kernel(AttnArgs a) {
    using S = Stream<K, V, RT, TC>;
    constexpr int R = S::R;
    __shared__ __align__(16) char lds[S::kLds];
    __shared__ float stat[2][kWaves][R];
    __shared__ int64_t sh[kWaves];
    __shared__ int sh_n;
    __shared__ int64_t sh_before;
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    char *lk = lds + w * (S::KB + S::VB), *lv = lk + S::KB;

    Line<R> line;
    line.scan(a, tid, sh, blockIdx.x == 0 ? static_cast<int64_t *>(a.ws) : nullptr);
    const int64_t U = line.total;
    if (U == 0) return;
    const int64_t W = line_workgroups(U, a.W);
    if (static_cast<int64_t>(blockIdx.x) >= W) return;
    int64_t u = line_begin(blockIdx.x, U, W);
    const int64_t u_end = line_begin(blockIdx.x + 1, U, W);
    if (u >= u_end) return;
    int n;
    int64_t before;
    line.find(a, u, tid, sh, n, before, sh_n, sh_before);
    Seq q = seq_of(a, n, R);
    bool first = true;

    S st;
    while (u < u_end) {
        while (u >= before + q.units(a.Hk)) {  // the next sequence with work: there is one, u < U
            before += q.units(a.Hk);
            q = seq_of(a, ++n, R);
        }
        const int64_t in = u - before;
        const int item = static_cast<int>(in / q.steps), t0 = static_cast<int>(in - static_cast<int64_t>(item) * q.steps);
        const int t1 = static_cast<int>(min(static_cast<int64_t>(q.steps), t0 + (u_end - u)));
        const int kvh = item / q.tiles, r0 = (item - kvh * q.tiles) * R;
        const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(q.count) * a.G - r0));
        const bool whole = t0 == 0 && t1 == q.steps;
        const int tok0 = r0 / a.G, tok1 = (r0 + rows - 1) / a.G;
        // tokens below `open` are seen by all rows, none from `last` on is seen by any
        const int open = min(q.end, a.mask ? q.ctx : q.ctx + tok0 + 1);
        const int last = min(q.end, a.mask ? q.end : q.ctx + tok1 + 1);

        st.reset();
        st.load_q(a, q.start, kvh, r0, rows, lane);
        int pg[2], pn[2];
        const int32_t *table = a.table + static_cast<int64_t>(n) * a.max_pages;
        auto pages = [&](int t, int (&p)[2]) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int pos = t * kStep + w * kStepWave + 16 * b;
                const int id = pos < last ? ld_meta(table, pos >> a.page_shift) : -1;
                p[b] = id < a.num_pages ? id : -1;
            }
        };
        pages(t0, pg);
        if (t0 * kStep + w * kStepWave < last) st.load_cache(a, kvh, t0 * kStep + w * kStepWave, pg, lane);
        for (int t = t0; t < t1; ++t) {
            const int p0 = t * kStep + w * kStepWave;
            if (p0 >= last) break;  // wave-uniform; later steps lie further on
            const bool here[2] = {pg[0] >= 0, pg[1] >= 0};
            const bool masked = p0 + kStepWave > open || !here[0] || !here[1];
            const uint32_t kx[2] = {st.ke[0], st.ke[1]}, vx[2] = {st.ve[0], st.ve[1]};
            uint32_t sees[RT];
            if (masked) st.visible(sees, a, q.start, r0, rows, p0, q.ctx, q.end, here, lane);
            const bool odd = st.stage(lk, lv, masked, p0, q.end, here, lane);
            pages(t + 1 < t1 ? t + 1 : t, pn);
            if (t + 1 < t1 && p0 + kStep < last) st.load_cache(a, kvh, p0 + kStep, pn, lane);
            pg[0] = pn[0];
            pg[1] = pn[1];
            __builtin_amdgcn_wave_barrier();
            st.step(lk, lv, a.c, masked, sees, odd, kx, vx, lane);
            __builtin_amdgcn_wave_barrier();
        }
        __syncthreads();  // the join takes the waves' LDS
        if (whole) {
            st.join(lds, stat, w, lane, rows, [&](int row, int ch, float, f32x4 x, float l) {
                store_out(a, q.start, kvh, r0 + row, ch, x, l);
            });
        } else {
            float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + prefix_bytes(a.N)) +
                          (2 * static_cast<size_t>(blockIdx.x) + (first ? 0 : 1)) * part_floats(R, V);
            st.join(lds, stat, w, lane, rows, [&](int row, int ch, float m, f32x4 x, float l) {
                *reinterpret_cast<f32x4 *>(part + row * V + ch) = x;
                if (ch == 0) {
                    part[R * V + row] = m;
                    part[R * V + R + row] = l;
                }
            });
        }
        first = false;
        u += t1 - t0;
    }
}

// One workgroup per output row (token, query head): joins the pieces of its
// (sequence, kv head, row tile) if the line was cut inside it.
constexpr int kJoinThreads = 256;
template <int V, int R>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a) {
    constexpr int LPR = V / 4, GR = kJoinThreads / LPR;
    __shared__ __align__(16) f32x4 red[GR][LPR];
    __shared__ float red_l[GR], red_m[kJoinThreads / 64];
    const int tid = threadIdx.x;
    const int tok = blockIdx.x / a.H, h = blockIdx.x - tok * a.H, kvh = h / a.G;
    const int n = seq_of_token(a.cu, a.N, tok);
    const Seq q = seq_of(a, n, R);
    if (tok < q.start || tok >= q.start + q.count) return;
    const int64_t *prefix = static_cast<const int64_t *>(a.ws);
    const int64_t U = prefix[a.N], W = line_workgroups(U, a.W);
    const int r = (tok - q.start) * a.G + (h - kvh * a.G), tile = r / R, row = r - tile * R;
    const int64_t s = prefix[n] + (static_cast<int64_t>(kvh) * q.tiles + tile) * q.steps, e = s + q.steps;
    const int64_t w0 = line_owner(s, U, W), w1 = line_owner(e - 1, U, W);
    if (w0 == w1) return;
    const float *parts = reinterpret_cast<const float *>(static_cast<const char *>(a.ws) + prefix_bytes(a.N));
    auto part = [&](int64_t w) {
        const bool last = w == w0 && line_begin(w0, U, W) < s;  // w0 had other work before this
        return parts + (2 * w + (last ? 1 : 0)) * part_floats(R, V);
    };
    float m = -INFINITY;
    for (int64_t w = w0 + tid; w <= w1; w += kJoinThreads) m = fmaxf(m, part(w)[R * V + row]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    if ((tid & 63) == 0) red_m[tid >> 6] = m;
    __syncthreads();
    m = red_m[0];
#pragma unroll
    for (int i = 1; i < kJoinThreads / 64; ++i) m = fmaxf(m, red_m[i]);
    const int gr = tid / LPR, c = tid % LPR;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int64_t w = w0 + gr; w <= w1; w += GR) {
        const float *p = part(w);
        const float mw = p[R * V + row], f = mw == -INFINITY ? 0.f : exp2f(mw - m);
        x += *reinterpret_cast<const f32x4 *>(p + row * V + 4 * c) * f;
        l += p[R * V + R + row] * f;
    }
    red[gr][c] = x;
    if (c == 0) red_l[gr] = l;
    __syncthreads();
    if (gr == 0) {
#pragma unroll
        for (int i = 1; i < GR; ++i) {
            x += red[i][c];
            l += red_l[i];
        }
        store_out(a, q.start, kvh, r, 4 * c, x, l);
    }
}

// Rows per tile by the call's mean rows per (sequence, kv head). More rows than that
// cost registers and products on rows that do not exist; fewer read the cache again.
int row_blocks(int64_t T, int64_t N, int64_t G, bool f32) {
    const int64_t rows = (T + N - 1) / N * G;
    if (rows <= 16) return 1;
    return rows <= 32 || f32 ? 2 : 4;
}

template <int K, int V, int RT, typename TC>
hipError_t launch_rt(const AttnArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((attn_cache_kernel<K, V, RT, TC>), dim3(a.W), dim3(64 * kWaves), 0, st, a);
    hipError_t e = hipGetLastError();
    // one step per (sequence, kv head, row tile) at most: the line is never cut inside one
    if (e != hipSuccess || (a.max_pages << a.page_shift) <= kStep) return e;
    hipLaunchKernelGGL((attn_join_kernel<V, 16 * RT>), dim3(static_cast<unsigned>(a.T) * a.H), dim3(kJoinThreads), 0, st, a);
    return hipGetLastError();
}

template <int K, int V> hipError_t launch_dims(const AttnArgs &a, hipStream_t st) {
    const int rt = row_blocks(a.T, a.N, a.G, a.in_dtype == KDA_F32);
    if (a.kv_dtype == KDA_KV_F32) return rt == 1 ? launch_rt<K, V, 1, float>(a, st) : launch_rt<K, V, 2, float>(a, st);
    if (a.kv_dtype == KDA_KV_BF16)
        return rt == 1 ? launch_rt<K, V, 1, bf16_t>(a, st) : rt == 2 ? launch_rt<K, V, 2, bf16_t>(a, st)
                                                                    : launch_rt<K, V, 4, bf16_t>(a, st);
    return rt == 1 ? launch_rt<K, V, 1, e4m3_t>(a, st) : rt == 2 ? launch_rt<K, V, 2, e4m3_t>(a, st)
                                                                : launch_rt<K, V, 4, e4m3_t>(a, st);
}

}  // namespace

int32_t attn_cache_workgroups() { return 2 * compute_units(); }

size_t attn_cache_workspace(int32_t N, int32_t T, int32_t H, int32_t Hk, int32_t V, kda_dtype_t in_dtype) {
    const int R = 16 * row_blocks(T, N, H / Hk, in_dtype == KDA_F32);
    return prefix_bytes(N) + 2 * static_cast<size_t>(attn_cache_workgroups()) * part_floats(R, V) * sizeof(float);
}

hipError_t launch_attn_cache(const AttnArgs &args, hipStream_t st) {
    AttnArgs a = args;
    a.W = attn_cache_workgroups();
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace kda
