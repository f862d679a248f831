// Causal attention inside packed sequences (kda_attn_fwd).
//
// A workgroup takes one tile of R rows of a (sequence, kv head), row r being
// token r / G and query head r % G, and streams the keys and values up to the
// tile's last token. fp32 inputs take tiles of 16 rows of the streaming form
// (kda_attn_stream.h), two workgroups to a compute unit: 71 us for prompts of
// 1000, 37 and 411 tokens, H = 16, Hk = 4, d = 128 (tiles of 32 rows, whose registers leave
// room for one workgroup, were a sixth slower). Each of them stages all its keys and values
// through registers for those 16 rows, which is what it waits for beside its products.
#include "kda_attn_rows.h"
#include "kda_attn_stream.h"

namespace kda {
namespace {

template <int K, int V>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_prompt_kernel(AttnArgs a, int slots) {
    using S = Stream<K, V, float>;
    constexpr int R = S::R;
    __shared__ __align__(16) char lds[S::kLds];
    __shared__ float stat[2][kWaves][R];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    char *lk = lds + w * (S::KB + S::VB), *lv = lk + S::KB;

    const int kvh = blockIdx.x % a.Hk;
    const int64_t slot = slots - 1 - static_cast<int>(blockIdx.x / a.Hk);  // the longest first
    const int n = seq_of_slot(a.cu, a.N, a.T, a.G, R, slot, lane);
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
    const uint32_t none[S::NB] = {};
    auto &ahead = st.next;
    if (w * S::kStepWave < last) S::load_packed(ahead, a, start, kvh, w * S::kStepWave, lane);
    for (int p0 = w * S::kStepWave; p0 < last; p0 += S::kStep) {
        const bool masked = p0 + S::kStepWave > open;
        uint32_t sees = 0;
        if (masked) sees = st.visible(a, start, r0, rows, p0, 0, count, ahead.here, lane);
        const bool odd = S::stage(ahead, lk, lv, masked, p0, count, lane);
        if (p0 + S::kStep < last) S::load_packed(ahead, a, start, kvh, p0 + S::kStep, lane);
        __builtin_amdgcn_wave_barrier();
        st.step(lk, lv, a.c, masked, sees, odd, none, none, lane);
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    st.join(lds, stat, w, lane, rows, [&](int row, int ch, float m, f32x4 x, float l) {
        store_out(a, start, kvh, r0 + row, ch, m, x, l);
    });
}

// ---- bf16
//
// NW = 8 waves of 32 rows each share tiles of 64 keys and values in LDS, copied there
// directly from memory ahead of their use (two buffers each). Where there are too few
// rows for all compute units (halves()), a tile is 128 keys and values, its PARTS = 2
// halves go to one half of the waves each, both with the same rows, and their maxima,
// sums and outputs are joined in LDS in the end.
//
// What bounds it: at d = 128 the matrix cores (2 L^2 d H operations for L tokens)
// under the card's power limit: 7.3 to 8.0 ms by the card's state for one prompt of 32768, H =
// 32, Hk = 8 (1200 to 1100 TFLOP/s; a large library product reaches 1385). At d = 64 the softmax's
// latencies: its vector instructions per score are the same for half the products, one of a
// SIMD's two waves issues them at a time, and neither pipe is full (59 % and 32 %): 185 to 198 us
// for 4 x 4096, H = Hk = 16 (740 to 690 TFLOP/s). Short prompts add each workgroup's start and its
// store, which nothing overlaps here: 409 to 434 us for 16 prompts of 217 to 3448 tokens, H = 32
// (860 to 810 TFLOP/s).

constexpr int NW = 8;

// Copies of the tiles of keys or values (D channels), in order: 64 rows from the next one on
// to LDS at dst.
template <typename R, int D, bool KEYS> struct Copier {
    static constexpr int C = D / 8, N = kTile * D * 2 / (1024 * NW);
    static_assert(N >= 1, "a tile is at least one copy per wave");
    const bf16_t *next;
    int64_t stride;
    int left;         // rows that the packed tensor has from `next` on
    uint32_t off[N];  // this lane's, for 64 rows that are all there

    __device__ __forceinline__ void begin(const bf16_t *src, int64_t stride_, int row, int T, int w, int lane) {
        next = src + row * stride_;
        stride = stride_;
        left = T - row;
#pragma unroll
        for (int i = 0; i < N; ++i) off[i] = place(i, kTile - 1, w, lane);
    }
    // bytes of chunk i from row 0, rows past `top` replaced by it: less than 2^31, strides are at most 2^24 elements
    __device__ __forceinline__ uint32_t place(int i, int top, int w, int lane) const {
        const int e = (i * NW + w) * 64 + lane, t = e / C, c = (e % C) ^ (KEYS ? R::swz_k(t) : R::swz_v(t));
        return 2 * (static_cast<uint32_t>(min(t, top)) * static_cast<uint32_t>(stride) + 8 * c);
    }
    __device__ __forceinline__ void tile(uint32_t dst, int w, int lane) {
        if (left >= kTile) {
#pragma unroll
            for (int i = 0; i < N; ++i) copy_to_lds(dst + (i * NW + w) * 1024, next, off[i]);
        } else {  // behind the tensor's end: its last row
            const bf16_t *from = next + min(left - 1, 0) * stride;
#pragma unroll
            for (int i = 0; i < N; ++i) copy_to_lds(dst + (i * NW + w) * 1024, from, place(i, max(left - 1, 0), w, lane));
        }
        next += kTile * stride;
        left -= kTile;
    }
};

template <int K, int V, int PARTS>
__global__ __launch_bounds__(64 * NW, 2) void attn_prompt_bf16_kernel(AttnArgs a, int slots) {
    using P = Rows<K, V>;
    constexpr int R = 32 * NW / PARTS, kTurn = PARTS * kTile;  // rows; tokens of a tile
    constexpr int KB = PARTS * P::KB, VB = PARTS * P::VB;
    __shared__ __align__(1024) char lds[2 * (KB + VB)];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int kvh = blockIdx.x % a.Hk;
    // The longest first, sequence by sequence: the tiles at work at a time then share their keys and
    // values in L2 (taking the longest tiles of all sequences first was slower: 421 against 400 us
    // for 16 prompts of 200 to 4000 tokens).
    const int64_t slot = slots - 1 - static_cast<int>(blockIdx.x / a.Hk);
    const int n = seq_of_slot(a.cu, a.N, a.T, a.G, R, slot, lane);
    int start, count;
    seq_rows(a.cu, n, a.T, start, count);
    const int64_t first = (slot - static_cast<int64_t>(start) * a.G / R - n) * R, all = static_cast<int64_t>(count) * a.G;
    if (first < 0 || first >= all) return;
    const int last = static_cast<int>((min(first + R, all) - 1) / a.G);  // last token of the tile

    // this wave's rows; rows past the sequence's repeat its last one and are not stored
    const int part = PARTS == 1 ? 0 : w / (NW / PARTS), shift = part * kTile;  // its tokens of a tile
    const int64_t wr0 = first + 32 * (w - part * (NW / PARTS)), wr1 = min(wr0 + 32, all);
    const bool some = wr0 < all;
    const int tok1 = static_cast<int>((max(wr1, static_cast<int64_t>(1)) - 1) / a.G);
    const int64_t row = min(wr0 + (lane & 31), all - 1);
    const int own = static_cast<int>(row / a.G), h = kvh * a.G + static_cast<int>(row - static_cast<int64_t>(own) * a.G);

    P st;
    const float c = fabsf(a.c);
    st.reset();

    const uint32_t base = lds_address(lds);
    // LDS: keys of even and odd tiles, values of even and odd tiles
    auto lk = [&](int j) { return (j & 1) * KB; };
    auto lv = [&](int j) { return 2 * KB + (j & 1) * VB; };
    const char *const own_k = lds + part * P::KB, *const own_v = lds + part * P::VB;
    Copier<P, K, true> kc;
    Copier<P, V, false> vc;
    kc.begin(static_cast<const bf16_t *>(a.k) + kvh * K, a.ks, start, a.T, w, lane);
    vc.begin(static_cast<const bf16_t *>(a.v) + kvh * V, a.vs, start, a.T, w, lane);
    // The two waves of a SIMD take turns: one is in its products (the values of the tile before,
    // the scores of this one) while the other is in its softmax, and every barrier swaps them.
    // Copies for a tile are issued two turns before its first use, which is when the last reader
    // of that buffer has gone; those of tile 0's values and tile 1's keys at the start. The first
    // J tiles are seen whole by every row of the workgroup.
    const int J = (static_cast<int>(first / a.G) + 1) / kTurn, tiles = last / kTurn + 1;
    const bool ahead = w < NW / 2;
    auto copy_k = [&](int j) {
        if (j >= tiles) return;
#pragma unroll
        for (int i = 0; i < PARTS; ++i) kc.tile(base + lk(j) + i * P::KB, w, lane);
    };
    auto copy_v = [&](int j) {
        if (j >= tiles) return;
#pragma unroll
        for (int i = 0; i < PARTS; ++i) vc.tile(base + lv(j) + i * P::VB, w, lane);
    };
    auto swap = [&](bool wait) {
        if (wait) wait_copies();
        phase_barrier();
    };
    auto sees = [&](int j) { return some && j * kTurn + shift <= tok1; };  // the wave has work in tile j
    copy_k(0);
    st.load_q(static_cast<const bf16_t *>(a.q) + static_cast<int64_t>(start + own) * a.qs + h * K, a.c < 0.f, lane);
    copy_v(0);
    copy_k(1);
    // tile 0's keys; a call of one tile has no copies of tile 1 behind them
    if (tiles > 1) wait_copies<PARTS * (Copier<P, V, false>::N + Copier<P, K, true>::N)>();
    else wait_copies<PARTS * Copier<P, V, false>::N>();
    phase_barrier();
    if (!ahead) swap(false);
    // The wave in its products issues first where they are the longer turn (two heads of 64
    // channels have half the products for the same softmax): 7.27 against 7.41 ms for 32768
    // tokens at 128 channels, and 191 against 188 us for 4 x 4096 at 64.
    constexpr bool kProductsFirst = K + V > 128;
    int j = 0;
    for (; j < J; ++j) {
        if (ahead && j > 0) {
            copy_k(j + 1);
            copy_v(j);
        }
        if (kProductsFirst) __builtin_amdgcn_s_setprio(1);
        if (j > 0) {
            st.values(own_v + lv(j - 1), lane);
            st.scores(own_k + lk(j), lane);
            P::template interleave<true>();
        } else {
            st.scores(own_k + lk(0), lane);
            P::template interleave<false>();
        }
        if (kProductsFirst) __builtin_amdgcn_s_setprio(0);
        swap(!ahead);
        if (!ahead) {
            copy_k(j + 2);
            copy_v(j + 1);
        }
        st.template softmax<false>(c, 0);
        swap(ahead);
    }
    uint32_t seen = ~0u;  // of tile j - 1
    for (; j < tiles; ++j) {
        if (ahead && j > 0) {
            copy_k(j + 1);
            copy_v(j);
        }
        if (j > 0 && sees(j - 1)) st.values_masked(own_v + lv(j - 1), seen, lane);
        if (sees(j)) st.scores(own_k + lk(j), lane);
        swap(!ahead);
        if (!ahead) {
            copy_k(j + 2);
            copy_v(j + 1);
        }
        if (sees(j)) {
            seen = P::of_lane(low_bits(own - j * kTurn - shift + 1), lane);
            st.template softmax<true>(c, seen);
        }
        swap(ahead);
    }
    if (sees(j - 1)) st.values_masked(own_v + lv(j - 1), seen, lane);
    if (ahead) swap(false);
    float l = swap32_sum(st.l);
    if (PARTS == 2) {
        // the later part's rows are added to the first's, in LDS: [V / 4][R] of four channels, then m and l
        f32x4 *const ro = reinterpret_cast<f32x4 *>(lds);
        float *const rm = reinterpret_cast<float *>(lds + R * V * 4), *const rl = rm + R;
        const int at = (w & (NW / 2 - 1)) * 32 + (lane & 31);
        phase_barrier();  // all are done with the tiles
        if (part == 1) {
            st.each(lane, [&](int ch, f32x4 x) { ro[(ch >> 2) * R + at] = x; });
            if (lane < 32) {
                rm[at] = st.m;
                rl[at] = l;
            }
        }
        phase_barrier();
        if (part == 1) return;
        const float m = fmaxf(st.m, rm[at]);
        const float f = m == -INFINITY ? 1.f : exp2f(st.m - m), g = m == -INFINITY ? 1.f : exp2f(rm[at] - m);
        l = l * f + rl[at] * g;
        if (wr0 + (lane & 31) >= all) return;
        st.each(lane, [&](int ch, f32x4 x) {
            store_out(a, start, kvh, static_cast<int>(row), ch, m, x * f + ro[(ch >> 2) * R + at] * g, l);
        });
        return;
    }
    if (wr0 + (lane & 31) >= all) return;
    st.each(lane, [&](int ch, f32x4 x) { store_out(a, start, kvh, static_cast<int>(row), ch, st.m, x, l); });
}

template <int K, int V, int PARTS> hipError_t launch_bf16(const AttnArgs &a, hipStream_t st) {
    const int64_t slots = static_cast<int64_t>(a.T) * a.G / (32 * NW / PARTS) + a.N;
    hipLaunchKernelGGL((attn_prompt_bf16_kernel<K, V, PARTS>), dim3(static_cast<unsigned>(slots * a.Hk)), dim3(64 * NW), 0, st, a,
                       static_cast<int>(slots));
    return hipGetLastError();
}

template <int K, int V>
hipError_t launch_f32(const AttnArgs &a, hipStream_t st) {
    const int64_t slots = static_cast<int64_t>(a.T) * a.G / Stream<K, V, float>::R + a.N;
    hipLaunchKernelGGL((attn_prompt_kernel<K, V>), dim3(static_cast<unsigned>(slots * a.Hk)), dim3(64 * kWaves), 0, st,
                       a, static_cast<int>(slots));
    return hipGetLastError();
}

// Whether tiles of 128 rows, whose keys two halves of the workgroup share, are faster than tiles
// of 256 rows. They halve what a workgroup walks, which is what a call takes whose tiles all run
// at once, but each row's share of the copies is twice as large. `tiles`: about how many there
// are of 128 rows, some of them cut short by the sequences' ends. Up to 9/8 to a compute unit
// they were faster throughout (whole against halves, us, H = 8, Hk = 2, d = 128: 1 x 1000 30 and
// 22, 1 x 3500 81 and 53, 4 x 1100 35 and 27; H = 32, Hk = 8: 1 x 65 10.9 and 9.5, 1 x 1100 36
// and 26); up to two they were if the walks are long (H = 32: 1 x 1500 46 and 38, 1 x 2000 58
// and 51; H = 8: 1 x 8000 181 and 140; but 16 x 300 18 and 25); beyond, they were slower (H =
// 32: 1 x 3500 109 and 123, 4 x 1100 66 and 81). (At d_k = 64, d_v = 128 the halves' form spills 10
// registers; 1 x 1100, H = 32 takes 21 us there, between 17 at 64 / 64 and 23 at 128 / 128.)
bool halves(const AttnArgs &a) {
    const int64_t units = compute_units(), tiles = (static_cast<int64_t>(a.T) * a.G / 64 + a.N) * a.Hk / 2;
    return 8 * tiles <= 9 * units || (tiles <= 2 * units && a.T >= static_cast<int64_t>(1024) * a.N);
}

template <int K, int V> hipError_t launch_dims(const AttnArgs &a, hipStream_t st) {
    if (a.in_dtype == KDA_F32) return launch_f32<K, V>(a, st);
    return halves(a) ? launch_bf16<K, V, 2>(a, st) : launch_bf16<K, V, 1>(a, st);
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace kda
