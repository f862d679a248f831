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

// ---- bf16
//
// NW waves of 32 rows each share a tile of 64 keys and values in LDS, copied
// there directly from memory one tile ahead (two buffers). 32 x 32 matrix
// instructions, 16-deep: S^T = K Q^T leaves the scores of row l % 32 for tokens
// 32 b + 8 (i / 4) + 4 (l / 32) + i % 4 in register i of lane l, and those
// registers, rounded to bf16, are the B operand of O^T = V^T P^T when V^T's
// fragments take the tokens in the same order, which the transposing LDS reads
// do. P never moves between lanes.
__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16 bytes per lane from base (wave-uniform) + off to LDS at dst (wave-uniform) + 16 * lane. Unknown to the
// compiler's wait insertion: awaited by wait_copies() before a barrier.
__device__ __forceinline__ void copy_to_lds(uint32_t dst, const void *base, uint32_t off) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void wait_copies() { __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// One instruction, where fmaxf of two would first make quiet NaNs of its operands. A NaN
// operand is passed over, as by fmaxf.
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    __asm__("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(x), "v"(y), "v"(z));
    return r;
}

// A workgroup barrier that nothing is moved across, without waiting for copies.
__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

constexpr int kTile = 64;  // tokens per tile

template <int K, int V, int NW> struct Prompt {
    static constexpr int R = 32 * NW;
    static constexpr int CK = K / 8, CV = V / 8;            // 16-byte chunks per row
    static constexpr int KB = kTile * K * 2, VB = kTile * V * 2;
    static constexpr int KS = K / 16, DB = V / 32;
    static_assert(KB >= 1024 * NW && VB >= 1024 * NW, "a tile is at least one copy per wave");

    // chunk c of token t lies at chunk c ^ swz(t) of its row: the tokens that one read takes
    // the same chunk of are spread over the banks
    static __device__ __forceinline__ int swz_k(int t) { return CK == 16 ? t & 15 : (t >> 1) & 7; }
    static __device__ __forceinline__ int swz_v(int t) { return CV == 16 ? (t & 3) * 4 : ((t >> 1) & 1) * 4; }

    // Copies of the tiles of keys or values (D channels), in order: 64 rows from the next one on
    // to LDS at dst.
    template <int D, bool KEYS> struct Copier {
        static constexpr int C = D / 8, N = kTile * D * 2 / (1024 * NW);
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
            const int e = (i * NW + w) * 64 + lane, t = e / C, c = (e % C) ^ (KEYS ? swz_k(t) : swz_v(t));
            return 2 * (static_cast<uint32_t>(min(t, top)) * static_cast<uint32_t>(stride) + 8 * c);
        }
        __device__ __forceinline__ void tile(uint32_t dst, int w, int lane) {
            if (left >= kTile) {
#pragma unroll
                for (int i = 0; i < N; ++i) copy_to_lds(dst + (i * NW + w) * 1024, next, off[i]);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) copy_to_lds(dst + (i * NW + w) * 1024, next, place(i, left - 1, w, lane));
            }
            next += kTile * stride;
            left -= kTile;
        }
    };

    bf16x8 q[KS];
    f32x16 o[DB], s[2];
    bf16x8 p[4];
    float m, l;

    __device__ __forceinline__ void scores(const char *lk, int lane) {
        s[0] = s[1] = f32x16{};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int t = 32 * b + (lane & 31);
                const bf16x8 kf = *reinterpret_cast<const bf16x8 *>(lk + t * (2 * K) + 16 * ((2 * ks + (lane >> 5)) ^ swz_k(t)));
                s[b] = mma32(kf, q[ks], s[b]);
            }
    }

    // Order of the LDS reads (two per value fragment, one per key fragment) and products of a
    // values() [if VALUES] and scores() in a row: reads run kAhead products ahead of their use,
    // which covers their latency. Left to itself the compiler reads right before each product.
    template <bool VALUES> static __device__ __forceinline__ void interleave() {
        constexpr int kAhead = 4, PV = VALUES ? 4 * DB : 0, QK = 2 * KS;
        auto reads = [](int i) { return i < PV ? 2 : i < PV + QK ? 1 : 0; };
        int first = 0;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) first += reads(i);
        group_reads(first);
#pragma unroll
        for (int i = 0; i < PV + QK; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            group_reads(reads(i + kAhead));
        }
    }
    static __device__ __forceinline__ void group_reads(int n) {
        if (n >= 8) __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
        else if (n >= 4) __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
        else if (n == 2) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        else if (n == 1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }

    // 2^(c s - m) in bf16, the running maximum and sum (c >= 0: q carries the scale's sign);
    // `own`: the last position the lane's row sees
    template <bool MASKED> __device__ __forceinline__ void softmax(float c, int p0, int own, int lane) {
        if (MASKED) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (p0 + 32 * b + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3) > own) s[b][i] = -INFINITY;
        }
        float t = max3(s[0][0], s[1][0], s[0][1]), u = max3(s[1][1], s[0][2], s[1][2]);
#pragma unroll
        for (int i = 3; i < 15; i += 2) {
            t = max3(t, s[0][i], s[1][i]);
            u = max3(u, s[0][i + 1], s[1][i + 1]);
        }
        t = max3(t, s[0][15], s[1][15]);
        t = swap32_max(fmaxf(t, u));
        t = t == -INFINITY ? t : t * c;  // a scale of 0 leaves "nothing seen" as it is
        // m only has to keep the powers in range: it moves when the tile passes it by more than 2^8
        if (__any(t > m + 8.f)) {
            const float mn = fmaxf(m, t);
            const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] *= f;
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // with a scale of 0, -infinity would be 0 * infinity
                const float x = MASKED && s[b][i] == -INFINITY ? -INFINITY : fmaf(s[b][i], c, -ref);
                s[b][i] = __builtin_amdgcn_exp2f(x);
                sum[i & 1] += s[b][i];
            }
        l += sum[0] + sum[1];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = s[x >> 1][8 * (x & 1) + j];
            p[x] = to_frag(e, bf16x8{});
        }
    }

    // channels 32 d + l % 32, tokens 16 x + {0..3, 8..11} + 4 (l / 32)
    static __device__ __forceinline__ bf16x8 v_frag(const char *lv, int x, int d, int lane) {
        typedef __attribute__((address_space(3))) i16x4 lds4;
        const int i = lane & 15, t = 16 * x + 4 * (lane >> 5) + (i >> 2);
        const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((i >> 1) & 1);
        const char *at = lv + t * (2 * V) + 16 * (c ^ swz_v(t)) + 8 * (i & 1);
        const char *at2 = lv + (t + 8) * (2 * V) + 16 * (c ^ swz_v(t + 8)) + 8 * (i & 1);
        const bf16x4 y = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)at));
        const bf16x4 z = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)at2));
        return (bf16x8){y[0], y[1], y[2], y[3], z[0], z[1], z[2], z[3]};
    }

    __device__ __forceinline__ void values(const char *lv, int lane) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] = mma32(v_frag(lv, x, d, lane), p[x], o[d]);
    }

    // The same where some rows do not see some tokens. A weight of zero would not keep an
    // infinity or NaN out of a product: such values are taken out of the fragments of 16 tokens
    // that some row does not see, and added to the rows that see them.
    __device__ __forceinline__ void values_masked(const char *lv, int p0, int own, int tok0, int tok1, int lane) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (p0 + 16 * x > tok1) continue;  // no row of the wave sees any of the 16
            bf16x8 vf[DB];
            uint32_t odd = 0;
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                vf[d] = v_frag(lv, x, d, lane);
                const u32x4 u = __builtin_bit_cast(u32x4, vf[d]);
#pragma unroll
                for (int i = 0; i < 4; ++i) odd |= (u[i] & 0x7F807F80u) + 0x00800080u;  // an exponent of ones carries
            }
            const bool strange = p0 + 16 * x + 15 > tok0 && __any(odd & 0x80008000u);
            if (strange) {
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    u32x4 u = __builtin_bit_cast(u32x4, vf[d]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t t = ((u[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
                        u[i] &= ~((t >> 15) * 0xFFFFu);
                    }
                    vf[d] = __builtin_bit_cast(bf16x8, u);
                }
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) o[d] = mma32(vf[d], p[x], o[d]);
            if (strange) {
#pragma unroll 1
                for (int j = 0; j < 16; ++j) {  // token 16 x + j: its weights are in the lanes of half (j / 4) % 2
                    float w = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i == (j >> 3) * 4 + (j & 3)) w = s[x >> 1][8 * (x & 1) + i];
                    w = __shfl(w, 32 * ((j >> 2) & 1) + (lane & 31));
                    const int t = 16 * x + j;
                    const bool see = p0 + t <= own;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int ch = 32 * d + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3);
                            const float y = bf16_to_f32(*reinterpret_cast<const bf16_t *>(
                                lv + t * (2 * V) + 16 * ((ch >> 3) ^ swz_v(t)) + 2 * (ch & 7)));
                            if (see && !(fabsf(y) < INFINITY)) o[d][i] = fmaf(w, y, o[d][i]);
                        }
                }
            }
        }
    }
};

template <int K, int V, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attn_prompt_bf16_kernel(AttnArgs a, int slots) {
    using P = Prompt<K, V, NW>;
    __shared__ __align__(1024) char lds[2 * (P::KB + P::VB)];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);

    const int kvh = blockIdx.x % a.Hk;
    const int64_t slot = slots - 1 - static_cast<int>(blockIdx.x / a.Hk);  // the longest first
    const int n = seq_of_slot(a.cu, a.N, a.T, a.G, P::R, slot);
    int start, count;
    seq_rows(a.cu, n, a.T, start, count);
    const int64_t first = (slot - static_cast<int64_t>(start) * a.G / P::R - n) * P::R;
    const int64_t all = static_cast<int64_t>(count) * a.G;
    if (first < 0 || first >= all) return;
    const int last = static_cast<int>((min(first + P::R, all) - 1) / a.G);  // last token of the tile

    // this wave's rows; rows past the sequence's repeat its last one and are not stored
    const int64_t wr0 = first + 32 * w, wr1 = min(wr0 + 32, all);
    const bool some = wr0 < all;
    const int tok0 = static_cast<int>(min(wr0, all - 1) / a.G), tok1 = static_cast<int>((max(wr1, static_cast<int64_t>(1)) - 1) / a.G);
    const int64_t row = min(wr0 + (lane & 31), all - 1);
    const int own = static_cast<int>(row / a.G), h = kvh * a.G + static_cast<int>(row - static_cast<int64_t>(own) * a.G);

    P st;
    const float c = fabsf(a.c);
    st.m = -INFINITY;
    st.l = 0.f;
#pragma unroll
    for (int d = 0; d < P::DB; ++d) st.o[d] = f32x16{};

    const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char *)lds));
    // LDS: keys of even and odd tiles, values of even and odd tiles
    auto lk = [&](int j) { return (j & 1) * P::KB; };
    auto lv = [&](int j) { return 2 * P::KB + (j & 1) * P::VB; };
    typename P::template Copier<K, true> kc;
    typename P::template Copier<V, false> vc;
    kc.begin(static_cast<const bf16_t *>(a.k) + kvh * K, a.ks, start, a.T, w, lane);
    vc.begin(static_cast<const bf16_t *>(a.v) + kvh * V, a.vs, start, a.T, w, lane);
    // The two waves of a SIMD take turns: one is in its products (the values of the tile before,
    // the scores of this one) while the other is in its softmax, and every barrier swaps them.
    // Copies for a tile are issued two turns before its first use, which is when the last reader
    // of that buffer has gone. The first J tiles are seen whole by every row of the workgroup.
    const int J = (static_cast<int>(first / a.G) + 1) / kTile, tiles = last / kTile + 1;
    const bool ahead = w < NW / 2;
    auto copy_k = [&](int j) { if (j < tiles) kc.tile(base + lk(j), w, lane); };
    auto copy_v = [&](int j) { if (j < tiles) vc.tile(base + lv(j), w, lane); };
    auto swap = [&](bool wait) {
        if (wait) wait_copies();
        phase_barrier();
    };
    auto sees = [&](int j) { return some && j * kTile <= tok1; };  // the wave has work in tile j
    copy_k(0);
    {
        const bf16_t *src = static_cast<const bf16_t *>(a.q) + static_cast<int64_t>(start + own) * a.qs + h * K + 8 * (lane >> 5);
#pragma unroll
        for (int ks = 0; ks < P::KS; ++ks) st.q[ks] = load_frag(src + 16 * ks);
        const uint32_t sign = a.c < 0.f ? 0x80008000u : 0u;  // a negative scale is q's sign
#pragma unroll
        for (int ks = 0; ks < P::KS; ++ks)
            st.q[ks] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, st.q[ks]) ^ (u32x4){sign, sign, sign, sign});
    }
    swap(true);
    if (!ahead) {
        copy_k(1);
        copy_v(0);
        swap(false);
    }
    // The wave in its products issues first where they are the longer turn (two heads of 64
    // channels have half the products for the same softmax): 7.27 against 7.41 ms for 32768
    // tokens at 128 channels, and 191 against 188 us for 4 x 4096 at 64.
    constexpr bool kProductsFirst = K + V > 128;
    int j = 0;
    for (; j < J; ++j) {
        if (ahead) {
            copy_k(j + 1);
            copy_v(j);
        }
        if (kProductsFirst) __builtin_amdgcn_s_setprio(1);
        if (j > 0) {
            st.values(lds + lv(j - 1), lane);
            st.scores(lds + lk(j), lane);
            P::template interleave<true>();
        } else {
            st.scores(lds + lk(0), lane);
            P::template interleave<false>();
        }
        if (kProductsFirst) __builtin_amdgcn_s_setprio(0);
        swap(!ahead);
        if (!ahead) {
            copy_k(j + 2);
            copy_v(j + 1);
        }
        st.template softmax<false>(c, 0, own, lane);
        swap(ahead);
    }
    for (; j < tiles; ++j) {
        if (ahead) {
            copy_k(j + 1);
            copy_v(j);
        }
        if (j > 0 && sees(j - 1)) st.values_masked(lds + lv(j - 1), (j - 1) * kTile, own, tok0, tok1, lane);
        if (sees(j)) st.scores(lds + lk(j), lane);
        swap(!ahead);
        if (!ahead) {
            copy_k(j + 2);
            copy_v(j + 1);
        }
        if (sees(j)) st.template softmax<true>(c, j * kTile, own, lane);
        swap(ahead);
    }
    if (sees(j - 1)) st.values_masked(lds + lv(j - 1), (j - 1) * kTile, own, tok0, tok1, lane);
    if (ahead) swap(false);
    if (wr0 + (lane & 31) >= all) return;
    const float l = swap32_sum(st.l);
#pragma unroll
    for (int d = 0; d < P::DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            store_out(a, start, kvh, static_cast<int>(row), 32 * d + 8 * i + 4 * (lane >> 5),
                      (f32x4){st.o[d][4 * i], st.o[d][4 * i + 1], st.o[d][4 * i + 2], st.o[d][4 * i + 3]}, l);
}

template <int K, int V, int NW> hipError_t launch_bf16(const AttnArgs &a, hipStream_t st) {
    const int64_t slots = static_cast<int64_t>(a.T) * a.G / (32 * NW) + a.N;
    hipLaunchKernelGGL((attn_prompt_bf16_kernel<K, V, NW>), dim3(static_cast<unsigned>(slots * a.Hk)), dim3(64 * NW), 0, st, a,
                       static_cast<int>(slots));
    return hipGetLastError();
}

template <int K, int V, int RT>
hipError_t launch_f32(const AttnArgs &a, hipStream_t st) {
    const int64_t slots = static_cast<int64_t>(a.T) * a.G / (16 * RT) + a.N;
    hipLaunchKernelGGL((attn_prompt_kernel<K, V, RT, float>), dim3(static_cast<unsigned>(slots * a.Hk)), dim3(64 * kWaves), 0, st,
                       a, static_cast<int>(slots));
    return hipGetLastError();
}

template <int K, int V> hipError_t launch_dims(const AttnArgs &a, hipStream_t st) {
    if (a.in_dtype == KDA_F32) return launch_f32<K, V, 2>(a, st);
#ifdef KDA_NW
    return launch_bf16<K, V, KDA_NW>(a, st);
#else
    return launch_bf16<K, V, 8>(a, st);
#endif
}

}  // namespace

hipError_t launch_attn_prompt(const AttnArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace kda
