// Attention of 32 rows per wave over tiles of 64 keys and values in LDS, in bf16.
//
// 32 x 32 matrix instructions, 16-deep: S^T = K Q^T leaves the scores of row
// l % 32 for tokens 32 b + 8 (i / 4) + 4 (l / 32) + i % 4 in register i of lane l,
// and those registers, rounded to bf16, are the B operand of O^T = V^T P^T when
// V^T's fragments take the tokens in the same order, which the transposing LDS
// reads do. P never moves between lanes.
#pragma once

#include "kda_attn_device.h"

namespace kda {

__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Copies from memory straight to LDS: 16 (4) bytes per lane from base (wave-uniform) + off, to
// dst (wave-uniform) + 16 (4) * lane. Unknown to the compiler's wait insertion: awaited by
// wait_copies() before a barrier. A scalar base may come from a vector instruction (a spilled
// register's return), and may be read five wait states later: the s_nop 3. (The clobber keeps
// the compiler from holding anything in M0 across them; its warning only says that it will not
// save and restore M0.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy_to_lds(uint32_t dst, const void *base, uint32_t off) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void copy_word_to_lds(uint32_t dst, const void *src) {
    __asm__ volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(dst), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop
// all but the newest N of the wave's memory operations
template <int N = 0> __device__ __forceinline__ void wait_copies() { __asm__ volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint32_t lds_address(const char *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char *)p));
}

// The largest of three, a NaN passed over: one instruction, where fmaxf of two would first make
// quiet NaNs of its operands. Not as inline assembly: it is the first to read the products'
// results, and the compiler leaves the wait states that these need only before instructions that
// it knows.
__device__ __forceinline__ float max3(float x, float y, float z) {
    return __builtin_elementwise_maximumnum(__builtin_elementwise_maximumnum(x, y), z);
}

// A workgroup barrier that nothing is moved across, without waiting for copies.
__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

constexpr int kTile = 64;  // tokens per tile

// A row's running maximum is -infinity until the row has seen a token, and at least this from then
// on, also if the scores are -infinity or NaN: a row that sees no token is 0, one whose scores are
// all -infinity is 0 / 0.
constexpr float kLowest = -3.402823466e38f;

template <int K, int V> struct Rows {
    static constexpr int CK = K / 8, CV = V / 8;  // 16-byte chunks per row
    static constexpr int KB = kTile * K * 2, VB = kTile * V * 2;
    static constexpr int KS = K / 16, DB = V / 32;

    // chunk c of token t lies at chunk c ^ swz(t) of its row: the tokens that one read takes
    // the same chunk of are spread over the banks
    static __device__ __forceinline__ int swz_k(int t) { return CK == 16 ? t & 15 : (t >> 1) & 7; }
    static __device__ __forceinline__ int swz_v(int t) { return CV == 16 ? (t & 3) * 4 : ((t >> 1) & 1) * 4; }

    bf16x8 q[KS];
    f32x16 o[DB], s[2];
    bf16x8 p[4];
    float m, l;

    // a negative scale is q's sign
    __device__ __forceinline__ void load_q(const bf16_t *row, bool negative, int lane) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = load_frag(row + 16 * ks + 8 * (lane >> 5));
        if (negative) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                q[ks] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, q[ks]) ^ (u32x4){0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u});
        }
    }
    __device__ __forceinline__ void reset() {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int d = 0; d < DB; ++d) o[d] = f32x16{};
    }

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
    // values() [if VALUES] and scores() [if SCORES] in a row: reads run kAhead products ahead of their use,
    // which covers their latency. Left to itself the compiler reads right before each product.
    template <bool VALUES, bool SCORES = true> static __device__ __forceinline__ void interleave() {
        constexpr int kAhead = 4, PV = VALUES ? 4 * DB : 0, QK = SCORES ? 2 * KS : 0;
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

    // of a row's bits for the 64 tokens, those of the lane's registers: bit 16 b + i of the result
    // is token 32 b + 8 (i / 4) + 4 (l / 32) + i % 4
    static __device__ __forceinline__ uint32_t of_lane(uint64_t w, int lane) {
        w >>= 4 * (lane >> 5);
        uint32_t v = 0;
#pragma unroll
        for (int n = 0; n < 8; ++n) v |= (static_cast<uint32_t>(w >> (8 * n)) & 15u) << (4 * n);
        return v;
    }

    // 2^(c s - m) in bf16, the running maximum and sum (c >= 0: q carries the scale's sign). A weight
    // is one bf16 number, off by at most 2^-8 of it: a second one, as in the streaming form, would
    // double the products with the values. Measured against 64 bits, bf16 outputs are off by 0.0018 to
    // 0.0023 of their size so, and by 0.0014 to 0.0017 with fp32 weights.
    // `sees`: a bit for each of the lane's 32 tokens that its row sees, used if MASKED
    template <bool MASKED> __device__ __forceinline__ void softmax(float c, uint32_t sees) {
        if (MASKED) {
            // by a word of ones where the lane's token i is seen: 104.5 against 106.3 us for 24 drafted tokens
            // of 16 sequences, e4m3, with conditions (words kept for the weights below as well: they spill)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint32_t seen = static_cast<uint32_t>(static_cast<int32_t>(sees << (31 - i)) >> 31);
                s[i >> 4][i & 15] = __uint_as_float((__float_as_uint(s[i >> 4][i & 15]) & seen) | (0xFF800000u & ~seen));
            }
        }
        float t = max3(s[0][0], s[1][0], s[0][1]), u = max3(s[1][1], s[0][2], s[1][2]);
#pragma unroll
        for (int i = 3; i < 15; i += 2) {
            t = max3(t, s[0][i], s[1][i]);
            u = max3(u, s[0][i + 1], s[1][i + 1]);
        }
        t = max3(t, s[0][15], s[1][15]);
        t = fmaxf(fmaxf(t, u) * c, kLowest);
        if (MASKED) t = sees ? t : -INFINITY;
        t = swap32_max(t);
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
                s[b][i] = __builtin_amdgcn_exp2f(fmaf(s[b][i], c, -ref));
                // not left to the exponential: with a scale of 0, -infinity is 0 * infinity
                if (MASKED && !((sees >> (16 * b + i)) & 1u)) s[b][i] = 0.f;
                sum[i & 1] += s[b][i];
            }
        l += sum[0] + sum[1];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                e[j] = s[x >> 1][8 * (x & 1) + j];
            }
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
    // channel ch of token t
    static __device__ __forceinline__ float v_at(const char *lv, int t, int ch) {
        return bf16_to_f32(*reinterpret_cast<const bf16_t *>(lv + t * (2 * V) + 16 * ((ch >> 3) ^ swz_v(t)) + 2 * (ch & 7)));
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
    __device__ __forceinline__ void values_masked(const char *lv, uint32_t sees, int lane) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t mine = (sees >> (8 * x)) & 255u;  // bits 8 x .. 8 x + 7 are the lane's of these 16 tokens
            if (!__any(mine != 0)) continue;                 // no row of the wave sees any of them
            bf16x8 vf[DB];
#pragma unroll
            for (int d = 0; d < DB; ++d) vf[d] = v_frag(lv, x, d, lane);
            bool strange = false;
            if (__any(mine != 255u)) {
                uint32_t odd = 0;
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const u32x4 u = __builtin_bit_cast(u32x4, vf[d]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) odd |= (u[i] & 0x7F807F80u) + 0x00800080u;  // an exponent of ones carries
                }
                strange = __any((odd & 0x80008000u) != 0);
            }
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
                    const int reg = (j >> 3) * 4 + (j & 3), src = 32 * ((j >> 2) & 1) + (lane & 31);
                    float w = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i == reg) w = s[x >> 1][8 * (x & 1) + i];
                    w = __shfl(w, src);
                    const bool see = (__shfl(mine, src) >> reg) & 1u;
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float y = v_at(lv, 16 * x + j, 32 * d + 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3));
                            if (see && !(fabsf(y) < INFINITY)) o[d][i] = fmaf(w, y, o[d][i]);
                        }
                }
            }
        }
    }

    // put(channel, four outputs) for the lane's row: channels 32 d + 8 i + 4 (l / 32) + 0..3
    template <typename Put> __device__ __forceinline__ void each(int lane, Put put) const {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                put(32 * d + 8 * i + 4 * (lane >> 5), (f32x4){o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]});
    }
};

// o of one row: channels ch .. ch + 3 of row r of a tile, from its maximum, unnormalised outputs and sum
__device__ __forceinline__ void store_out(const AttnArgs &a, int start, int kvh, int r, int ch, float m, f32x4 x, float l) {
    const int tok = r / a.G, h = kvh * a.G + (r - tok * a.G);
    const int64_t at = (static_cast<int64_t>(start + tok) * a.H + h) * a.V + ch;
    const bool none = m == -INFINITY;  // the row saw no token: x and l are 0
    x *= none ? 0.f : 1.f / l;
    if (a.out_dtype == KDA_BF16) {
        const bf16x2 lo = pack_bf16(x[0], x[1]), hi = pack_bf16(x[2], x[3]);
        *reinterpret_cast<bf16x4 *>(static_cast<bf16_t *>(a.o) + at) = (bf16x4){lo[0], lo[1], hi[0], hi[1]};
    } else {
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.o) + at) = x;
    }
}

}  // namespace kda
