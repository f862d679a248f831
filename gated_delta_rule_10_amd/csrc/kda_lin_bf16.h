// The chunk step of kda_lin_chunk.hip for bf16 inputs, on the matrix cores.
//
// 64 tokens to a chunk. A wave holds 32 value channels: its part of the state as
// K / 32 results of 32 x 32 products, S[m] register r of lane l being value channel
// l % 32 and key channel 32 m + 16 (r / 8) + 8 (l / 32) + r % 8: the rows of these
// products are taken in an order that leaves 8 neighbouring key channels in a lane.
// In that form the state feeds products without moving between lanes, and what it
// is multiplied with is read 16 bytes at a time:
//
//     O^T = S^T Q^T e^(G_i) + V^T P^T        P = (Q K^T) * e^(G_i - G_j), j <= i
//     S   = e^(G_C) S + K^T (V e^(G_C - G_j))
//
// P is formed once per workgroup, a quarter of 32 x 32 to a wave, and shared in LDS.
// q, k and v are exact bf16 operands. V e^(..) is three bf16 parts (24 bits, all of
// fp32): its rounding would stay in the state. S and P only go into the outputs: one
// part for bf16 outputs, which round them as much again, two for fp32 ones.
#pragma once

#include "kda_attn_rows.h"
#include "kda_lin_device.h"

namespace kda {

// x as a sum of bf16 parts, the first the nearest to it; x keeps what is left. The subtraction is a
// dot product of two with (-1, 0) or (0, -1), one instruction instead of an unpacking and a
// difference, and exact: what is left has fewer bits than x.
// (The factors are in scalar registers: as an inline constant, -1.0 is not the pair (-1, 0).)
__device__ __forceinline__ float less_first(bf16x2 p, float x) {
    uint32_t f = 0x0000BF80u;
    __asm__("" : "+s"(f));
    return __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2, f), x, false);
}
__device__ __forceinline__ float less_second(bf16x2 p, float x) {
    uint32_t f = 0xBF800000u;
    __asm__("" : "+s"(f));
    return __builtin_amdgcn_fdot2_f32_bf16(p, __builtin_bit_cast(bf16x2, f), x, false);
}
__device__ __forceinline__ void split_bf16(float (&x)[8], bf16x8 &part) {
    part = to_frag(x, bf16x8{});
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 p = {part[2 * i], part[2 * i + 1]};
        x[2 * i] = less_first(p, x[2 * i]);
        x[2 * i + 1] = less_second(p, x[2 * i + 1]);
    }
}
__device__ __forceinline__ void widen(const bf16x8 &v, float (&x)[8]) {
    const u32x4 u = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

// The lane's number as a value that the compiler does not see through: addresses in LDS, an exclusive
// or away from it, are then made where they are used instead of being kept over the chunks, which
// takes more registers than there are.
__device__ __forceinline__ int opaque(int lane) {
    __asm__ volatile("" : "+v"(lane));
    return lane;
}

// PARTS: of S and P; 0 where there are no outputs
template <int K, int V, int PARTS> struct LinBf16 {
    using T = bf16_t;
    static constexpr bool OUT = PARTS > 0;
    static constexpr int C = 64, NW = V / 32, NT = 64 * NW, M = K / 32;
    // with two waves a thread holds twice as much of the next chunk, and 256 registers do not do
    static constexpr int kWavesPerSimd = OUT && NW == 2 && K == 128 ? 1 : 2;
    static constexpr int CK = K / 8, CV = V / 8;          // 16-byte pieces of a row
    static constexpr int LK = C * CK / NT, LV = C * CV / NT;  // of a thread
    static constexpr int kQ = 0, kK = OUT ? C * K * 2 : 0, kV = kK + C * K * 2, kP = kV + C * V * 2;
    static constexpr int kLds = kP + PARTS * C * C * 2;

    // Piece c of token t lies at piece c ^ swz(t) of its row: 16 rows read at one piece, and 4 rows
    // read at 4 pieces (the transposing reads), fall on different banks.
    static __device__ __forceinline__ int swz16(int t) { return ((t & 3) << 2) | ((t >> 2) & 3); }
    static __device__ __forceinline__ int swz8(int t) { return (((t >> 1) & 1) << 2) | ((t >> 2) & 3); }
    template <int CH> static __device__ __forceinline__ int at(int t, int c) {
        return t * (CH * 16) + 16 * (c ^ (CH == 16 ? swz16(t) : swz8(t)));
    }

    u32x4 q[OUT ? LK : 1], k[LK], v[LV];  // the next chunk, on its way
    f32x16 S[M];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[m][r] = 0.f;
    }

    static __device__ __forceinline__ void prepare(char *, int) {}  // nothing in LDS outlasts a chunk

    // Rows from `count` on are the last one again: their scores are masked and their values weigh 0.
    template <int CH, int L> static __device__ __forceinline__ void load_rows(u32x4 (&x)[L], const T *p, int64_t stride, int count, int tid) {
        const char *base = reinterpret_cast<const char *>(p);
        constexpr int STEP = NT / CH;  // rows from one load to the next
        if (count == C) {
            const uint32_t off = static_cast<uint32_t>(tid / CH) * static_cast<uint32_t>(2 * stride) + 16 * (tid % CH);
#pragma unroll
            for (int i = 0; i < L; ++i) x[i] = *reinterpret_cast<const u32x4 *>(base + i * STEP * 2 * stride + off);
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const uint32_t t = min(i * STEP + tid / CH, count - 1);
                x[i] = *reinterpret_cast<const u32x4 *>(base + t * static_cast<uint32_t>(2 * stride) + 16 * (tid % CH));
            }
        }
    }
    template <int CH, int L> static __device__ __forceinline__ void store_rows(const u32x4 (&x)[L], char *p, int tid) {
#pragma unroll
        for (int i = 0; i < L; ++i) *reinterpret_cast<u32x4 *>(p + at<CH>((i * NT + tid) / CH, tid % CH)) = x[i];
    }
    // rows of the chunk that starts at these
    __device__ __forceinline__ void load(const T *qp, const T *kp, const T *vp, const LinArgs &a, int count, int tid) {
        if (OUT) load_rows<CK>(q, qp, a.qs, count, tid);
        load_rows<CK>(k, kp, a.ks, count, tid);
        load_rows<CV>(v, vp, a.vs, count, tid);
    }
    // whether some of this thread's values is an infinity or NaN
    __device__ __forceinline__ bool to_lds(char *lds, int tid) {
        if (OUT) store_rows<CK>(q, lds + kQ, tid);
        store_rows<CK>(k, lds + kK, tid);
        store_rows<CV>(v, lds + kV, tid);
        if (!OUT) return false;
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < LV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= not_finite<bf16_t>(v[i][j]);
        return odd != 0;
    }

    // Columns 32 d .. of a tile as rows of a product, tokens 16 x + 8 (l / 32) + 0..7. Each read gives 16
    // lanes 4 tokens of 16 columns, 4 neighbouring ones from the address of every fourth lane. Of the
    // 8 groups of 4 rows of a product, the 2nd and 3rd (6th and 7th) change places where `swap`.
    template <int CH, bool SWAP> static __device__ __forceinline__ bf16x8 transposed(const char *p, int x, int d, int lane) {
        typedef __attribute__((address_space(3))) i16x4 lds4;
        const int i = lane & 15, t = 16 * x + 8 * (lane >> 5) + (i >> 2);
        const int hi = SWAP ? i & 1 : (i >> 1) & 1, lo = SWAP ? (i >> 1) & 1 : i & 1;
        const int c = 4 * d + 2 * ((lane >> 4) & 1) + hi;
        const bf16x4 y = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + at<CH>(t, c) + 8 * lo)));
        const bf16x4 z = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + at<CH>(t + 4, c) + 8 * lo)));
        return (bf16x8){y[0], y[1], y[2], y[3], z[0], z[1], z[2], z[3]};
    }
    // row t, elements 16 x + 8 half + 0..7
    template <int CH> static __device__ __forceinline__ bf16x8 eight(const char *p, int x, int t, int half) {
        return *reinterpret_cast<const bf16x8 *>(p + at<CH>(t, 2 * x + half));
    }

    // The quarter of P of rows i0.. and columns j0.., in bf16 parts in LDS
    static __device__ __forceinline__ void scores(char *lds, const Decays &d, float scale, int i0, int j0, int lane) {
        lane = opaque(lane);
        const int l = lane & 31, half = lane >> 5, i = i0 + l;
        f32x16 p = {};
#pragma unroll
        for (int x = 0; x < K / 16; ++x) p = mma32(eight<CK>(lds + kK, x, j0 + l, half), eight<CK>(lds + kQ, x, i, half), p);
        const float hi = d.hi[i], lo = d.lo[i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int j = j0 + 8 * c + 4 * half;  // p[4 c + r]: row i, column j + r
            const f32x4 dh = *reinterpret_cast<const f32x4 *>(d.hi + j), dl = *reinterpret_cast<const f32x4 *>(d.lo + j);
            float e[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                e[r] = j + r <= i ? p[4 * c + r] * (scale * __builtin_amdgcn_exp2f((hi - dh[r]) + (lo - dl[r]))) : 0.f;
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
                const bf16x2 a = pack_bf16(e[0], e[1]), b = pack_bf16(e[2], e[3]);
                *reinterpret_cast<bf16x4 *>(lds + kP + part * C * C * 2 + at<8>(i, j >> 3) + 8 * half) = (bf16x4){a[0], a[1], b[0], b[1]};
                if (part + 1 < PARTS) {
                    e[0] = less_first(a, e[0]);
                    e[1] = less_second(a, e[1]);
                    e[2] = less_first(b, e[2]);
                    e[3] = less_second(b, e[3]);
                }
            }
        }
    }

    // O^T (channels 32 w + ..) from the state before the chunk: column l % 32 is token 32 b + l % 32
    __device__ __forceinline__ void from_state(f32x16 (&o)[2], const char *lds, const Decays &d, float scale, int lane) const {
        lane = opaque(lane);
        const f32x16 zero = {};
#pragma unroll
        for (int x = 0; x < K / 16; ++x) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = S[x / 2][8 * (x & 1) + i];
            bf16x8 p[PARTS], f[2];
#pragma unroll
            for (int i = 0; i < PARTS - 1; ++i) split_bf16(s, p[i]);
            p[PARTS - 1] = to_frag(s, bf16x8{});

#pragma unroll
            for (int b = 0; b < 2; ++b) f[b] = eight<CK>(lds + kQ, x, 32 * b + (lane & 31), lane >> 5);
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                for (int b = 0; b < 2; ++b) o[b] = mma32(p[i], f[b], x + i == 0 ? zero : o[b]);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float e = scale * d.grown[32 * b + (lane & 31)];
#pragma unroll
            for (int r = 0; r < 16; ++r) o[b][r] *= e;
        }
    }

    // adds V^T P^T
    static __device__ __forceinline__ void from_chunk(f32x16 (&o)[2], const bf16x8 (&vf)[4], const char *lds, int lane) {
        lane = opaque(lane);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int b = x / 2; b < 2; ++b)
                    o[b] = mma32(vf[x], eight<8>(lds + kP + part * C * C * 2, x, 32 * b + (lane & 31), lane >> 5), o[b]);
    }
    // The same where some value is an infinity or NaN: a masked score's 0 times it would be NaN, so such
    // values are taken out of the products and added to the rows that they reach one by one.
    static __device__ __forceinline__ void from_odd_chunk(f32x16 (&o)[2], const bf16x8 (&vf)[4], const char *lds, int w, int lane) {
        bf16x8 fine[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            u32x4 u = __builtin_bit_cast(u32x4, vf[x]);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] &= ~((not_finite<bf16_t>(u[i]) >> 15) * 0xFFFFu);
            fine[x] = __builtin_bit_cast(bf16x8, u);
        }
        from_chunk(o, fine, lds, lane);
        lane = opaque(lane);
        const int half = lane >> 5;
#pragma unroll 1
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = 32 * b + (lane & 31), p = kP + at<8>(i, j >> 3) + 2 * (j & 7);
                float s = 0.f;
#pragma unroll
                for (int part = 0; part < PARTS; ++part) s += bf16_to_f32(*reinterpret_cast<const bf16_t *>(lds + p + part * C * C * 2));
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int c = 32 * w + 8 * (r >> 2) + 4 * half + (r & 3);
                    const float x = bf16_to_f32(*reinterpret_cast<const bf16_t *>(lds + kV + at<CV>(j, c >> 3) + 2 * (c & 7)));
                    if (j <= i && !(fabsf(x) < INFINITY)) o[b][r] += s * x;
                }
            }
    }

    // rows of o through the wave's own columns of v's tile, whose values are in registers by now
    static __device__ __forceinline__ void store(bf16_t *out, int64_t stride, const f32x16 (&o)[2], char *lds, int count, int w, int lane) {
        lane = opaque(lane);
        const int half = lane >> 5;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bf16x2 x = pack_bf16(o[b][4 * c], o[b][4 * c + 1]), y = pack_bf16(o[b][4 * c + 2], o[b][4 * c + 3]);
                *reinterpret_cast<bf16x4 *>(lds + kV + at<CV>(32 * b + (lane & 31), 4 * w + c) + 8 * half) = (bf16x4){x[0], x[1], y[0], y[1]};
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 16 * i + (lane >> 2), c = 4 * w + (lane & 3);
            const u32x4 x = *reinterpret_cast<const u32x4 *>(lds + kV + at<CV>(t, c));
            if (t < count) *reinterpret_cast<u32x4 *>(out + t * stride + 8 * c) = x;
        }
    }
    static __device__ __forceinline__ void store(float *out, int64_t stride, const f32x16 (&o)[2], char *, int count, int w, int lane) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int t = 32 * b + (lane & 31);
            if (t >= count) continue;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<f32x4 *>(out + t * stride + 32 * w + 8 * c + 4 * (lane >> 5)) =
                    (f32x4){o[b][4 * c], o[b][4 * c + 1], o[b][4 * c + 2], o[b][4 * c + 3]};
        }
    }

    // S = e^(G_C) S + K^T (V e^(G_C - G_j)), the first factor only where DECAY
    template <bool DECAY> __device__ __forceinline__ void update(const char *lds, const Decays &d, int w, int lane) {
        bf16x8 vf[4];
        values(vf, lds, w, lane);
        update<DECAY>(vf, lds, d, lane);
    }
    static __device__ __forceinline__ void values(bf16x8 (&vf)[4], const char *lds, int w, int lane) {
#pragma unroll
        for (int x = 0; x < 4; ++x) vf[x] = transposed<CV, false>(lds + kV, x, w, opaque(lane));
    }
    template <bool DECAY> __device__ __forceinline__ void update(const bf16x8 (&vf)[4], const char *lds, const Decays &d, int lane) {
        // first in line for the matrix cores: the products here are most of a chunk's (1 x 131072 1480 -> 1461 us)
        __builtin_amdgcn_s_setprio(1);
        lane = opaque(lane);
        const int half = lane >> 5;
        if (DECAY) {
            const float all = d.grown[C - 1];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) S[m][r] *= all;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            float f[8];
            widen(vf[x], f);
            const f32x4 a = *reinterpret_cast<const f32x4 *>(d.left + 16 * x + 8 * half), b = *reinterpret_cast<const f32x4 *>(d.left + 16 * x + 8 * half + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] *= a[i];
                f[4 + i] *= b[i];
            }
            bf16x8 p[3];
            split_bf16(f, p[0]);
            split_bf16(f, p[1]);
            p[2] = to_frag(f, bf16x8{});
            bf16x8 kf[M];
#pragma unroll
            for (int m = 0; m < M; ++m) kf[m] = transposed<CK, true>(lds + kK, x, m, lane);
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int m = 0; m < M; ++m) S[m] = mma32(kf[m], p[i], S[m]);
        }
        __builtin_amdgcn_s_setprio(0);
    }

    // one chunk, whose tiles are in LDS; odd: not 0 if some value is an infinity or NaN
    template <typename TOut, typename Next>
    __device__ __forceinline__ void chunk(TOut *out, int64_t stride, float scale, char *lds, const Decays &d, const int &odd, int count, int w, int lane, Next next) {
        f32x16 o[2];
        // the three quarters on and below the diagonal; the last wave has the next chunk's decays to sum
        if (w < 3 && w < NW) scores(lds, d, scale, w ? 32 : 0, w == 2 ? 32 : 0, lane);
        if (NW == 2 && w == 0) scores(lds, d, scale, 32, 32, lane);
        next();  // the loads of the next chunk leave
        from_state(o, lds, d, scale, lane);
        __syncthreads();
        bf16x8 vf[4];
        values(vf, lds, w, lane);
        if (__builtin_amdgcn_readfirstlane(odd) == 0)
            from_chunk(o, vf, lds, lane);
        else
            from_odd_chunk(o, vf, lds, w, lane);
        store(out, stride, o, lds, count, w, lane);
        update<true>(vf, lds, d, lane);
    }

    // the state as the registers hold it, in memory
    __device__ __forceinline__ void put(float *p, int w, int lane) const {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                *reinterpret_cast<f32x4 *>(p + (((w * M + m) * 4 + r) * 64 + lane) * 4) =
                    (f32x4){S[m][4 * r], S[m][4 * r + 1], S[m][4 * r + 2], S[m][4 * r + 3]};
    }
    __device__ __forceinline__ void get(const float *p, int w, int lane) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const f32x4 x = *reinterpret_cast<const f32x4 *>(p + (((w * M + m) * 4 + r) * 64 + lane) * 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) S[m][4 * r + i] = x[i];
            }
    }

    // a [K, V] state
    __device__ __forceinline__ void take(const float *p, int w, int lane) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[m][r] = p[element(m, r, w, lane)];
    }
    __device__ __forceinline__ void give(float *p, int w, int lane) const {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) p[element(m, r, w, lane)] = S[m][r];
    }
    // register r of S[m] and its element
    static __device__ __forceinline__ int element(int m, int r, int w, int lane) {
        return (32 * m + 16 * (r >> 3) + 8 * (lane >> 5) + (r & 7)) * V + 32 * w + (lane & 31);
    }
};

}  // namespace kda
