// The chunk step of kda_lin_chunk.hip for bf16 inputs, on the matrix cores.
//
// 64 tokens to a chunk. A wave holds 16 value channels: its part of the state as
// K / 16 results of 16 x 16 products, S[m] register r of lane l being value channel
// l % 16 and key channel 32 (m / 2) + 8 (l / 16) + 4 (m % 2) + r: the rows of these
// products are taken in an order that leaves 8 neighbouring key channels of each
// pair of results in a lane. In that form the state feeds products without moving
// between lanes, and what it is multiplied with is read 16 bytes at a time:
//
//     O^T = S^T Q^T e^(G_i) + V^T P^T        P = (Q K^T) * e^(G_i - G_j), j <= i
//     S   = e^(G_C) S + K^T (V e^(G_C - G_j))
//
// P is formed once per workgroup, in tiles of 16 x 16 spread over the waves, and
// shared in LDS. q, k and v are exact bf16 operands. V e^(..) is three bf16 parts
// (24 bits, all of fp32): its rounding would stay in the state (two parts: states
// off by 2.6e-6 of their size instead of 4e-7, and 150 us of 1450 less for 131072 tokens,
// H = 32). S and P only go into the outputs and are two parts (16 bits), also for bf16 outputs:
// one part would be rounded as much as those are, and they would be off by 0.0024 of their
// size instead of 0.0017 (131072 tokens 1420 us instead of 1550).
//
// 16 value channels to a wave and 8 waves to a workgroup, one to a compute unit: S is 32
// registers of a lane, and the chunk's tiles are read by 8 waves at once. (Four waves of
// 32 channels, two workgroups to a compute unit: 1446 us against 1421, and 16 prompts of
// 217 to 3448 tokens 252 against 199, both with one part of S and P.) A chunk's loads,
// products, LDS reads and conversions hardly overlap within a wave: a workgroup alone
// takes 3.5 us a chunk.
#pragma once

#include "kda_attn_device.h"
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
// or away from it, are then made where they are used instead of being kept over the chunks. The walk to
// the ends has room for 4 waves on a SIMD that way; the outputs' has two at most for their state and
// outputs, and is faster with the addresses kept (1421 against 1467 us, with one part of S and P).
__device__ __forceinline__ int opaque(int lane) {
    __asm__ volatile("" : "+v"(lane));
    return lane;
}

// TOut: of the outputs; void where there are none
template <int K, int V, typename TOut> struct LinBf16 {
    using T = bf16_t;
    static constexpr bool OUT = !__is_void(TOut), kHalf = __is_same(TOut, bf16_t);
    static constexpr int PARTS = OUT ? 2 : 0;  // of S and P
    static constexpr int C = 64, NW = V / 16, NT = 64 * NW, M = K / 16;
    static constexpr int kWavesPerSimd = OUT ? 2 : 4;
    static constexpr int CK = K / 8, CV = V / 8;              // 16-byte pieces of a row
    static constexpr int LK = C * CK / NT, LV = C * CV / NT;  // of a thread
    // in LDS: q, k and v of a chunk; P
    static constexpr int kQ = 0, kK = OUT ? C * K * 2 : 0, kV = kK + C * K * 2;
    static constexpr int kTiles = kV + C * V * 2, kScores = PARTS * C * C * 2;
    static constexpr int kOutBytes = kHalf ? 2 : 4, kOuts = C * V * kOutBytes;  // the outputs of a chunk

    // Piece c of token t lies at piece c ^ swz(t) of its row, so that what is read at once falls on different
    // banks. A read of 16 bytes a lane is served in groups of 16 lanes, 0 to 3, 12 to 15 and 20 to 27 the
    // first and the other 16 of 32 the second (so the bank conflicts counted for such patterns say): half of
    // 16 rows at one piece, the other half at the next one. A transposing read is served in groups of 32: of 8
    // rows apart by 1 or 8, either 2 pieces each or 4 half ones, for which k's rows with bit 3 of t set have the
    // halves of their pieces changed over. (With order 0, 1, 2, 3 instead of 0, 2, 3, 1 in the low bits, and
    // halves in place, 40 % of LDS cycles are conflicts: 8 x 2000 tokens 2 us more of 140.)
    static __device__ __forceinline__ int low(int t) { return (((t >> 1) ^ (t >> 2)) & 2) | ((t >> 3) & 1); }
    static __device__ __forceinline__ int swz16(int t) { return ((t & 3) << 2) | low(t); }
    static __device__ __forceinline__ int swz8(int t) { return ((t & 2) << 1) | low(t); }
    static __device__ __forceinline__ u32x4 halves(const u32x4 &x, bool changed) {
        return changed ? u32x4{x[2], x[3], x[0], x[1]} : x;
    }
    template <int CH> static __device__ __forceinline__ int at(int t, int c) {
        return t * (CH * 16) + 16 * (c ^ (CH == 16 ? swz16(t) : swz8(t)));
    }

    u32x4 q[OUT ? LK : 1], k[LK], v[LV];  // the next chunk, on its way
    f32x4 S[M], o[4];                     // the state; the chunk's outputs, transposed
    bf16x8 vf[2];                         // the wave's values

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int m = 0; m < M; ++m) S[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // what no chunk writes: the scores of rows 0.. (32..) for columns 16.. (48..), right of the diagonal, are 0
    static __device__ __forceinline__ void prepare(char *scores, int tid) {
        if (OUT && tid < 64 * PARTS) {
            const int t = 32 * ((tid >> 5) & 1) + (tid & 15), c = 4 * ((tid >> 5) & 1) + 2 + ((tid >> 4) & 1);
            *reinterpret_cast<u32x4 *>(scores + (tid >> 6) * C * C * 2 + at<8>(t, c)) = u32x4{0, 0, 0, 0};
        }
    }

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
#pragma unroll
        for (int i = 0; i < LK; ++i) {
            const int t = (i * NT + tid) / CK;
            *reinterpret_cast<u32x4 *>(lds + kK + at<CK>(t, tid % CK)) = halves(k[i], t & 8);
        }
        store_rows<CV>(v, lds + kV, tid);
        if (!OUT) return false;
        uint32_t odd = 0;
#pragma unroll
        for (int i = 0; i < LV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) odd |= not_finite<bf16_t>(v[i][j]);
        return odd != 0;
    }

    // Two reads, each of which gives 16 lanes 4 tokens of 16 columns, 4 neighbouring ones from the address of
    // every fourth lane: tokens 32 y + 8 (l / 16) + 0..7 of a column to a lane.
    template <int CH> static __device__ __forceinline__ bf16x8 transposed(const char *p, int t, int c, int b) {
        typedef __attribute__((address_space(3))) i16x4 lds4;
        const bf16x4 y = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + at<CH>(t, c) + b)));
        const bf16x4 z = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + at<CH>(t + 4, c) + b)));
        return (bf16x8){y[0], y[1], y[2], y[3], z[0], z[1], z[2], z[3]};
    }
    static __device__ __forceinline__ bf16x8 keys(const char *lds, int y, int m, int lane) {  // rows of S[m]
        const int i = lane & 15;
        return transposed<CK>(lds + kK, 32 * y + 8 * (lane >> 4) + (i >> 2), 4 * (m >> 1) + (i & 3), 8 * ((m ^ (lane >> 4)) & 1));
    }
    static __device__ __forceinline__ bf16x8 values(const char *lds, int y, int w, int lane) {  // channels 16 w + ..
        const int i = lane & 15;
        return transposed<CV>(lds + kV, 32 * y + 8 * (lane >> 4) + (i >> 2), 2 * w + ((i >> 1) & 1), 8 * (i & 1));
    }
    template <int CH> static __device__ __forceinline__ bf16x8 row(const char *p, int t, int c) {
        return *reinterpret_cast<const bf16x8 *>(p + at<CH>(t, c));
    }

    // tile n of the 10 of 16 x 16 of P on and below the diagonal, row by row, in bf16 parts in LDS
    static __device__ __forceinline__ void score_tile(char *scores, const char *lds, const Decays &d, float scale, int n, int lane) {
        const int it = n < 1 ? 0 : n < 3 ? 1 : n < 6 ? 2 : 3, i0 = 16 * it, j0 = 16 * (n - it * (it + 1) / 2);
        const int l = lane & 15, g = lane >> 4, i = i0 + l, j = j0 + 4 * g;  // p[r]: row i, column j + r
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < K / 32; ++x) {
            const u32x4 kx = halves(__builtin_bit_cast(u32x4, row<CK>(lds + kK, j0 + l, 4 * x + g)), l & 8);
            p = mma16(__builtin_bit_cast(bf16x8, kx), row<CK>(lds + kQ, i, 4 * x + g), p);
        }
        const float hi = d.hi[i], lo = d.lo[i];
        const f32x4 dh = *reinterpret_cast<const f32x4 *>(d.hi + j), dl = *reinterpret_cast<const f32x4 *>(d.lo + j);
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = j + r <= i ? p[r] * (scale * __builtin_amdgcn_exp2f((hi - dh[r]) + (lo - dl[r]))) : 0.f;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
            const bf16x2 a = pack_bf16(p[0], p[1]), b = pack_bf16(p[2], p[3]);
            *reinterpret_cast<bf16x4 *>(scores + part * C * C * 2 + at<8>(i, j >> 3) + 8 * (g & 1)) = (bf16x4){a[0], a[1], b[0], b[1]};
            if (part + 1 < PARTS) {
                p[0] = less_first(a, p[0]);
                p[1] = less_second(a, p[1]);
                p[2] = less_first(b, p[2]);
                p[3] = less_second(b, p[3]);
            }
        }
    }

    // The last wave has a later chunk's decays to sum meanwhile, and takes no tile (of four waves: one less).
    static __device__ __forceinline__ void scores(char *scores, const char *lds, const Decays &d, float scale, int w, int lane) {
        if (NW == 8) {
            if (w < 7) score_tile(scores, lds, d, scale, w, lane);
            if (w < 3) score_tile(scores, lds, d, scale, 7 + w, lane);
        } else {
            score_tile(scores, lds, d, scale, w, lane);
            score_tile(scores, lds, d, scale, 4 + w, lane);
            if (w < 2) score_tile(scores, lds, d, scale, 8 + w, lane);
        }
    }

    // O^T from the state before the chunk: o[b] register r is channel 16 w + 4 (l / 16) + r, token 16 b + l % 16
    __device__ __forceinline__ void from_state(const char *lds, const Decays &d, float scale, int lane) {
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        const int l = lane & 15, g = lane >> 4;
#pragma unroll
        for (int x = 0; x < K / 32; ++x) {
            float s[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] = S[2 * x + (i >> 2)][i & 3];
            bf16x8 p[PARTS], f[4];
#pragma unroll
            for (int i = 0; i < PARTS - 1; ++i) split_bf16(s, p[i]);
            p[PARTS - 1] = to_frag(s, bf16x8{});
#pragma unroll
            for (int b = 0; b < 4; ++b) f[b] = row<CK>(lds + kQ, 16 * b + l, 4 * x + g);
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b) o[b] = mma16(p[i], f[b], x + i == 0 ? zero : o[b]);
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const float e = scale * d.grown[16 * b + l];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[b][r] *= e;
        }
    }

    // adds V^T P^T
    __device__ __forceinline__ void from_chunk(const char *scores, const char *lds, bool odd, int w, int lane) {
#pragma unroll
        for (int y = 0; y < 2; ++y) vf[y] = values(lds, y, w, lane);
        if (odd)
            from_odd_chunk(scores, lds, w, lane);
        else
            times_scores(vf, scores, lane);
    }
    __device__ __forceinline__ void times_scores(const bf16x8 (&vf)[2], const char *scores, int lane) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
#pragma unroll
                for (int b = 2 * y; b < 4; ++b)
                    o[b] = mma16(vf[y], row<8>(scores + part * C * C * 2, 16 * b + (lane & 15), 4 * y + (lane >> 4)), o[b]);
    }
    // The same where some value is an infinity or NaN: a masked score's 0 times it would be NaN, so such
    // values are taken out of the products and added to the rows that they reach one by one.
    __device__ __forceinline__ void from_odd_chunk(const char *scores, const char *lds, int w, int lane) {
        bf16x8 fine[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            u32x4 u = __builtin_bit_cast(u32x4, vf[y]);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] &= ~((not_finite<bf16_t>(u[i]) >> 15) * 0xFFFFu);
            fine[y] = __builtin_bit_cast(bf16x8, u);
        }
        times_scores(fine, scores, lane);
#pragma unroll 1
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int i = 16 * b + (lane & 15), p = at<8>(i, j >> 3) + 2 * (j & 7);
                float s = 0.f;
#pragma unroll
                for (int part = 0; part < PARTS; ++part) s += bf16_to_f32(*reinterpret_cast<const bf16_t *>(scores + p + part * C * C * 2));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int c = 16 * w + 4 * (lane >> 4) + r;
                    const float x = bf16_to_f32(*reinterpret_cast<const bf16_t *>(lds + kV + at<CV>(j, c >> 3) + 2 * (c & 7)));
                    if (j <= i && !(fabsf(x) < INFINITY)) o[b][r] += s * x;
                }
            }
    }

    // the wave's columns of the outputs into their tile
    __device__ __forceinline__ void stage(char *outs, int w, int lane) const {
        const int l = lane & 15, g = lane >> 4;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            if (kHalf) {
                const bf16x2 x = pack_bf16(o[b][0], o[b][1]), y = pack_bf16(o[b][2], o[b][3]);
                *reinterpret_cast<bf16x4 *>(outs + at<CV>(16 * b + l, 2 * w + (g >> 1)) + 8 * (g & 1)) = (bf16x4){x[0], x[1], y[0], y[1]};
            } else {
                *reinterpret_cast<f32x4 *>(outs + wide_at(16 * b + l, 4 * w + g)) = o[b];
            }
        }
    }
    static __device__ __forceinline__ int wide_at(int t, int c) { return t * (V * 4) + 16 * (c ^ (t & 15)); }
    // whole rows of that tile, `count` of them, to memory
    static __device__ __forceinline__ void store(char *out, int64_t stride, const char *outs, int count, int tid) {
        constexpr int P = V * kOutBytes / 16;
#pragma unroll
        for (int i = 0; i < C * P / NT; ++i) {
            const int t = (i * NT + tid) / P, c = tid % P;
            const u32x4 x = *reinterpret_cast<const u32x4 *>(outs + (kHalf ? at<CV>(t, c) : wide_at(t, c)));
            if (t < count) __builtin_nontemporal_store(x, reinterpret_cast<u32x4 *>(out + t * stride + 16 * c));
        }
    }

    // S = e^(G_C) S + K^T (V e^(G_C - G_j)), the first factor only where DECAY
    template <bool DECAY> __device__ __forceinline__ void update(const bf16x8 (&vf)[2], const char *lds, const Decays &d, int lane) {
        if (DECAY) {
            const float all = d.grown[C - 1];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][r] *= all;
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float f[8];
            widen(vf[y], f);
            const float *e = d.left + 32 * y + 8 * (lane >> 4);
            const f32x4 a = *reinterpret_cast<const f32x4 *>(e), b = *reinterpret_cast<const f32x4 *>(e + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] *= a[i];
                f[4 + i] *= b[i];
            }
            bf16x8 p[3];
            split_bf16(f, p[0]);
            split_bf16(f, p[1]);
            p[2] = to_frag(f, bf16x8{});
#pragma unroll
            for (int m0 = 0; m0 < M; m0 += 4) {
                bf16x8 kf[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) kf[m] = keys(lds, y, m0 + m, lane);
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int m = 0; m < 4; ++m) S[m0 + m] = mma16(kf[m], p[i], S[m0 + m]);
            }
        }
    }
    template <bool DECAY> __device__ __forceinline__ void update(const char *lds, const Decays &d, int w, int lane) {
        lane = opaque(lane);
        const bf16x8 vf[2] = {values(lds, 0, w, lane), values(lds, 1, w, lane)};
        update<DECAY>(vf, lds, d, lane);
    }

    __device__ __forceinline__ void advance(const char *lds, const Decays &d, int, int lane) { update<true>(vf, lds, d, lane); }

    // the state as the registers hold it, in memory
    __device__ __forceinline__ void put(float *p, int w, int lane) const {
#pragma unroll
        for (int m = 0; m < M; ++m) *reinterpret_cast<f32x4 *>(p + ((w * M + m) * 64 + lane) * 4) = S[m];
    }
    __device__ __forceinline__ void get(const float *p, int w, int lane) {
#pragma unroll
        for (int m = 0; m < M; ++m) S[m] = *reinterpret_cast<const f32x4 *>(p + ((w * M + m) * 64 + lane) * 4);
    }
    // S = S + e first
    __device__ __forceinline__ void add(const LinBf16 &first, float e) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = fmaf(e, first.S[m][r], S[m][r]);
    }
    // a [K, V] state
    __device__ __forceinline__ void take(const float *p, int w, int lane) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[m][r] = p[element(m, r, w, lane)];
    }
    __device__ __forceinline__ void give(float *p, int w, int lane) const {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) p[element(m, r, w, lane)] = S[m][r];
    }
    static __device__ __forceinline__ int element(int m, int r, int w, int lane) {
        return (32 * (m >> 1) + 8 * (lane >> 4) + 4 * (m & 1) + r) * V + 16 * w + (lane & 15);
    }
};

}  // namespace kda
