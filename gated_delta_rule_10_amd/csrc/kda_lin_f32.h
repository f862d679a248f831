// The chunk step of kda_lin_chunk.hip for fp32 inputs, with fp32 matrix
// instructions: the products of kda_lin_bf16.h, nothing rounded below fp32.
//
// 32 tokens to a chunk. A wave holds 16 value channels: S[m] register r of lane l
// is value channel l % 16 and key channel 64 (m / 4) + 16 (l / 16) + 4 r + m % 4, so
// that one read of 4 neighbouring key channels serves 4 products, both where k is
// multiplied into the state and where the state is read. (A piece of 4 key channels is
// 16 bytes as 8 are in bf16: 32 tokens fill the LDS that 64 fill there.)
//
// Bound by the matrix instructions, at an eighth of the bf16 rate: a chunk of 32 tokens
// takes 5.9 us of one workgroup. Sequences of 4000, 37 and 411 tokens, H = 16, 128
// channels: 111 us (35 for the ends, 73 for the outputs). The definition's operations are
// 4.7 GFLOP, 30 us at the rate of a large fp32 product (154 TFLOP/s); these are 7.9, 51 us: 0.9
// more for the scores and their products with v in tiles of 16 x 16, and 2.3 for the
// ends' updates, which the outputs repeat.
#pragma once

#include "kda_attn_device.h"
#include "kda_lin_device.h"

namespace kda {

// 4 products: one a lane of the lanes of one l / 16
__device__ __forceinline__ f32x4 mma16(float a, float b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

template <int K, int V, bool OUT_> struct LinF32 {
    using T = float;
    static constexpr bool OUT = OUT_;
    static constexpr int C = 32, NW = V / 16, NT = 64 * NW, M = K / 16;
    static constexpr int kWavesPerSimd = 2;
    static constexpr int CK = K / 4, CV = V / 4;              // 16-byte pieces of a row
    static constexpr int LK = C * CK / NT, LV = C * CV / NT;  // of a thread
    static constexpr int kQ = 0, kK = OUT ? C * K * 4 : 0, kV = kK + C * K * 4;  // in LDS
    static constexpr int kTiles = kV + C * V * 4, kScores = OUT ? C * C * 4 : 0, kOuts = C * V * 4;

    // piece c of row t: 16 rows read at one piece, and one piece of 4 rows in a row's order, fall on different banks
    template <int CH> static __device__ __forceinline__ int at(int t, int c) { return t * (CH * 16) + 16 * (c ^ (CH == 8 ? (t >> 1) & 7 : t & 15)); }

    f32x4 q[OUT ? LK : 1], k[LK], v[LV];  // the next chunk, on its way
    f32x4 S[M], o[2];                     // the state; the chunk's outputs, transposed

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int m = 0; m < M; ++m) S[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // (no product reads the scores of the first 16 rows for the last 16 columns, which no chunk writes)
    static __device__ __forceinline__ void prepare(char *, int) {}

    // Rows from `count` on are the last one again: their scores are masked and their values weigh 0.
    template <int CH, int L> static __device__ __forceinline__ void load_rows(f32x4 (&x)[L], const T *p, int64_t stride, int count, int tid) {
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int t = min(i * (NT / CH) + tid / CH, count - 1);
            x[i] = *reinterpret_cast<const f32x4 *>(p + t * stride + 4 * (tid % CH));
        }
    }
    template <int CH, int L> static __device__ __forceinline__ void store_rows(const f32x4 (&x)[L], char *p, int tid) {
#pragma unroll
        for (int i = 0; i < L; ++i) *reinterpret_cast<f32x4 *>(p + at<CH>(i * (NT / CH) + tid / CH, tid % CH)) = x[i];
    }
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
        bool odd = false;
        if (OUT)
#pragma unroll
            for (int i = 0; i < LV; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd |= !(fabsf(v[i][j]) < INFINITY);
        return odd;
    }

    static __device__ __forceinline__ float value(const char *lds, int t, int c) {
        return *reinterpret_cast<const float *>(lds + kV + at<CV>(t, c >> 2) + 4 * (c & 3));
    }
    template <int CH> static __device__ __forceinline__ f32x4 row(const char *p, int t, int c) {
        return *reinterpret_cast<const f32x4 *>(p + at<CH>(t, c));
    }

    // 16 x 16 scores
    static __device__ __forceinline__ void score_tile(char *scores, const char *lds, const Decays &d, float scale, int i0, int j0, int lane) {
        const int l = lane & 15, g = lane >> 4, i = i0 + l, j = j0 + 4 * g;  // p[r]: row i, column j + r
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < CK / 4; ++x) p = mma16(row<CK>(lds + kK, j0 + l, 4 * x + g), row<CK>(lds + kQ, i, 4 * x + g), p);
        const f32x4 dh = *reinterpret_cast<const f32x4 *>(d.hi + j), dl = *reinterpret_cast<const f32x4 *>(d.lo + j);
        const float hi = d.hi[i], lo = d.lo[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = j + r <= i ? p[r] * (scale * __builtin_amdgcn_exp2f((hi - dh[r]) + (lo - dl[r]))) : 0.f;
        *reinterpret_cast<f32x4 *>(scores + at<8>(i, j >> 2)) = p;
    }
    // the three tiles on and below the diagonal; the last wave has a later chunk's decays to sum
    static __device__ __forceinline__ void scores(char *scores, const char *lds, const Decays &d, float scale, int w, int lane) {
        if (w < 3) score_tile(scores, lds, d, scale, w ? 16 : 0, w == 2 ? 16 : 0, lane);
    }

    // O^T from the state before the chunk: o[b] register r is channel 16 w + 4 (l / 16) + r, token 16 b + l % 16
    __device__ __forceinline__ void from_state(const char *lds, const Decays &d, float scale, int lane) {
        const int l = lane & 15, g = lane >> 4;
        o[0] = o[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < M / 4; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                f32x4 f[2];
#pragma unroll
                for (int b = 0; b < 2; ++b) f[b] = row<CK>(lds + kQ, 16 * b + l, 16 * x + 4 * g + r);
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int b = 0; b < 2; ++b) o[b] = mma16(S[4 * x + m][r], f[b][m], o[b]);
            }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const float e = scale * d.grown[16 * b + l];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[b][r] *= e;
        }
    }

    // Adds V^T P^T, tokens 16 u + 4 (l / 16) + e at a time. A masked score's 0 times an infinity or NaN
    // would be NaN: such values are left out of the products and added to the rows that they reach.
    __device__ __forceinline__ void from_chunk(const char *scores, const char *lds, bool odd, int w, int lane) {
        const int l = lane & 15, g = lane >> 4;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            f32x4 p[2];
#pragma unroll
            for (int b = u; b < 2; ++b) p[b] = row<8>(scores, 16 * b + l, 4 * u + g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = value(lds, 16 * u + 4 * g + e, 16 * w + l);
                if (odd && !(fabsf(x) < INFINITY)) x = 0.f;
#pragma unroll
                for (int b = u; b < 2; ++b) o[b] = mma16(x, p[b][e], o[b]);
            }
        }
        if (!odd) return;
#pragma unroll 1
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int i = 16 * b + l;
                const float p = *reinterpret_cast<const float *>(scores + at<8>(i, j >> 2) + 4 * (j & 3));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = value(lds, j, 16 * w + 4 * g + r);
                    if (j <= i && !(fabsf(x) < INFINITY)) o[b][r] += p * x;
                }
            }
    }

    // the wave's columns of the outputs into their tile
    __device__ __forceinline__ void stage(char *outs, int w, int lane) const {
#pragma unroll
        for (int b = 0; b < 2; ++b) *reinterpret_cast<f32x4 *>(outs + at<CV>(16 * b + (lane & 15), 4 * w + (lane >> 4))) = o[b];
    }
    // whole rows of that tile, `count` of them, to memory
    static __device__ __forceinline__ void store(char *out, int64_t stride, const char *outs, int count, int tid) {
#pragma unroll
        for (int i = 0; i < LV; ++i) {
            const int t = i * (NT / CV) + tid / CV, c = tid % CV;
            const f32x4 x = row<CV>(outs, t, c);
            if (t < count) __builtin_nontemporal_store(x, reinterpret_cast<f32x4 *>(out + t * stride + 16 * c));
        }
    }

    // S = e^(G_C) S + K^T (V e^(G_C - G_j)), the first factor only where DECAY
    template <bool DECAY> __device__ __forceinline__ void update(const char *lds, const Decays &d, int w, int lane) {
        const int l = lane & 15, g = lane >> 4;
        if (DECAY) {
            const float all = d.grown[C - 1];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[m][r] *= all;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4 e = *reinterpret_cast<const f32x4 *>(d.left + 16 * u + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * u + 4 * g + i;
                const float x = e[i] * value(lds, t, 16 * w + l);
#pragma unroll
                for (int y = 0; y < M / 4; ++y) {
                    const f32x4 f = row<CK>(lds + kK, t, 16 * y + l);
#pragma unroll
                    for (int m = 0; m < 4; ++m) S[4 * y + m] = mma16(f[m], x, S[4 * y + m]);
                }
            }
        }
    }
    __device__ __forceinline__ void advance(const char *lds, const Decays &d, int w, int lane) { update<true>(lds, d, w, lane); }

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
    __device__ __forceinline__ void add(const LinF32 &first, float e) {
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
        return (64 * (m >> 2) + 16 * (lane >> 4) + 4 * r + (m & 3)) * V + 16 * w + (lane & 15);
    }
};

}  // namespace kda
