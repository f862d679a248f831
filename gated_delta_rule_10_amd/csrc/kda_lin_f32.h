// The chunk step of kda_lin_chunk.hip for fp32 inputs, with fp32 matrix
// instructions: the products of kda_lin_bf16.h, nothing rounded below fp32.
//
// 32 tokens to a chunk. A wave holds 32 value channels: S[m] register r of lane l
// is value channel l % 32 and key channel M (8 (r / 4) + 4 (l / 32) + r % 4) + m,
// so that one read of M neighbouring key channels serves M products, both where k
// is multiplied into the state and where the state is read.
#pragma once

#include "kda_attn_device.h"
#include "kda_lin_device.h"

namespace kda {

__device__ __forceinline__ f32x16 mma32(float a, float b, f32x16 c) { return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0); }

template <int K, int V, bool OUT_> struct LinF32 {
    using T = float;
    static constexpr bool OUT = OUT_;
    static constexpr int C = 32, NW = V / 32, NT = 64 * NW, M = K / 32;
    static constexpr int kWavesPerSimd = 2;
    static constexpr int CK = K / 4, CV = V / 4;              // 16-byte pieces of a row
    static constexpr int LK = C * CK / NT, LV = C * CV / NT;  // of a thread
    static constexpr int kQ = 0, kK = OUT ? C * K * 4 : 0, kV = kK + C * K * 4;  // in LDS
    static constexpr int kTiles = kV + C * V * 4, kScores = OUT ? C * C * 4 : 0;
    typedef float keys_t __attribute__((ext_vector_type(M)));

    // piece c of row t: 16 rows read at one piece fall on different banks
    template <int CH> static __device__ __forceinline__ int at(int t, int c) { return t * (CH * 16) + 16 * (c ^ (CH == 8 ? (t >> 1) & 7 : t & 15)); }

    f32x4 q[OUT ? LK : 1], k[LK], v[LV];  // the next chunk, on its way
    f32x16 S[M], o;                       // the state; the chunk's outputs, transposed

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[m][r] = 0.f;
    }
    // what no chunk writes: the scores of the first 16 rows for the last 16 columns are 0
    static __device__ __forceinline__ void prepare(char *scores, int tid) {
        if (OUT && tid < 64) *reinterpret_cast<f32x4 *>(scores + at<8>(tid & 15, 4 + (tid >> 4))) = f32x4{0.f, 0.f, 0.f, 0.f};
    }

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
    // M neighbouring key channels of a row
    static __device__ __forceinline__ keys_t keys(const char *p, int t, int group) {
        return *reinterpret_cast<const keys_t *>(p + at<CK>(t, group * M / 4) + (M == 2 ? 8 * (group & 1) : 0));
    }

    // 16 x 16 scores
    static __device__ __forceinline__ void score_tile(char *scores, const char *lds, const Decays &d, float scale, int i0, int j0, int lane) {
        const int l = lane & 15, g = lane >> 4, i = i0 + l, j = j0 + 4 * g;  // p[r]: row i, column j + r
        f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < CK / 4; ++x)
            p = mma16(*reinterpret_cast<const f32x4 *>(lds + kK + at<CK>(j0 + l, 4 * x + g)),
                      *reinterpret_cast<const f32x4 *>(lds + kQ + at<CK>(i, 4 * x + g)), p);
        const f32x4 dh = *reinterpret_cast<const f32x4 *>(d.hi + j), dl = *reinterpret_cast<const f32x4 *>(d.lo + j);
        const float hi = d.hi[i], lo = d.lo[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = j + r <= i ? p[r] * (scale * __builtin_amdgcn_exp2f((hi - dh[r]) + (lo - dl[r]))) : 0.f;
        *reinterpret_cast<f32x4 *>(scores + at<8>(i, j >> 2)) = p;
    }
    // the three tiles on and below the diagonal; the last wave has a later chunk's decays to sum
    static __device__ __forceinline__ void scores(char *scores, const char *lds, const Decays &d, float scale, int w, int lane) {
        if (w < 3 && w < NW) score_tile(scores, lds, d, scale, w ? 16 : 0, w == 2 ? 16 : 0, lane);
        if (NW == 2 && w == 0) score_tile(scores, lds, d, scale, 16, 16, lane);
    }

    // O^T from the state before the chunk: column l % 32 is the token
    __device__ __forceinline__ void from_state(const char *lds, const Decays &d, float scale, int lane) {
        o = f32x16{};
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const keys_t x = keys(lds + kQ, lane & 31, 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3));
#pragma unroll
            for (int m = 0; m < M; ++m) o = mma32(S[m][r], x[m], o);
        }
        const float e = scale * d.grown[lane & 31];
#pragma unroll
        for (int r = 0; r < 16; ++r) o[r] *= e;
    }

    // Adds V^T P^T, tokens 8 (r / 4) + 4 (l / 32) + r % 4 in step r. A masked score's 0 times an infinity or
    // NaN would be NaN: such values are left out of the products and added to the rows that they reach.
    __device__ __forceinline__ void from_chunk(const char *scores, const char *lds, bool odd, int w, int lane) {
        const int half = lane >> 5, i = lane & 31;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x4 p = *reinterpret_cast<const f32x4 *>(scores + at<8>(i, 2 * c + half));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = value(lds, 8 * c + 4 * half + e, 32 * w + i);
                if (odd && !(fabsf(x) < INFINITY)) x = 0.f;
                o = mma32(x, p[e], o);
            }
        }
        if (!odd) return;
#pragma unroll 1
        for (int j = 0; j < C; ++j) {
            const float p = *reinterpret_cast<const float *>(scores + at<8>(i, j >> 2) + 4 * (j & 3));
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float x = value(lds, j, 32 * w + 8 * (r >> 2) + 4 * half + (r & 3));
                if (j <= i && !(fabsf(x) < INFINITY)) o[r] += p * x;
            }
        }
    }

    template <bool DECAY> __device__ __forceinline__ void update(const char *lds, const Decays &d, int w, int lane) {
        const int half = lane >> 5, l = lane & 31;
        if (DECAY) {
            const float all = d.grown[C - 1];
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int r = 0; r < 16; ++r) S[m][r] *= all;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const f32x4 e = *reinterpret_cast<const f32x4 *>(d.left + 8 * c + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 8 * c + 4 * half + i;
                const float x = e[i] * value(lds, t, 32 * w + l);
                const keys_t y = keys(lds + kK, t, l);
#pragma unroll
                for (int m = 0; m < M; ++m) S[m] = mma32(y[m], x, S[m]);
            }
        }
    }

    __device__ __forceinline__ void store(float *out, int64_t stride, char *, int count, int w, int lane) const {
        const int half = lane >> 5, t = lane & 31;
        if (t < count)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<f32x4 *>(out + t * stride + 32 * w + 8 * c + 4 * half) = (f32x4){o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]};
    }
    __device__ __forceinline__ void advance(const char *lds, const Decays &d, int w, int lane) { update<true>(lds, d, w, lane); }

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
    // S = S + e first
    __device__ __forceinline__ void add(const LinF32 &first, float e) {
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int r = 0; r < 16; ++r) S[m][r] = fmaf(e, first.S[m][r], S[m][r]);
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
    static __device__ __forceinline__ int element(int m, int r, int w, int lane) {
        return (M * (8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) + m) * V + 32 * w + (lane & 31);
    }
};

}  // namespace kda
