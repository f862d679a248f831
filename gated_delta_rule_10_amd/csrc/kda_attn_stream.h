// Attention of a tile of R = 16 rows over a run of keys and values, streamed
// once: o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m), s_j = c q.k_j in the
// log2 domain, with the running maximum m and sum kept per row in fp32.
//
// Rows. The rows of a (sequence, kv head) are its tokens times the G query
// heads that share the kv head: row r is token r / G, head r % G, so that every
// key and value read serves all of them.
//
// Work of a workgroup: four waves; a step gives each wave 32 consecutive
// tokens (fp32: 16, so that two workgroups fit a compute unit's LDS). Each wave
// keeps its own m, sum and output over its tokens (no barrier while streaming)
// and the four are joined at the end. A wave holds the next step's keys and
// values in registers while it works on the current ones, which lie in its own
// part of LDS. Two steps ahead, and three or four workgroups to a compute unit
// with smaller steps, were slower for an e4m3 cache.
//
// Products (16 x 16 matrix instructions, 32-deep). S^T = K Q^T puts a row's
// scores for tokens 16 b + 4 g + i (g = lane / 16) into registers of the lanes
// of that row, so the softmax needs two lane swaps per step. These registers
// are the B operand of O^T = V^T P^T as they are, once V^T's fragments take the
// tokens in the same order {4 g + 0..3, 16 + 4 g + 0..3}, which the transposing
// LDS reads give without any movement of P.
#pragma once

#include <type_traits>

#include "kda_attn_rows.h"

namespace kda {

constexpr int kWaves = 4;

template <int K, int V, typename TC> struct Stream {
    using Frag = typename mma_of<TC>::frag;
    using Elem = typename mma_of<TC>::elem;  // of q
    static constexpr int R = 16;
    static constexpr int ES = sizeof(TC);
    static constexpr bool kCodes = sizeof(TC) == 1;
    static constexpr int NB = ES == 4 ? 1 : 2;             // groups of 16 tokens per wave and step
    static constexpr int kStepWave = 16 * NB;              // tokens per wave and step
    static constexpr int kStep = kWaves * kStepWave;       // tokens per workgroup and step
    static constexpr int NT = 4 * NB;                      // of them, tokens in a lane's registers
    using PFrag = typename std::conditional<ES == 4, f32x4, bf16x8>::type;  // weights, values: NT tokens
    static constexpr int CK = K * ES / 16, CV = V * ES / 16;  // 16-byte chunks per row
    static constexpr int NK = kStepWave * CK / 64, NV = kStepWave * CV / 64;  // chunks per lane and step
    static constexpr int KT = K / 32, VT = V / 16;
    static constexpr int KB = kStepWave * K * ES, VB = kStepWave * V * ES;    // LDS bytes per wave
    static constexpr int kJoinRow = V + 4;                                    // floats per row of a join tile
    static constexpr int kJoin = kWaves * R * kJoinRow * 4;
    static constexpr int kRing = kWaves * (KB + VB);
    static constexpr int kLds = kRing > kJoin ? kRing : kJoin;

    // Chunk places in LDS: the tokens that one read instruction takes from a
    // column of chunks are spread over the banks.
    static __device__ __forceinline__ int swz_k(int t) { return t & (CK < 8 ? CK - 1 : 7); }
    static __device__ __forceinline__ int swz_v(int t) {
        if (ES == 2) return (2 * t) & (CV - 1);
        if (ES == 1) return (t + (t >> 4) * 4) & (CV - 1);
        return (4 * (t >> 2)) & (CV - 1);
    }

    Frag q[KT];
    f32x4 o[VT];
    float m, l;  // of row l % 16; the sum is this lane's share
    // keys, values and exponents on their way, of the next step
    struct Ahead {
        u32x4 kr[NK], vr[NV];
        uint32_t ke[NB], ve[NB];
        bool here[NB];  // whether the pages of the groups of 16 tokens exist
    } next;

    __device__ __forceinline__ void reset() {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int d = 0; d < VT; ++d) o[d] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }

    // Rows from r0 on of (sequence rows from `start`, kv head kvh): fragments of q.
    // Rows past `rows` repeat the last one and are not stored.
    __device__ __forceinline__ void load_q(const AttnArgs &a, int start, int kvh, int r0, int rows, int lane) {
        const int g = lane >> 4, r = r0 + min(lane & 15, rows - 1);
        const int tok = r / a.G, h = kvh * a.G + (r - tok * a.G);
        const Elem *p = static_cast<const Elem *>(a.q) + static_cast<int64_t>(start + tok) * a.qs + h * K + 8 * g;
#pragma unroll
        for (int s = 0; s < KT; ++s) q[s] = load_frag(p + 32 * s);
    }

    // ---- sources: chunk x of a wave's kStepWave tokens
    // cache: row[b] is the cache row of the first of tokens 16 b .. 16 b + 15 (a page ends at a multiple of
    // 16, so the 16 rows lie behind one another)
    static __device__ __forceinline__ void load_cache(Ahead &n, const AttnArgs &a, const int64_t (&row)[NB], int lane) {
        const char *k[NB], *v[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            k[b] = static_cast<const char *>(a.k) + row[b] * (K * ES);
            v[b] = static_cast<const char *>(a.v) + row[b] * (V * ES);
        }
        const uint32_t at = 16 * lane;
#pragma unroll
        for (int x = 0; x < NK; ++x)
            n.kr[x] = *reinterpret_cast<const u32x4 *>(k[NB * x / NK] + at + (x % (NK / NB)) * 1024);
#pragma unroll
        for (int x = 0; x < NV; ++x)
            n.vr[x] = *reinterpret_cast<const u32x4 *>(v[NB * x / NV] + at + (x % (NV / NB)) * 1024);
        if (kCodes) {
            const uint32_t g = 4 * (lane >> 4);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                n.ke[b] = *reinterpret_cast<const uint32_t *>(a.kexp + row[b] + g);
                n.ve[b] = *reinterpret_cast<const uint32_t *>(a.vexp + row[b] + g);
            }
        }
    }
    // packed tokens of the call (fp32): a position past the last token reads the last one and is masked
    static __device__ __forceinline__ void load_packed(Ahead &n, const AttnArgs &a, int start, int kvh, int p0, int lane) {
        static_assert(ES == 4, "bf16 prompts have their own kernel");
        n.here[0] = true;
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int e = x * 64 + lane, t = e / CK, c = e % CK;
            const int64_t row = min(start + p0 + t, a.T - 1);
            n.kr[x] = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(
                        static_cast<const TC *>(a.k) + row * a.ks + kvh * K) + 16 * c);
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int e = x * 64 + lane, t = e / CV, c = e % CV;
            const int64_t row = min(start + p0 + t, a.T - 1);
            n.vr[x] = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const char *>(
                        static_cast<const TC *>(a.v) + row * a.vs + kvh * V) + 16 * c);
        }
    }

    // Registers to this wave's LDS. `masked`: tokens that nobody may see (their page is missing,
    // or position >= end) get zero values. The result says whether values that step() must not
    // multiply as they are, infinities and NaN, are among the rest: of masked steps in any
    // type (a row that does not see them), of bf16 in all steps (the second part of a weight may
    // be 0 or negative: an infinity times it would be NaN). The check on all steps costs nothing
    // beside the loads: 248 us with and without it for 64 sequences of 1000 to 16000 tokens.
    static __device__ __forceinline__ bool stage(Ahead &n, char *lk, char *lv, bool masked, int p0, int end, int lane) {
        uint32_t odd = 0;
        if (masked) {
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const int t = (x * 64 + lane) / CV;
                if (p0 + t >= end || !n.here[NB == 1 || t < 16 ? 0 : NB - 1]) n.vr[x] = (u32x4){0, 0, 0, 0};
            }
        }
        if (masked || ES == 2) {
#pragma unroll
            for (int x = 0; x < NV; ++x)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd |= not_finite<TC>(n.vr[x][j]);
        }
#pragma unroll
        for (int x = 0; x < NK; ++x) {
            const int e = x * 64 + lane, t = e / CK, c = e % CK;
            *reinterpret_cast<u32x4 *>(lk + t * (K * ES) + 16 * (c ^ swz_k(t))) = n.kr[x];
        }
#pragma unroll
        for (int x = 0; x < NV; ++x) {
            const int e = x * 64 + lane, t = e / CV, c = e % CV;
            *reinterpret_cast<u32x4 *>(lv + t * (V * ES) + 16 * (c ^ swz_v(t))) = n.vr[x];
        }
        return __any(odd != 0);
    }

    __device__ __forceinline__ Frag k_frag(const char *lk, int b, int s, int lane) const {
        const int t = 16 * b + (lane & 15), g = lane >> 4;
        const char *row = lk + t * (K * ES);
        if constexpr (ES == 2) {
            return *reinterpret_cast<const Frag *>(row + 16 * ((4 * s + g) ^ swz_k(t)));
        } else if constexpr (ES == 1) {
            const uint2 w = *reinterpret_cast<const uint2 *>(row + 16 * ((2 * s + (g >> 1)) ^ swz_k(t)) + 8 * (g & 1));
            return codes_to_bf16(w.x, w.y, 1.f);
        } else {
            const f32x4 x = *reinterpret_cast<const f32x4 *>(row + 16 * ((8 * s + 2 * g) ^ swz_k(t)));
            const f32x4 y = *reinterpret_cast<const f32x4 *>(row + 16 * ((8 * s + 2 * g + 1) ^ swz_k(t)));
            return (f32x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        }
    }
    // V^T: channel 16 d + l % 16, tokens 4 g + 0..3 and (bf16 products) 16 + 4 g + 0..3
    __device__ __forceinline__ PFrag v_frag(const char *lv, int d, int lane) const {
        const int i = lane & 15, g = lane >> 4;
        if constexpr (ES == 2) {
            typedef __attribute__((address_space(3))) i16x4 lds4;
            const int t = 4 * g + (i >> 2), c = 2 * d + ((i >> 1) & 1);
            const char *p = lv + t * (V * 2) + 16 * (c ^ swz_v(t)) + 8 * (i & 1);
            const char *p2 = lv + (t + 16) * (V * 2) + 16 * (c ^ swz_v(t + 16)) + 8 * (i & 1);
            const bf16x4 x = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p));
            const bf16x4 y = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p2));
            return (bf16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
        } else if constexpr (ES == 1) {
            typedef __attribute__((address_space(3))) i32x2 lds2;
            const int r = i >> 1, t = (r & 3) + 4 * g + (r >> 2) * 16;
            const char *p = lv + t * V + 16 * (d ^ swz_v(t)) + 8 * (i & 1);
            const i32x2 w = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2 *)p);
            return codes_to_bf16(w[0], w[1], 1.f);
        } else {
            f32x4 x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = j + 4 * g, ch = 16 * d + i;
                x[j] = *reinterpret_cast<const float *>(lv + t * (V * 4) + 16 * ((ch >> 2) ^ swz_v(t)) + 4 * (ch & 3));
            }
            return x;
        }
    }
    // channels 16 d + 4 g + 0..3 of token t, as floats (the slow product below)
    __device__ __forceinline__ f32x4 v_row(const char *lv, int t, int d, int lane) const {
        const int ch = 16 * d + 4 * (lane >> 4), byte = ch * ES;
        const char *p = lv + t * (V * ES) + 16 * ((byte >> 4) ^ swz_v(t)) + (byte & 15);
        if constexpr (ES == 4) return *reinterpret_cast<const f32x4 *>(p);
        if constexpr (ES == 2) {
            const float4 x = io<bf16_t>::load4(reinterpret_cast<const bf16_t *>(p));
            return (f32x4){x.x, x.y, x.z, x.w};
        }
        const bf16x8 x = codes_to_bf16(*reinterpret_cast<const uint32_t *>(p), 0, 1.f);
        return (f32x4){static_cast<float>(x[0]), static_cast<float>(x[1]), static_cast<float>(x[2]), static_cast<float>(x[3])};
    }

    // One step over the kStepWave staged tokens. sees bit (4 b + j): row l % 16 sees token 16 b + 4 g + j
    // (read only when masked). kx, vx: exponents of these tokens.
    __device__ __forceinline__ void step(const char *lk, const char *lv, float c, bool masked, uint32_t sees, bool odd, const uint32_t (&kx)[NB], const uint32_t (&vx)[NB], int lane) {
        f32x4 s[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            s[b] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KT; ++ks) s[b] = mma16(k_frag(lk, b, ks, lane), q[ks], s[b]);
        }
        float x[NT], pf[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            x[j] = s[j >> 2][j & 3] * c;
            if (kCodes) x[j] = scaled_by(x[j], kx[j >> 2], j & 3);
            if (masked) x[j] = (sees >> j) & 1u ? x[j] : -INFINITY;
        }
        float t = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
        for (int j = 4; j < NT; j += 4) t = fmaxf(t, fmaxf(fmaxf(x[j], x[j + 1]), fmaxf(x[j + 2], x[j + 3])));
        t = fmaxf(t, kLowest);
        if (masked) t = sees ? t : -INFINITY;
        t = swap32_max(swap16_max(t));
        // The reference m only has to keep 2^(s - m) in range, so it moves when the
        // step's maximum passes it by more than 2^8, not at every step.
        if (__any(t > m + 8.f)) {
            const float mn = fmaxf(m, t);
            const float f = mn == -INFINITY ? 1.f : exp2f(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int d = 0; d < VT; ++d) o[d] *= f;
        }
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            pf[j] = __builtin_amdgcn_exp2f(x[j] - ref);
            l += pf[j];
            if (kCodes) pf[j] = scaled_by(pf[j], vx[j >> 2], j & 3);
        }
        const PFrag p = to_frag(pf, PFrag{});
        if (!odd) {
            PFrag rest;  // of the weights, what bf16 leaves
            if constexpr (ES != 4) {
                float r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = pf[j] - static_cast<float>(p[j]);
                rest = to_frag(r, PFrag{});
            }
#pragma unroll
            for (int d = 0; d < VT; ++d) {
                const PFrag vf = v_frag(lv, d, lane);
                if constexpr (ES != 4) o[d] = mma16(vf, rest, o[d]);
                o[d] = mma16(vf, p, o[d]);
            }
            return;
        }
        // An infinity or NaN among the values (stage()): a weight of zero would not keep it out of a
        // matrix product, so each token is added to the rows that see it.
#pragma unroll 1
        for (int t = 0; t < kStepWave; ++t) {
            const int j = 4 * (t >> 4) + (t & 3), src = 4 * (t & 12) + (lane & 15);  // its register, its lanes
            float w = 0.f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i == j) w = pf[i];
            w = __shfl(w, src);
            const bool see = !masked || (__shfl(sees, src) >> j) & 1u;
#pragma unroll
            for (int d = 0; d < VT; ++d) {
                const f32x4 y = v_row(lv, t, d, lane);
                if (see) o[d] += y * w;
            }
        }
    }

    // Which tokens the lane's row sees in a masked step (seen_tokens), as step() takes them
    __device__ __forceinline__ uint32_t visible(const AttnArgs &a, int start, int r0, int rows, int p0, int ctx, int end,
                                                const bool (&here)[NB], int lane) const {
        const int g = 4 * (lane >> 4), tok = (r0 + min(lane & 15, rows - 1)) / a.G;
        const uint64_t bits = a.mask ? a.mask[start + tok] : 0;
        const uint32_t w = static_cast<uint32_t>(
            seen_tokens(a.mask != nullptr, bits, p0, ctx, ctx + tok, end, (here[0] ? 1 : 0) | (here[NB - 1] ? 2 : 0)));
        const uint32_t sees = (w >> g) & 15u;
        return NB == 2 ? sees | ((w >> (16 + g)) & 15u) << 4 : sees;
    }

    // Join the four waves' results and hand out rows: put(row in tile, channel, maximum, float4
    // of unnormalised outputs, sum). Every thread of the workgroup calls it.
    template <typename Put>
    __device__ __forceinline__ void join(char *lds, float (&stat)[2][kWaves][R], int w, int lane, int rows, Put put) {
        const int r = lane & 15, g = lane >> 4, tid = w * 64 + lane;
        l = swap32_sum(swap16_sum(l));
        if (g == 0) stat[0][w][r] = m;
        __syncthreads();
        float mm = stat[0][0][r];
#pragma unroll
        for (int u = 1; u < kWaves; ++u) mm = fmaxf(mm, stat[0][u][r]);
        // a wave that saw nothing of a row holds zeros for it
        const float f = m == -INFINITY ? 0.f : exp2f(m - mm);
        if (g == 0) stat[1][w][r] = l * f;
        float *tile = reinterpret_cast<float *>(lds);
#pragma unroll
        for (int d = 0; d < VT; ++d) *reinterpret_cast<f32x4 *>(tile + (w * R + r) * kJoinRow + 16 * d + 4 * g) = o[d] * f;
        __syncthreads();
        for (int e = tid; e < R * (V / 4); e += 64 * kWaves) {
            const int row = e / (V / 4), ch = 4 * (e % (V / 4));
            if (row < rows) {
                f32x4 x = *reinterpret_cast<const f32x4 *>(tile + row * kJoinRow + ch);
                float mj = stat[0][0][row], ll = stat[1][0][row];
#pragma unroll
                for (int u = 1; u < kWaves; ++u) {
                    x += *reinterpret_cast<const f32x4 *>(tile + (u * R + row) * kJoinRow + ch);
                    mj = fmaxf(mj, stat[0][u][row]);
                    ll += stat[1][u][row];
                }
                put(row, ch, mj, x, ll);
            }
        }
        __syncthreads();
    }
};

}  // namespace kda
