// Device pieces shared by the attention kernels: matrix-instruction fragments
// for the element types, e4m3 codes and their scales, and the map from a
// (sequence, kv head)'s rows to tokens and query heads.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_attn_internal.h"
#include "kda_device.h"

namespace kda {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

struct e4m3_t { uint8_t bits; };  // a code of an E4M3 cache

// Type of the products for a cache element: bf16 products hold bf16 and e4m3
// exactly (8 bits of significand against 4).
template <typename TC> struct mma_of { using frag = bf16x8; using elem = bf16_t; };
template <> struct mma_of<float> { using frag = f32x8; using elem = float; };

// c += a b over 32 products, 16 x 16: lane l holds row (column) l % 16 of a (b)
// at 8 places of the contraction, the same places for a and b in the lanes of
// one l / 16; c has column l % 16, rows 4 (l / 16) + 0..3.
__device__ __forceinline__ f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma16(f32x8 a, f32x8 b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// eight consecutive elements, 16-byte aligned
__device__ __forceinline__ bf16x8 load_frag(const bf16_t *p) { return *reinterpret_cast<const bf16x8 *>(p); }
__device__ __forceinline__ f32x8 load_frag(const float *p) {
    const f32x4 x = reinterpret_cast<const f32x4 *>(p)[0], y = reinterpret_cast<const f32x4 *>(p)[1];
    return (f32x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
}

__device__ __forceinline__ f32x4 mma16(f32x4 a, f32x4 b, f32x4 c) {  // 16 products, fp32
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
}

// two fp32 to bf16, nearest even (the gfx950 conversion keeps NaN)
__device__ __forceinline__ bf16x2 pack_bf16(float x, float y) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_convertvector((f32x2){x, y}, bf16x2);
}
__device__ __forceinline__ bf16x8 to_frag(const float *x, bf16x8) {
    const bf16x2 a = pack_bf16(x[0], x[1]), b = pack_bf16(x[2], x[3]), c = pack_bf16(x[4], x[5]), d = pack_bf16(x[6], x[7]);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ f32x4 to_frag(const float *x, f32x4) { return (f32x4){x[0], x[1], x[2], x[3]}; }

// eight e4m3 codes times a power of two as bf16, exactly
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t lo, uint32_t hi, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return (bf16x8){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x * 2^(byte - 127), byte i of w
__device__ __forceinline__ float scaled_by(float x, uint32_t w, int i) {
    return __builtin_ldexpf(x, static_cast<int>((w >> (8 * i)) & 255u) - 127);
}

__device__ __forceinline__ float swap16_max(float m) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float swap32_max(float m) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float swap16_sum(float m) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
__device__ __forceinline__ float swap32_sum(float m) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(m), __float_as_uint(m), false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// Not 0 if a register of elements holds an infinity or a NaN (e4m3: a NaN).
template <typename TC> __device__ __forceinline__ uint32_t not_finite(uint32_t x);
// an exponent of ones carries into the sign's place, no other does
template <> __device__ __forceinline__ uint32_t not_finite<float>(uint32_t x) { return ((x & 0x7F800000u) + 0x00800000u) & 0x80000000u; }
template <> __device__ __forceinline__ uint32_t not_finite<bf16_t>(uint32_t x) { return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
template <> __device__ __forceinline__ uint32_t not_finite<e4m3_t>(uint32_t x) {
    // a byte whose low seven bits are all ones: no borrow from the byte above
    const uint32_t y = ~x & 0x7F7F7F7Fu;
    return (y - 0x01010101u) & 0x80808080u & ~y;
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// the n lowest bits (none for n <= 0, all 64 from 64 on)
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Which of the 64 tokens from position p0 on a row sees, as bits: all before position `ctx`, and
// new token b = position - ctx if bit b of `bits` is set or, without a mask, up to `own`;
// none from position `end` on, and none of a group of 16 tokens whose bit in `here` is not set.
__device__ __forceinline__ uint64_t seen_tokens(bool mask, uint64_t bits, int p0, int ctx, int own, int end, uint32_t here) {
    const int b = p0 - ctx;  // of the first token
    uint64_t w = low_bits(own - p0 + 1);
    if (mask) w = b >= 64 ? 0 : b >= 0 ? bits >> b : b <= -64 ? ~0ull : bits << -b | low_bits(-b);
    const uint64_t groups = (here & 1 ? 0xFFFFull : 0) | (here & 2 ? 0xFFFFull << 16 : 0) | (here & 4 ? 0xFFFFull << 32 : 0) |
                            (here & 8 ? 0xFFFFull << 48 : 0);
    return w & low_bits(end - p0) & groups;
}

// Rows [start, start + count) of sequence n, inside [0, T] whatever cu holds.
__device__ __forceinline__ void seq_rows(const int32_t *cu, int n, int T, int &start, int &count) {
    start = clampi(ld_meta(cu, n), 0, T);
    count = clampi(ld_meta(cu, n + 1), start, T) - start;
}

// The last n in [0, N) with key(n) <= s, for keys that do not fall (0 if there is none; in [0, N)
// whatever the keys). A wave looks at 64 of them at a time: one load for up to 64 sequences, and
// none for one. All lanes take part and get the same answer.
template <typename Key> __device__ __forceinline__ int wave_last_upto(int N, int64_t s, int lane, Key key) {
    int lo = 0, len = N;
    while (len > 1) {
        const int step = (len + 63) / 64, at = lane * step;
        const bool upto = at < len && key(lo + at) <= s;
        const int some = static_cast<int>(__popcll(__ballot(upto)));  // (unsigned: less 1, none would be 2^32 - 1)
        const int i = (some > 0 ? some - 1 : 0) * step;
        lo += i;
        len = min(step, len - i);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Slot s of the slots that tiles of R rows take: a sequence with G rows per
// token owns the slots from floor(G cu[n] / R) + n on, at least as many as its
// ceil(G L / R) tiles, so a slot finds its sequence from cu alone.
__device__ __forceinline__ int seq_of_slot(const int32_t *cu, int N, int T, int G, int R, int64_t s, int lane) {
    return wave_last_upto(N, s, lane, [&](int n) { return static_cast<int64_t>(clampi(cu[n], 0, T)) * G / R + n; });
}

// Sequence of token t < cu[N]: the last n with cu[n] <= t.
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int N, int t) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace kda
