// The paged key/value cache: writing new tokens (kda_kv_write), with the
// rounding to e4m3 where the cache holds codes, and reading them back
// (kda_kv_read). Both move each byte once; they are bound by memory.
//
// A (token, kv head) row of d elements is handled by d / 8 lanes (8 elements
// each), keys and values in the same launch.
//
// e4m3: with a = max |x| of the row's finite elements = f 2^p (1/2 <= f < 1),
// the least e with a <= 448 2^e = (7/8) 2^(9 + e) is p - 9 if f <= 7/8, else
// p - 8. x 2^-e is exact in fp32, so the rounding to the code is the only one.
#include <type_traits>

#include "kda_attn_device.h"

namespace kda {
namespace {

// Where new token t of the call lies: its page's first row (of Hk * page rows) and offset,
// or false if it has no place.
struct Place { int64_t page; int off; };
__device__ __forceinline__ bool place_of(const KvArgs &a, int t, Place &p) {
    const int n = seq_of_token(a.cu, a.N, t);
    const int start = clampi(a.cu[n], 0, a.T), end = clampi(a.cu[n + 1], start, a.T);
    if (t < start || t >= end) return false;
    const int64_t pos = static_cast<int64_t>(a.lens[n]) - (end - t);
    if (pos < 0 || (pos >> a.page_shift) >= a.max_pages) return false;
    const int id = a.table[static_cast<int64_t>(n) * a.max_pages + (pos >> a.page_shift)];
    if (id < 0 || id >= a.num_pages) return false;
    p.page = id;
    p.off = static_cast<int>(pos & ((1 << a.page_shift) - 1));
    return true;
}
// whether t belongs to a sequence at all
__device__ __forceinline__ bool in_batch(const KvArgs &a, int t) {
    const int n = seq_of_token(a.cu, a.N, t);
    const int start = clampi(a.cu[n], 0, a.T), end = clampi(a.cu[n + 1], start, a.T);
    return t >= start && t < end;
}

template <typename T> struct alignas(16) Eight { T x[8]; };

template <int D, typename T, kda_kv_dtype_t KV>
__device__ __forceinline__ void write_row(const T *src, void *cache, uint8_t *exps, int64_t row, int c) {
    const Eight<T> in = *reinterpret_cast<const Eight<T> *>(src + 8 * c);
    if constexpr (KV != KDA_KV_E4M3) {
        *reinterpret_cast<Eight<T> *>(static_cast<T *>(cache) + row * D + 8 * c) = in;
    } else {
        float x[8], top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = io<T>::load(&in.x[i]);
            const float ax = fabsf(x[i]);
            if (!(ax < INFINITY)) x[i] = NAN;
            else top = fmaxf(top, ax);
        }
#pragma unroll
        for (int d = 1; d < D / 8; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        int e = -127;
        if (top > 0.f) {
            int p;
            const float f = frexpf(top, &p);
            e = max(f <= 0.875f ? p - 9 : p - 8, -127);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_ldexpf(x[i], -e);
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
        *reinterpret_cast<int2 *>(static_cast<uint8_t *>(cache) + row * D + 8 * c) = make_int2(lo, hi);
        if (c == 0) exps[row] = static_cast<uint8_t>(e + 127);
    }
}

template <int D, typename T, kda_kv_dtype_t KV>
__device__ __forceinline__ void read_row(T *dst, const void *cache, const uint8_t *exps, int64_t row, bool there, int c) {
    if (!there) {
        Eight<T> z{};
        *reinterpret_cast<Eight<T> *>(dst + 8 * c) = z;
        return;
    }
    float x[8];
    if constexpr (KV == KDA_KV_E4M3) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(cache) + row * D + 8 * c);
        const bf16x8 v = codes_to_bf16(w.x, w.y, 1.f);
        const int e = static_cast<int>(exps[row]) - 127;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __builtin_ldexpf(static_cast<float>(v[i]), e);
    } else {
        using C = typename std::conditional<KV == KDA_KV_F32, float, bf16_t>::type;
        const Eight<C> v = *reinterpret_cast<const Eight<C> *>(static_cast<const C *>(cache) + row * D + 8 * c);
        if constexpr (std::is_same<C, T>::value) {
            *reinterpret_cast<Eight<T> *>(dst + 8 * c) = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = io<C>::load(&v.x[i]);
    }
    if constexpr (std::is_same<T, float>::value) {
        Eight<T> out;
#pragma unroll
        for (int i = 0; i < 8; ++i) out.x[i] = x[i];
        *reinterpret_cast<Eight<T> *>(dst + 8 * c) = out;
    } else {
        *reinterpret_cast<bf16x8 *>(dst + 8 * c) = to_frag(x, bf16x8{});
    }
}

constexpr int kThreads = 256;
__host__ __device__ inline unsigned key_blocks(int64_t rows, int d) {
    return static_cast<unsigned>((rows * (d / 8) + kThreads - 1) / kThreads);
}

template <int K, int V, typename T, kda_kv_dtype_t KV, bool WRITE>
__global__ __launch_bounds__(kThreads) void kv_kernel(KvArgs a) {
    constexpr int LK = K / 8, LV = V / 8;  // lanes of a (token, head) row
    // the first key_blocks workgroups take the keys, the others the values
    const int64_t rows = static_cast<int64_t>(a.T) * a.Hk;
    const unsigned kb = key_blocks(rows, K);
    const bool isv = blockIdx.x >= kb;
    const int64_t at = static_cast<int64_t>(isv ? blockIdx.x - kb : blockIdx.x) * kThreads + threadIdx.x;
    const int64_t row = isv ? at / LV : at / LK;
    const int c = static_cast<int>(isv ? at % LV : at % LK);
    if (row >= rows) return;
    const int t = static_cast<int>(row / a.Hk), h = static_cast<int>(row - static_cast<int64_t>(t) * a.Hk);
    Place p{0, 0};
    const bool there = place_of(a, t, p);
    const int64_t crow = ((p.page * a.Hk + h) << a.page_shift) + p.off;
    if constexpr (WRITE) {
        if (!there) return;
        if (!isv) write_row<K, T, KV>(static_cast<const T *>(a.k) + t * a.ks + h * K, a.kc, a.kexp, crow, c);
        else write_row<V, T, KV>(static_cast<const T *>(a.v) + t * a.vs + h * V, a.vc, a.vexp, crow, c);
    } else {
        if (!there && !in_batch(a, t)) return;
        if (!isv) read_row<K, T, KV>(static_cast<T *>(a.k) + t * a.ks + h * K, a.kc, a.kexp, crow, there, c);
        else read_row<V, T, KV>(static_cast<T *>(a.v) + t * a.vs + h * V, a.vc, a.vexp, crow, there, c);
    }
}

template <int K, int V, bool WRITE> hipError_t launch_dims(const KvArgs &a, hipStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.T) * a.Hk;
    const dim3 grid(key_blocks(rows, K) + key_blocks(rows, V)), block(kThreads);
    if (a.kv_dtype == KDA_KV_F32)
        hipLaunchKernelGGL((kv_kernel<K, V, float, KDA_KV_F32, WRITE>), grid, block, 0, st, a);
    else if (a.kv_dtype == KDA_KV_BF16 && a.dtype == KDA_BF16)
        hipLaunchKernelGGL((kv_kernel<K, V, bf16_t, KDA_KV_BF16, WRITE>), grid, block, 0, st, a);
    else if (a.kv_dtype == KDA_KV_E4M3 && a.dtype == KDA_BF16)
        hipLaunchKernelGGL((kv_kernel<K, V, bf16_t, KDA_KV_E4M3, WRITE>), grid, block, 0, st, a);
    else if constexpr (!WRITE) {
        if (a.kv_dtype == KDA_KV_BF16)
            hipLaunchKernelGGL((kv_kernel<K, V, float, KDA_KV_BF16, WRITE>), grid, block, 0, st, a);
        else
            hipLaunchKernelGGL((kv_kernel<K, V, float, KDA_KV_E4M3, WRITE>), grid, block, 0, st, a);
    }
    return hipGetLastError();
}

template <bool WRITE> hipError_t launch_kv(const KvArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128, WRITE>(a, st) : launch_dims<128, 64, WRITE>(a, st);
    return a.V == 128 ? launch_dims<64, 128, WRITE>(a, st) : launch_dims<64, 64, WRITE>(a, st);
}

}  // namespace

hipError_t launch_kv_write(const KvArgs &a, hipStream_t st) { return launch_kv<true>(a, st); }
hipError_t launch_kv_read(const KvArgs &a, hipStream_t st) { return launch_kv<false>(a, st); }

}  // namespace kda
