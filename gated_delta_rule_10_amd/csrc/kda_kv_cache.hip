// The paged key/value cache: writing new tokens (kda_kv_write), with the
// rounding to e4m3 where the cache holds codes, and reading them back
// (kda_kv_read). Both move each byte once; they are bound by memory.
// 32768 tokens, Hk = 8, d = 128, bf16 to e4m3 (202 MB each way): written in 54 us (3.7
// TB/s), read back in 33 us (6.2 TB/s, part of it from the last-level cache). To bf16 (268 MB)
// 42 and 42 us (6.4 TB/s), fp32 (537 MB) 91 and 133 us (5.9 and 4.0 TB/s).
//
// A workgroup takes 64 (token, kv head) rows of keys and of values, d / 8 lanes
// (8 elements each) to a row. One lane per row finds its place in the cache
// (sequence, page, offset) for all of them, while the first loads are on their way.
//
// e4m3: with a = max |x| of the row's finite elements = 1.m 2^E, the least e with
// a <= 448 2^e = 1.75 2^(8 + e) is E - 8 if 1.m <= 1.75, else E - 7, and both can
// be read from a's bits. x 2^-e is exact in fp32, so the rounding to the code is
// the only one.
#include <type_traits>

#include "kda_attn_device.h"

namespace kda {
namespace {

// Where new token t of the call lies: the row of its kv head h in [pages, Hk, page], kNowhere if
// it has no place, kOutside if it is in no sequence. Every lane of a wave calls it, with tokens
// that do not fall from lane to lane, `t0` the first one's. The sequences from t0's on are read
// by one load, a lane each; only a token behind 64 of them is searched for in memory.
constexpr int64_t kNowhere = -1, kOutside = -2;
__device__ __forceinline__ int64_t place_of(const KvArgs &a, int t0, int t, int h, int lane) {
    const int n0 = wave_last_upto(a.N, t0, lane, [&](int n) { return static_cast<int64_t>(a.cu[n]); });
    const int m = min(n0 + lane, a.N - 1);
    const int wstart = a.cu[m], wend = a.cu[m + 1], wlen = a.lens[m];
    int n = 0;  // of the window: the last whose start is not above t
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl(wstart, n + d) <= t && n0 + n + d < a.N ? d : 0;
    int start = __shfl(wstart, n), end = __shfl(wend, n), len = __shfl(wlen, n);
    n += n0;
    if (n - n0 == 63 && t >= end) {
        n = seq_of_token(a.cu, a.N, t);
        start = a.cu[n];
        end = a.cu[n + 1];
        len = a.lens[n];
    }
    start = clampi(start, 0, a.T);
    end = clampi(end, start, a.T);
    if (t < start || t >= end) return kOutside;
    const int64_t pos = static_cast<int64_t>(len) - (end - t);
    if (pos < 0 || (pos >> a.page_shift) >= a.max_pages) return kNowhere;
    const int id = a.table[static_cast<int64_t>(n) * a.max_pages + (pos >> a.page_shift)];
    if (id < 0 || id >= a.num_pages) return kNowhere;
    return ((static_cast<int64_t>(id) * a.Hk + h) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

template <typename T> struct alignas(16) Eight { T x[8]; };

// Tokens are read (written) past the caches: each byte is touched once by a call, and the cache's
// own pages, which the next call reads, stay there instead (32768 tokens written and read back:
// 92 against 103 us).
typedef unsigned once4 __attribute__((ext_vector_type(4)));
template <typename E> __device__ __forceinline__ E load_once(const E *p) {
    once4 r[sizeof(E) / 16];
#pragma unroll
    for (unsigned i = 0; i < sizeof(E) / 16; ++i) r[i] = __builtin_nontemporal_load(reinterpret_cast<const once4 *>(p) + i);
    E e;
    __builtin_memcpy(&e, r, sizeof(E));
    return e;
}
template <typename E> __device__ __forceinline__ void store_once(void *p, const E &e) {
    once4 r[sizeof(E) / 16];
    __builtin_memcpy(r, &e, sizeof(E));
#pragma unroll
    for (unsigned i = 0; i < sizeof(E) / 16; ++i) __builtin_nontemporal_store(r[i], reinterpret_cast<once4 *>(p) + i);
}

template <int D, typename T, kda_kv_dtype_t KV>
__device__ __forceinline__ void write_row(const Eight<T> &in, void *cache, uint8_t *exps, int64_t row, int c) {
    if constexpr (KV != KDA_KV_E4M3) {
        *reinterpret_cast<Eight<T> *>(static_cast<T *>(cache) + row * D + 8 * c) = in;
    } else {
        float x[8];
        uint32_t top = 0;  // bits of the largest magnitude: they order as the numbers do
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = io<T>::load(&in.x[i]);
            const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
            const bool fine = u < 0x7F800000u;
            top = max(top, fine ? u : 0);
            if (!fine) x[i] = NAN;
        }
#pragma unroll
        for (int d = 1; d < D / 8; d <<= 1) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
        const int byte = max(static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 0);  // e + 127, 0 to 247
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);                         // 2^-e
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
        *reinterpret_cast<int2 *>(static_cast<uint8_t *>(cache) + row * D + 8 * c) = make_int2(lo, hi);
        if (c == 0) exps[row] = static_cast<uint8_t>(byte);
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
            store_once(dst + 8 * c, v);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = io<C>::load(&v.x[i]);
    }
    if constexpr (std::is_same<T, float>::value) {
        Eight<T> out;
#pragma unroll
        for (int i = 0; i < 8; ++i) out.x[i] = x[i];
        store_once(dst + 8 * c, out);
    } else {
        store_once(dst + 8 * c, to_frag(x, bf16x8{}));
    }
}

constexpr int kThreads = 256, kRows = 64;

template <int K, int V, typename T, kda_kv_dtype_t KV, bool WRITE>
__global__ __launch_bounds__(kThreads) void kv_kernel(KvArgs a) {
    constexpr int LK = K / 8, LV = V / 8;  // lanes of a row
    constexpr int IK = kRows * LK / kThreads, IV = kRows * LV / kThreads;
    __shared__ int64_t place[kRows];
    const int tid = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows, left = static_cast<int64_t>(a.T) * a.Hk - r0;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kRows), left));
    const int t0 = static_cast<int>(r0 / a.Hk), h0 = static_cast<int>(r0 - static_cast<int64_t>(t0) * a.Hk);
    // row r of the workgroup: token t0 + x / Hk, head x % Hk, x = h0 + r
    auto at = [&](int r, int64_t stride, int d) {
        const int x = h0 + r, t = x / a.Hk;
        return static_cast<int64_t>(t0 + t) * stride + (x - t * a.Hk) * d;
    };
    Eight<T> k[IK], v[IV];
    if (WRITE) {
#pragma unroll
        for (int i = 0; i < IK; ++i) {
            const int r = i * (kThreads / LK) + tid / LK;
            if (r < rows) k[i] = load_once(reinterpret_cast<const Eight<T> *>(static_cast<const T *>(a.k) + at(r, a.ks, K) + 8 * (tid % LK)));
        }
#pragma unroll
        for (int i = 0; i < IV; ++i) {
            const int r = i * (kThreads / LV) + tid / LV;
            if (r < rows) v[i] = load_once(reinterpret_cast<const Eight<T> *>(static_cast<const T *>(a.v) + at(r, a.vs, V) + 8 * (tid % LV)));
        }
    }
    if (tid < kRows) {  // the first wave
        const int x = h0 + min(tid, rows - 1), t = x / a.Hk;
        place[tid] = place_of(a, t0, t0 + t, x - t * a.Hk, tid);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IK; ++i) {
        const int r = i * (kThreads / LK) + tid / LK, c = tid % LK;
        if (r >= rows) continue;
        const int64_t p = place[r];
        if (WRITE) {
            if (p >= 0) write_row<K, T, KV>(k[i], a.kc, a.kexp, p, c);
        } else if (p != kOutside) {
            read_row<K, T, KV>(static_cast<T *>(a.k) + at(r, a.ks, K), a.kc, a.kexp, p, p >= 0, c);
        }
    }
#pragma unroll
    for (int i = 0; i < IV; ++i) {
        const int r = i * (kThreads / LV) + tid / LV, c = tid % LV;
        if (r >= rows) continue;
        const int64_t p = place[r];
        if (WRITE) {
            if (p >= 0) write_row<V, T, KV>(v[i], a.vc, a.vexp, p, c);
        } else if (p != kOutside) {
            read_row<V, T, KV>(static_cast<T *>(a.v) + at(r, a.vs, V), a.vc, a.vexp, p, p >= 0, c);
        }
    }
}

template <int K, int V, bool WRITE> hipError_t launch_dims(const KvArgs &a, hipStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.T) * a.Hk;
    const dim3 grid(static_cast<unsigned>((rows + kRows - 1) / kRows)), block(kThreads);
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
