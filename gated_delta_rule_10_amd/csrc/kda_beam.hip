// Beam search over recurrent states: the choice of the next beams
// (kda_beam_select) and the states' reordering after it (kda_state_reorder).
//
// Selection. The K best candidates of a request are among the K best logits of
// each of its beams, so one pass over the logits is enough. A workgroup takes a
// piece of a row: the running maximum and sum of its softmax, and the tokens that
// can be among the K best, which are those not below a bar that K tokens reach.
// Any K lanes' own maxima are such tokens, so the bar is the K-th of them, at best
// over the waves, and few tokens pass it: they go to a list in LDS, in any order.
// A second launch, one workgroup to a request, joins the pieces: rows' sums in
// fp64, a bar over the lists' candidates, and the order of what passes it. Where a
// list overflows (many equal logits, rising ones), the workgroup looks at its
// piece again and keeps the K best in order, one insertion after the other.
//
// 16 x 8 rows of 100003 bf16 logits, K = 16, a third of the beams ended (17 MB are read): 16 us
// for the rows (1 TB/s: a row is short, and a wave's exponentials and comparisons take longer
// than its loads, vector instructions 55 % busy) and 9 for the joins, which are a chain of short
// steps that only N workgroups take; sorted lists in each wave instead of a bar took 42 in all.
// 4 rows of 32000 fp32: 6.5 and 7. Where many tokens reach the bar, lists overflow and rows are gone
// through again: the same rows all equal 69 us in all, all but 50 of a row at the lowest finite
// number 81 (at -infinity 23).
//
// Reordering moves bytes: 16 x 8 beams that all go on from few, 8 layers of 2 MB states,
// 1.6 GB read and written: 290 us, 5.55 TB/s.
#include <cfloat>

#include "kda_attn_internal.h"
#include "kda_beam_internal.h"
#include "kda_device.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;

// Candidates fall by value, equal ones rise by index. An empty place is -infinity.
template <typename F> struct Key {
    F v;
    uint32_t i;
    __device__ __forceinline__ bool before(const Key &o) const { return v > o.v || (v == o.v && i < o.i); }
};
template <typename F> __device__ __forceinline__ Key<F> no_key();
template <> __device__ __forceinline__ Key<float> no_key<float>() { return {-INFINITY, 0xFFFFFFFFu}; }
// (Put together from halves that the compiler does not see: it has set a pair of scalar registers to the
// constant by one instruction whose literal has 32 bits, which made it 0.)
template <> __device__ __forceinline__ Key<double> no_key<double>() {
    uint32_t hi = 0xFFF00000u;
    __asm__("" : "+s"(hi));
    return {__builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32), 0xFFFFFFFFu};
}
// the value of a lane that is the same in all lanes
__device__ __forceinline__ float read_lane(float x, int lane) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane)); }
__device__ __forceinline__ double read_lane(double x, int lane) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), lane), hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
template <typename F> __device__ __forceinline__ Key<F> read_lane(const Key<F> &k, int lane) {
    return {read_lane(k.v, lane), static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(k.i), lane))};
}
// the value of the lane below (lane 0: its own)
__device__ __forceinline__ uint32_t lane_below(uint32_t x) { return __builtin_amdgcn_update_dpp(x, x, 0x138, 0xF, 0xF, false); }
__device__ __forceinline__ float lane_below(float x) { return __uint_as_float(lane_below(__float_as_uint(x))); }
__device__ __forceinline__ double lane_below(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, static_cast<uint64_t>(lane_below(static_cast<uint32_t>(u >> 32))) << 32 | lane_below(static_cast<uint32_t>(u)));
}

// A value that K of the lanes' P numbers each reach (-infinity if they do not): the 16 highest bits of the
// K-th largest, in the order of unsigned numbers.
template <int P> __device__ __forceinline__ float reached_by(const float (&x)[P], int K) {
    uint32_t u[P], p = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const uint32_t bits = __float_as_uint(x[i]);
        u[i] = x[i] > -INFINITY ? (bits & 0x80000000u ? ~bits : bits | 0x80000000u) : 0;
    }
#pragma unroll
    for (int b = 31; b >= 16; --b) {
        const uint32_t q = p | 1u << b;
        int n = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) n += __popcll(__ballot(u[i] >= q));
        if (n >= K) p = q;
    }
    // below every number but -infinity: nothing is known
    return p <= 0x007FFFFFu ? -INFINITY : __uint_as_float(p & 0x80000000u ? p & 0x7FFFFFFFu : ~p);
}

// A sorted list of the wave's K best so far, entry l in lane l.
template <typename F> struct Best {
    Key<F> list, last;  // last: the K-th (the same in all lanes)
    int K, lane;
    __device__ __forceinline__ void start(int K_, int lane_) {
        list = last = no_key<F>();
        K = K_;
        lane = lane_;
    }
    // all lanes' keys for which `in` holds, one after the other
    __device__ __forceinline__ void insert(const Key<F> &k, bool in) {
        uint64_t m = __ballot(in && k.before(last));
        while (m) {
            const Key<F> x = read_lane(k, __ffsll(static_cast<unsigned long long>(m)) - 1);
            m &= m - 1;
            if (!x.before(last)) continue;
            const int at = __popcll(__ballot(list.before(x)));
            const Key<F> up = {lane_below(list.v), lane_below(list.i)};
            if (lane > at) list = up;
            if (lane == at) list = x;
            last = read_lane(list, K - 1);
        }
    }
};

// Parts of a row's workspace, written by the first launch, one per workgroup: 64 tokens, those that are
// none with the value -infinity.
struct Pieces {
    double *sum;
    float *top, *value;
    int32_t *token;
};
__host__ __device__ inline Pieces pieces_of(void *ws, int64_t rows, int S) {
    Pieces p;
    p.sum = static_cast<double *>(ws);
    p.top = reinterpret_cast<float *>(p.sum + rows * S);
    p.value = p.top + rows * S;
    p.token = reinterpret_cast<int32_t *>(p.value + rows * S * 64);
    return p;
}

template <typename T> struct Batch;
template <> struct Batch<float> {
    static constexpr int kPer = 4, kLoads = 4;  // elements of 16 bytes, loads of a lane
    static __device__ __forceinline__ void unpack(const uint4 &w, float *x) { __builtin_memcpy(x, &w, 16); }
    static constexpr uint32_t kNothing = 0xFF800000u;  // -infinity
};
template <> struct Batch<bf16_t> {
    static constexpr int kPer = 8, kLoads = 4;
    static constexpr uint32_t kNothing = 0xFF80FF80u;
    static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
};

// What a sum of e^x is counted in, from its largest x (`top`): e^base 2^R, base 0 but for tops so large that
// their product with log2 e would lose its integers, R the integer nearest to what is left in powers of 2.
constexpr float kLog2eRest = 1.925963033500844e-08f;  // log2 e less its fp32 number
constexpr double kLn2 = 0.6931471805599453;
struct Unit {
    float base, top, R;  // top less base
    explicit __device__ __forceinline__ Unit(float m) {
        const float x = m == -INFINITY ? 0.f : m;
        base = fabsf(x) < 0x1p21f ? 0.f : x;
        top = base == 0.f ? x : 0.f;
        R = rintf(top * kLog2e);
    }
};

// A lane's running maximum and sum of e^x, in units of the maximum; the sum is NaN from a NaN or +infinity on.
//
// e^x = 2^n 2^f, n the integer nearest to x log2 e: f is rounded at 1/2, not at x's distance from the maximum,
// which for equal tokens far below one other would leave the sum off by 6e-7. A term is right to 2^-23 (2^f) and
// 2^-25 (f), a sum of two of them to 2^-24 more, and the rest is fp64, the change to another unit a power of 2:
// a sum is right to 2^-22. n is found by rounding to the ones of a float about 1.5 2^23, in whose low bits
// it stays.
struct RowSum {
    float m;
    double s;
    // the sum's factor where its maximum grows to `now`
    __device__ __forceinline__ void grow(float now) {
        const Unit from(m), to(now);
        const float steps = from.R - to.R;
        if (m == -INFINITY || from.base == to.base)
            s = ldexp(s, m == -INFINITY ? -4000 : static_cast<int>(steps));
        else
            s *= exp((static_cast<double>(from.base) - static_cast<double>(to.base)) + static_cast<double>(steps) * kLn2);
        m = now;
    }
    template <int E> __device__ __forceinline__ float add(const float (&x)[E]) {
        float most = x[0];
#pragma unroll
        for (int i = 1; i < E; ++i) most = fmaxf(most, x[i]);
        grow(fmaxf(m, most));
        const Unit u(m);
        const float ones = 12582912.f - u.R, least = u.top - 80.f;  // e^-80 of 2^31 tokens is nothing in fp64
        double part[2] = {0.0, 0.0};
        float two = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float below = x[i] - u.base, z = below < least ? least : below;  // (NaN stays NaN)
            const float t = __builtin_fmaf(z, kLog2e, ones), n = t - ones;
            const float f = __builtin_fmaf(z, kLog2eRest, __builtin_fmaf(z, kLog2e, -n));
            const float power = __uint_as_float((__float_as_uint(t) << 23) + 0x3F800000u);  // 2^(n - R)
            two = __builtin_fmaf(__builtin_amdgcn_exp2f(f), power, i % 2 ? two : 0.f);
            if (i % 2 || i == E - 1) part[i / 2 % 2] += static_cast<double>(two);
        }
        s += part[0] + part[1];
        return most;
    }
    __device__ __forceinline__ void join(RowSum other) {
        const float now = fmaxf(m, other.m);
        grow(now);
        other.grow(now);
        s += other.s;
    }
    // of groups of `lanes` (a power of two) lanes
    __device__ __forceinline__ void join_lanes(int lanes) {
        float now = m;
        for (int d = lanes / 2; d > 0; d >>= 1) now = fmaxf(now, __shfl_xor(now, d));
        grow(now);
        for (int d = lanes / 2; d > 0; d >>= 1) s += __shfl_xor(s, d);
    }
    // ln of the sum of e^(x - m)
    __device__ __forceinline__ double log_sum() const {
        const Unit u(m);
        return log(s) + (static_cast<double>(u.R) * kLn2 - static_cast<double>(u.top));
    }
};

// Candidates in LDS, in no order.
template <typename F, int SIZE> struct List {
    F value[SIZE];
    uint32_t index[SIZE];
    int count;
    // what passes is added; the count goes on past the list's end
    __device__ __forceinline__ void add(const Key<F> &k, bool in, int lane) {
        const uint64_t m = __ballot(in);
        if (m == 0) return;
        int at = 0;
        if (lane == 0) at = atomicAdd(&count, __popcll(m));
        at = __builtin_amdgcn_readfirstlane(at) + __popcll(m & ((1ull << lane) - 1));
        if (in && at < SIZE) {
            value[at] = k.v;
            index[at] = k.i;
        }
    }
    // all of it (one wave)
    __device__ __forceinline__ void sort(Best<F> &best, int lane) const {
        for (int i = lane; i < count + lane; i += 64) best.insert({value[i < count ? i : 0], index[i < count ? i : 0]}, i < count);
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void select_pieces_kernel(SelectArgs a, int S) {
    constexpr int PER = Batch<T>::kPer, LOADS = Batch<T>::kLoads, E = PER * LOADS;
    __shared__ List<float, 256> list;
    __shared__ float lm[kWaves], lv[kWaves][64];
    __shared__ uint32_t li[kWaves][64];
    __shared__ double ls[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = blockIdx.x / S, split = blockIdx.x - row * S;
    if (a.done && a.done[row]) return;
    // blocks of 16 bytes from the row's start, whatever its alignment (equal rows give equal sums), and
    // the few elements behind them
    const T *x0 = static_cast<const T *>(a.logits) + row * a.stride;
    const int blocks = a.V / PER, tail = blocks * PER;
    const int pieces = S * kWaves, piece = split * kWaves + w;
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * piece / pieces);
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (piece + 1) / pieces);
    uint4 raw[LOADS];
    auto load = [&](int b) {
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int at = b + 64 * u + lane;
            raw[u] = make_uint4(Batch<T>::kNothing, Batch<T>::kNothing, Batch<T>::kNothing, Batch<T>::kNothing);
            if (at < b1) __builtin_memcpy(&raw[u], x0 + static_cast<int64_t>(at) * PER, 16);
        }
    };
    auto token = [&](int b, int u, int j) { return static_cast<uint32_t>((b + 64 * u + lane) * PER + j); };
    load(b0);
    const bool odd = w == 0 && split == 0 && tail + lane < a.V;
    const float last[1] = {odd ? io<T>::load(x0 + tail + lane) : -INFINITY};
    if (tid == 0) list.count = 0;

    RowSum sum = {-INFINITY, 0.0};
    sum.add(last);
    // (the lowest finite number where nothing is known: -infinity never passes)
    float bar = -FLT_MAX;
    for (int b = b0; b < b1 || b == b0; b += 64 * LOADS) {
        float x[E];
#pragma unroll
        for (int u = 0; u < LOADS; ++u) Batch<T>::unpack(raw[u], x + PER * u);
        if (b + 64 * LOADS < b1) load(b + 64 * LOADS);
        const float top = sum.add(x);
        if (b == b0) {  // once, all waves: of all lanes' maxima
            lv[w][lane] = top;
            __syncthreads();
            float tops[kWaves];
#pragma unroll
            for (int i = 0; i < kWaves; ++i) tops[i] = lv[i][lane];
            bar = fmaxf(bar, reached_by(tops, a.K));
            list.add({last[0], static_cast<uint32_t>(tail + lane)}, odd && last[0] >= bar, lane);
        } else if (__popcll(__ballot(top >= bar)) > a.K) {
            const float tops[1] = {top};
            bar = fmaxf(bar, reached_by(tops, a.K));
        }
        if (!__any(top >= bar)) continue;
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float v = x[PER * u + j];
                list.add({v, token(b, u, j)}, v >= bar, lane);
            }
    }
    sum.join_lanes(64);
    if (lane == 0) {
        lm[w] = sum.m;
        ls[w] = sum.s;
    }
    __syncthreads();
    const Pieces p = pieces_of(a.ws, static_cast<int64_t>(a.N) * a.W, S);
    const int64_t at = static_cast<int64_t>(row) * S + split;
    const int count = list.count;
    Best<float> best;
    best.start(a.K, lane);
    if (count > 256) {  // too many pass: the K best in order, after all
        best.insert({last[0], static_cast<uint32_t>(tail + lane)}, odd && last[0] > -INFINITY);
        for (int b = b0; b < b1; b += 64 * LOADS) {
            float x[E];
            load(b);
#pragma unroll
            for (int u = 0; u < LOADS; ++u) Batch<T>::unpack(raw[u], x + PER * u);
            float top[1] = {x[0]};
#pragma unroll
            for (int i = 1; i < E; ++i) top[0] = fmaxf(top[0], x[i]);
            bar = fmaxf(bar, reached_by(top, a.K));
#pragma unroll
            for (int u = 0; u < LOADS; ++u)
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const float v = x[PER * u + j];
                    best.insert({v, token(b, u, j)}, v >= bar);
                }
        }
        lv[w][lane] = best.list.v;
        li[w][lane] = best.list.i;
        __syncthreads();
    }
    if (w != 0) return;
    if (count > 256) {
        for (int i = 1; i < kWaves; ++i) best.insert({lv[i][lane], li[i][lane]}, lane < a.K && lv[i][lane] > -INFINITY);
    } else if (count > 64) {
        list.sort(best, lane);
    } else if (lane < count) {  // few enough to be handed on as they are
        best.list = {list.value[lane], list.index[lane]};
    }
    p.value[at * 64 + lane] = best.list.v;
    p.token[at * 64 + lane] = static_cast<int32_t>(best.list.i);
    if (lane == 0) {
        for (int i = 1; i < kWaves; ++i) sum.join({lm[i], ls[i]});
        p.top[at] = sum.m;
        p.sum[at] = sum.s;
    }
}

// A request's choice, four waves. A wave holds 16 lists of 64 at a time, each turned by 4 lanes more than
// the one before: their candidates are at their starts. What is below the bar for sure is sorted out in
// fp32, by sums that are off by less than the bar is lowered; what passes is computed in fp64. A row's
// maximum and the logarithm of its sum of e^(x - maximum) stay apart: in the sum of a large maximum (all
// tokens at a mask of the type's lowest value) and a logarithm, the logarithm is lost.
constexpr int kLists = 16;

__global__ __launch_bounds__(kThreads) void select_join_kernel(SelectArgs a, int S) {
    __shared__ double log_sum[64], score[64], lv[kWaves][64];
    __shared__ uint32_t li[kWaves][64];
    __shared__ float tops[kWaves][64];
    __shared__ float2 offset[64 * 64];  // of a list: its row's maximum, and score - logarithm
    __shared__ List<double, 256> some;
    __shared__ float top_of[64];
    __shared__ uint8_t ended[64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n = blockIdx.x;
    const Pieces p = pieces_of(a.ws, static_cast<int64_t>(a.N) * a.W, S);
    const int64_t row0 = static_cast<int64_t>(n) * a.W;
    const int lists = a.W * S;
    float v[kLists];
    int32_t token[kLists];
    // (what a row that has ended leaves is whatever was there: its offset is NaN)
    auto load = [&](int first) {
#pragma unroll
        for (int j = 0; j < kLists; ++j) {
            const int list = min(first + j * kWaves, lists - 1);
            const int64_t at = (row0 * S + list) * 64 + ((lane + 4 * j) & 63);
            v[j] = p.value[at];
            token[j] = p.token[at];
        }
    };
    load(w);
    if (tid == 0) some.count = 0;
    const int group = S <= 16 ? 16 : 64;  // lanes to a row's sum
    for (int r0 = 0; r0 < a.W; r0 += kThreads / group) {
        const int r = r0 + tid / group, i = tid % group;
        const bool row = r < a.W, over = row && a.done && a.done[row0 + r];
        RowSum sum = {-INFINITY, 0.0};
        if (row && !over && i < S) sum = {p.top[(row0 + r) * S + i], p.sum[(row0 + r) * S + i]};
        sum.join_lanes(group);
        if (row) {
            const double l = sum.log_sum(), c = static_cast<double>(a.scores[row0 + r]);
            for (int j = i; j < S; j += group) offset[r * S + j] = make_float2(sum.m, over ? NAN : static_cast<float>(c - l));
            if (i == 0) {
                top_of[r] = sum.m;
                log_sum[r] = l;
                score[r] = c;
                ended[r] = over;
            }
        }
    }
    __syncthreads();
    auto candidate = [&](float x, int r) { return (static_cast<double>(x) - static_cast<double>(top_of[r])) - log_sum[r] + score[r]; };
    const Key<double> done = tid < a.W && ended[tid] ? Key<double>{score[tid], static_cast<uint32_t>(tid) * a.V + a.done_token} : no_key<double>();
    // all lanes' own maxima give a bar that K candidates reach
    float top = static_cast<float>(done.v), far = 0.f;
    for (int list = w; list < lists; list += kLists * kWaves) {
        if (list != w) load(list);
#pragma unroll
        for (int j = 0; j < kLists; ++j)
            if (list + j * kWaves < lists) {
                const float2 o = offset[list + j * kWaves];
                const float below = v[j] - o.x, x = below + o.y;
                top = fmaxf(top, x);
                if (x > -INFINITY) far = fmaxf(far, fabsf(below));
            }
    }
    tops[w][lane] = top;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) far = fmaxf(far, __shfl_xor(far, d));
    if (lane == 0) lv[w][0] = static_cast<double>(far);
    __syncthreads();
    float all[kWaves];
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        all[i] = tops[i][lane];
        far = fmaxf(far, static_cast<float>(lv[i][0]));
    }
    // x rounds v - maximum (`below`), the offset and their sum, by 2^-24 of |below|, of |offset| <= |below| + |x|
    // and of |x|, in the K and in the one compared with them
    float bar = reached_by(all, a.K);
    if (bar > -INFINITY) bar -= 1e-6f * (fabsf(bar) + far);
    for (int list = w; list < lists; list += kLists * kWaves) {
        if (lists > kLists * kWaves) load(list);
#pragma unroll
        for (int j = 0; j < kLists; ++j) {
            const int at = list + j * kWaves;
            const float2 o = offset[min(at, lists - 1)];
            const float x = at < lists ? (v[j] - o.x) + o.y : -INFINITY;
            const bool in = x >= bar && x > -INFINITY;
            if (!__any(in)) continue;
            const int r = at / S;
            some.add({candidate(v[j], r), static_cast<uint32_t>(r) * a.V + token[j]}, in, lane);
        }
    }
    some.add(done, done.v > -INFINITY && done.v >= static_cast<double>(bar), lane);
    __syncthreads();
    auto write = [&](int rank, const Key<double> &k) {
        if (rank >= a.K) return;
        const float c = static_cast<float>(k.v);
        const bool found = c > -INFINITY;
        const int64_t at = static_cast<int64_t>(n) * a.K + rank;
        const uint32_t r = k.i / static_cast<uint32_t>(a.V);
        a.out_scores[at] = c;
        a.out_parent[at] = found ? static_cast<int32_t>(r) : -1;
        a.out_token[at] = found ? static_cast<int32_t>(k.i - r * a.V) : -1;
    };
    const int count = some.count;
    if (count <= 256) {  // the places of the few that reach the bar, by counting; behind them, places of none
        const Key<double> k = tid < count ? Key<double>{some.value[tid], some.index[tid]} : no_key<double>();
        int rank = 0;
        if (count <= 64) {
            if (w != 0) return;
            for (int i = 0; i < count; ++i) rank += read_lane(k, i).before(k);
        } else {
#pragma unroll 4
            for (int i = 0; i < count; ++i) rank += Key<double>{some.value[i], some.index[i]}.before(k);
        }
        write(tid < count ? rank : tid, k);
        return;
    }
    // too many reach it: in order, after all
    Best<double> best;
    best.start(a.K, lane);
    best.insert(done, done.v > -INFINITY);
    for (int list = w; list < lists; list += kLists * kWaves) {
#pragma unroll 1
        for (int j = 0; j < kLists; ++j) {
            const int at = list + j * kWaves, is = min(at, lists - 1), r = is / S;
            const int64_t place = (row0 * S + is) * 64 + lane;
            const float x = p.value[place], c = (x - offset[is].x) + offset[is].y;
            best.insert({candidate(x, r), static_cast<uint32_t>(r) * a.V + p.token[place]}, at < lists && c >= bar && c > -INFINITY);
        }
    }
    __syncthreads();  // lv is free
    lv[w][lane] = best.list.v;
    li[w][lane] = best.list.i;
    __syncthreads();
    if (w != 0) return;
    for (int i = 1; i < kWaves; ++i) best.insert({lv[i][lane], li[i][lane]}, lane < a.K && lv[i][lane] > -INFINITY);
    write(lane, best.list);
}

// Workgroups per row: up to 4 to a compute unit in all, of at least 4096 tokens (us: 16 x 8 rows of 100003
// bf16 at 2, 4 and 8 workgroups 29, 21, 24; 1 x 4 rows of 128000 at 2048, 4096 and 8192 tokens 22, 17, 18: the
// joins have fewer lists).
int splits_of(int32_t N, int32_t W, int32_t V) {
    const int64_t rows = static_cast<int64_t>(N) * W;
    const int64_t want = (4 * compute_units() + rows - 1) / rows, most = (static_cast<int64_t>(V) + 4095) / 4096;
    return static_cast<int>(min(static_cast<int64_t>(64), max(static_cast<int64_t>(1), min(want, most))));
}

// States. Every workgroup finds its request's plan by itself (a lane per beam), then copies its
// pieces of all slots that are moved. Slots of parents are only read, those of beams that nobody
// continues only written.
typedef unsigned u4 __attribute__((ext_vector_type(4)));
constexpr int kAhead = 4;                               // 16-byte blocks of a thread on their way
constexpr int kPiece = kThreads * kAhead;               // blocks of a piece

__global__ __launch_bounds__(kThreads) void reorder_kernel(ReorderArgs a, int X) {
    __shared__ int from[64], to[64], moves;
    const int tid = threadIdx.x, group = blockIdx.x / X, x = blockIdx.x - group * X;
    const int n = group / a.layers, layer = group - n * a.layers;
    if (tid < 64) {
        const int W = a.W, j = tid;
        const bool beam = j < W;
        const int64_t at = static_cast<int64_t>(n) * W + j;
        const int slot = beam ? a.slots[at] : -1;
        int par = beam ? a.parent[at] : -1;
        if (par < 0 || par >= W) par = -1;
        bool first = par >= 0, went_on = false;
        for (int i = 0; i < W; ++i) {  // beam i: is its parent mine, or me?
            const int q = __shfl(par, i);
            if (i < j && q == par) first = false;
            if (q == j) went_on = true;
        }
        const bool takes = beam && !first, lost = beam && !went_on;
        const uint64_t takers = __ballot(takes), free_slots = __ballot(lost);
        // the m-th taker gets the m-th free slot
        int get = 0;
        const int m = __popcll(takers & ((1ull << j) - 1));
        uint64_t f = free_slots;
        for (int i = 0; i < 64; ++i) {
            if (!__any(takes && i < m)) break;
            if (i < m) f &= f - 1;
        }
        get = f ? __ffsll(static_cast<unsigned long long>(f)) - 1 : j;
        const int old = __shfl(slot, par >= 0 ? par : 0), taken = __shfl(slot, get);
        const int now = first ? old : taken;
        const bool move = takes && par >= 0 && old >= 0 && old < a.nslots && now >= 0 && now < a.nslots;
        const uint64_t movers = __ballot(move);
        if (move) {
            const int k = __popcll(movers & ((1ull << j) - 1));
            from[k] = old;
            to[k] = now;
        }
        if (j == 0) moves = __popcll(movers);
        if (beam && layer == 0 && x == 0) a.slots_out[at] = now;
    }
    __syncthreads();
    const int64_t blocks = a.slot_bytes / 16;
    char *base = a.states + layer * a.layer_stride;
    for (int k = 0; k < moves; ++k) {
        const u4 *src = reinterpret_cast<const u4 *>(base + from[k] * a.slot_bytes);
        u4 *dst = reinterpret_cast<u4 *>(base + to[k] * a.slot_bytes);
        for (int64_t b = static_cast<int64_t>(x) * kPiece + tid; b < blocks; b += static_cast<int64_t>(X) * kPiece) {
            u4 r[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (b + i * kThreads < blocks) r[i] = __builtin_nontemporal_load(src + b + i * kThreads);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (b + i * kThreads < blocks) __builtin_nontemporal_store(r[i], dst + b + i * kThreads);
        }
    }
}

}  // namespace

size_t beam_select_workspace(int32_t N, int32_t W, int32_t V) {
    const size_t pieces = static_cast<size_t>(N) * W * splits_of(N, W, V);
    return pieces * (sizeof(double) + sizeof(float) + 64 * (sizeof(float) + sizeof(int32_t)));
}

hipError_t launch_beam_select(const SelectArgs &a, hipStream_t st) {
    const int S = splits_of(a.N, a.W, a.V);
    const dim3 grid(static_cast<unsigned>(a.N) * a.W * S), block(kThreads);
    if (a.dtype == KDA_F32)
        hipLaunchKernelGGL(select_pieces_kernel<float>, grid, block, 0, st, a, S);
    else
        hipLaunchKernelGGL(select_pieces_kernel<bf16_t>, grid, block, 0, st, a, S);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(select_join_kernel, dim3(a.N), block, 0, st, a, S);
    return hipGetLastError();
}

hipError_t launch_state_reorder(const ReorderArgs &a, hipStream_t st) {
    // A piece of 16 KB to a workgroup, up to 64 workgroups to a compute unit (16 of them, with several pieces
    // each: 302 us instead of 290 for the case above; 128: 290; pieces of 32 KB: 298).
    const int64_t pieces = (a.slot_bytes / 16 + kPiece - 1) / kPiece, groups = static_cast<int64_t>(a.N) * a.layers;
    const int64_t x = max(static_cast<int64_t>(1), min(pieces, (64 * compute_units() + groups - 1) / groups));
    hipLaunchKernelGGL(reorder_kernel, dim3(static_cast<unsigned>(x * groups)), dim3(kThreads), 0, st, a, static_cast<int>(x));
    return hipGetLastError();
}

}  // namespace kda
