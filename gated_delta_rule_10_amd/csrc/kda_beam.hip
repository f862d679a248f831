// Beam search over recurrent states: the choice of the next beams
// (kda_beam_select) and the states' reordering after it (kda_state_reorder).
//
// Selection. The K best candidates of a request are among the K best logits of
// each of its beams, so one pass over the logits is enough: every wave keeps, for
// its piece of a row, the running maximum and sum of the softmax and a list of
// the K best (logit, token), one entry to a lane, sorted. A piece's threshold
// starts at the K-th largest of the lanes' own maxima over the first batch (K
// tokens at least as good are there) and rises with the list, so that few tokens
// get as far as an insertion. A second launch, one workgroup to a request, joins
// the pieces: rows' sums in fp64, then the K best of the lists' candidates.
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
template <typename F> __device__ __forceinline__ Key<F> no_key() { return {static_cast<F>(-INFINITY), 0xFFFFFFFFu}; }
template <typename F> __device__ __forceinline__ Key<F> from_lane(const Key<F> &k, int lane) {
    return {__shfl(k.v, lane), static_cast<uint32_t>(__shfl(static_cast<int>(k.i), lane))};
}
// Lane l and its partner l ^ m: the better one to the lower lane where `down`.
template <typename F> __device__ __forceinline__ void exchange(Key<F> &k, int m, bool better) {
    const Key<F> o = {__shfl_xor(k.v, m), static_cast<uint32_t>(__shfl_xor(static_cast<int>(k.i), m))};
    if (o.before(k) == better) k = o;
}
// 64 keys, one a lane, into falling order
template <typename F> __device__ __forceinline__ void sort64(Key<F> &k, int lane) {
#pragma unroll
    for (int n = 2; n <= 64; n <<= 1)
#pragma unroll
        for (int m = n / 2; m > 0; m >>= 1) exchange(k, m, ((lane & m) == 0) == ((lane & n) == 0 || n == 64));
}
// The better half of two sorted lists, sorted: of a and the reversed b the better one in each lane
// is in neither order, but bitonic.
template <typename F> __device__ __forceinline__ void merge64(Key<F> &a, const Key<F> &b, int lane) {
    const Key<F> r = from_lane(b, 63 - lane);
    if (r.before(a)) a = r;
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) exchange(a, m, (lane & m) == 0);
}

// A sorted list of the wave's K best so far, entry l in lane l.
template <typename F> struct Best {
    Key<F> list, last;  // last: the K-th (wave-uniform)
    int K, lane;
    __device__ __forceinline__ void start(int K_, int lane_) {
        list = last = no_key<F>();
        K = K_;
        lane = lane_;
    }
    __device__ __forceinline__ void take_last() { last = from_lane(list, K - 1); }
    // all lanes' keys for which `in` holds, one after the other
    __device__ __forceinline__ void insert(const Key<F> &k, bool in) {
        uint64_t m = __ballot(in && k.before(last));
        while (m) {
            const Key<F> x = from_lane(k, __ffsll(static_cast<unsigned long long>(m)) - 1);
            m &= m - 1;
            if (!x.before(last)) continue;
            const int at = __popcll(__ballot(list.before(x)));
            const Key<F> up = {__shfl_up(list.v, 1), static_cast<uint32_t>(__shfl_up(static_cast<int>(list.i), 1))};
            if (lane > at) list = up;
            if (lane == at) list = x;
            take_last();
        }
    }
};

// Parts of a row's workspace: pieces are written by the first launch, one per workgroup.
struct Pieces {
    double *sum;
    float *top, *value;
    int32_t *token;
};
__host__ __device__ inline Pieces pieces_of(void *ws, int64_t rows, int S, int K) {
    Pieces p;
    p.sum = static_cast<double *>(ws);
    p.top = reinterpret_cast<float *>(p.sum + rows * S);
    p.value = p.top + rows * S;
    p.token = reinterpret_cast<int32_t *>(p.value + rows * S * K);
    return p;
}

template <typename T> struct Batch;
template <> struct Batch<float> {
    static constexpr int kPer = 4, kLoads = 4;  // elements of 16 bytes, loads of a lane
    static __device__ __forceinline__ void load(const float *p, float *x) { __builtin_memcpy(x, p, 16); }
};
template <> struct Batch<bf16_t> {
    static constexpr int kPer = 8, kLoads = 2;
    static __device__ __forceinline__ void load(const bf16_t *p, float *x) {
        uint32_t u[4];
        __builtin_memcpy(u, p, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
};

// A lane's running maximum and sum of e^(x - maximum); the sum is NaN from a NaN or +infinity on.
struct RowSum {
    float m;
    double s;
    template <int E> __device__ __forceinline__ float add(const float (&x)[E]) {
        float top = x[0];
#pragma unroll
        for (int i = 1; i < E; ++i) top = fmaxf(top, x[i]);
        const float now = fmaxf(m, top), ref = now == -INFINITY ? 0.f : now;
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) part += __builtin_amdgcn_exp2f((x[i] - ref) * kLog2e);
        s = s * static_cast<double>(__builtin_amdgcn_exp2f((m - ref) * kLog2e)) + static_cast<double>(part);
        m = now;
        return top;
    }
    __device__ __forceinline__ void join(float om, double os) {
        const float now = fmaxf(m, om), ref = now == -INFINITY ? 0.f : now;
        s = s * static_cast<double>(__builtin_amdgcn_exp2f((m - ref) * kLog2e)) +
            os * static_cast<double>(__builtin_amdgcn_exp2f((om - ref) * kLog2e));
        m = now;
    }
    __device__ __forceinline__ void join_wave() {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) {
            const float om = __shfl_xor(m, d);
            const double os = __shfl_xor(s, d);
            join(om, os);
        }
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void select_pieces_kernel(SelectArgs a, int S) {
    constexpr int PER = Batch<T>::kPer, LOADS = Batch<T>::kLoads, E = PER * LOADS;
    __shared__ float lv[kWaves][64], lm[kWaves];
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

    RowSum sum = {-INFINITY, 0.0};
    Best<float> best;
    best.start(a.K, lane);
    if (piece == 0 && tail < a.V) {
        const bool in = tail + lane < a.V;
        const float x[1] = {in ? io<T>::load(x0 + tail + lane) : -INFINITY};
        sum.add(x);
        best.insert({x[0], static_cast<uint32_t>(tail + lane)}, x[0] > -INFINITY);
    }
    float least = -INFINITY;  // K of the piece's elements are at least this
    for (int b = b0; b < b1; b += 64 * LOADS) {
        float x[E];
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int at = b + 64 * u + lane;
            if (at < b1) {
                Batch<T>::load(x0 + static_cast<int64_t>(at) * PER, x + PER * u);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j) x[PER * u + j] = -INFINITY;
            }
        }
        const float top = sum.add(x);
        if (b == b0) {
            Key<float> k = {top, static_cast<uint32_t>(lane)};
            sort64(k, lane);
            least = __shfl(k.v, a.K - 1);
        }
        const float bar = fmaxf(least, best.last.v);
        if (!__any(top >= bar && top > -INFINITY)) continue;
#pragma unroll
        for (int u = 0; u < LOADS; ++u)
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float v = x[PER * u + j];
                best.insert({v, static_cast<uint32_t>((b + 64 * u + lane) * PER + j)}, v >= bar && v > -INFINITY);
            }
    }
    sum.join_wave();
    lv[w][lane] = best.list.v;
    li[w][lane] = best.list.i;
    if (lane == 0) {
        lm[w] = sum.m;
        ls[w] = sum.s;
    }
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
        merge64(best.list, {lv[i][lane], li[i][lane]}, lane);
        sum.join(lm[i], ls[i]);
    }
    const Pieces p = pieces_of(a.ws, static_cast<int64_t>(a.N) * a.W, S, a.K);
    const int64_t at = static_cast<int64_t>(row) * S + split;
    if (lane < a.K) {
        p.value[at * a.K + lane] = best.list.v;
        p.token[at * a.K + lane] = static_cast<int32_t>(best.list.i);
    }
    if (lane == 0) {
        p.top[at] = sum.m;
        p.sum[at] = sum.s;
    }
}

__global__ __launch_bounds__(kThreads) void select_join_kernel(SelectArgs a, int S) {
    __shared__ double lse[64], score[64], lv[kWaves][64];
    __shared__ uint32_t li[kWaves][64];
    __shared__ uint8_t ended[64];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), n = blockIdx.x;
    const Pieces p = pieces_of(a.ws, static_cast<int64_t>(a.N) * a.W, S, a.K);
    const int64_t row0 = static_cast<int64_t>(n) * a.W;
    for (int r = w; r < a.W; r += kWaves) {
        RowSum sum = {-INFINITY, 0.0};
        const bool over = a.done && a.done[row0 + r];
        if (lane < S && !over) sum = {p.top[(row0 + r) * S + lane], p.sum[(row0 + r) * S + lane]};
        sum.join_wave();
        if (lane == 0) {
            lse[r] = static_cast<double>(sum.m) + log(sum.s);
            score[r] = static_cast<double>(a.scores[row0 + r]);
            ended[r] = over;
        }
    }
    __syncthreads();
    // the lists' first entries first: the rest seldom pass them
    Best<double> best;
    best.start(a.K, lane);
    const int lists = a.W * S, all = lists * a.K;
    for (int c = w * 64; c < all; c += kThreads) {
        const int i = c + lane, rank = i / lists, list = i - rank * lists, r = list / S;
        Key<double> k = no_key<double>();
        if (i < all) {
            if (!ended[r]) {
                const int64_t at = (row0 * S + list) * a.K + rank;
                const float v = p.value[at];
                if (v > -INFINITY) k = {static_cast<double>(v) - lse[r] + score[r], static_cast<uint32_t>(r) * a.V + p.token[at]};
            } else if (rank == 0 && list == r * S) {
                k = {score[r], static_cast<uint32_t>(r) * a.V + a.done_token};
            }
        }
        const bool in = k.v > -INFINITY;
        if (c == w * 64) {
            if (!in) k = no_key<double>();  // NaN
            sort64(k, lane);
            best.list = k;
            best.take_last();
        } else {
            best.insert(k, in);
        }
    }
    lv[w][lane] = best.list.v;
    li[w][lane] = best.list.i;
    __syncthreads();
    if (w != 0) return;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) merge64(best.list, {lv[i][lane], li[i][lane]}, lane);
    if (lane < a.K) {
        const bool some = best.list.v > -INFINITY;
        const int64_t at = static_cast<int64_t>(n) * a.K + lane;
        const uint32_t r = best.list.i / static_cast<uint32_t>(a.V);
        a.out_scores[at] = static_cast<float>(best.list.v);
        a.out_parent[at] = some ? static_cast<int32_t>(r) : -1;
        a.out_token[at] = some ? static_cast<int32_t>(best.list.i - r * a.V) : -1;
    }
}

// Workgroups per row: enough to fill the card, of at least 2048 tokens.
int splits_of(int32_t N, int32_t W, int32_t V) {
    const int64_t rows = static_cast<int64_t>(N) * W;
    const int64_t want = (4 * compute_units() + rows - 1) / rows, most = (static_cast<int64_t>(V) + 2047) / 2048;
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

size_t beam_select_workspace(int32_t N, int32_t W, int32_t V, int32_t K) {
    const size_t pieces = static_cast<size_t>(N) * W * splits_of(N, W, V);
    return pieces * (sizeof(double) + sizeof(float) + K * (sizeof(float) + sizeof(int32_t)));
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
    // pieces of 16 KB, fewer and longer ones where the card is full anyway
    const int64_t pieces = (a.slot_bytes / 16 + kPiece - 1) / kPiece, groups = static_cast<int64_t>(a.N) * a.layers;
    const int64_t x = max(static_cast<int64_t>(1), min(pieces, (16 * compute_units() + groups - 1) / groups));
    hipLaunchKernelGGL(reorder_kernel, dim3(static_cast<unsigned>(x * groups)), dim3(kThreads), 0, st, a, static_cast<int>(x));
    return hipGetLastError();
}

}  // namespace kda
