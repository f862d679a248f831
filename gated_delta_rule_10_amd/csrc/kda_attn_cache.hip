// Attention of new tokens over the paged cache (kda_attn_cache_fwd).
//
// The cache is what the call has to read, so it is read once: a workgroup
// takes all rows of a (sequence, kv head), the new tokens times the query heads
// of the group, in tiles of R rows, over a run of steps: 128 cached tokens, 64 of fp32, and 64
// where the waves share them (below).
//
// Two kernels, by the rows that a (sequence, kv head) has on average:
//  - up to 16 (single tokens, with the group's heads): the steps of a run are shared out
//    among the four waves, each of which streams its own tokens without a barrier
//    (kda_attn_stream.h). fp32 caches take this one for any number of rows.
//  - more (several or drafted tokens): the waves share each tile of 64 tokens in LDS and
//    take 32 rows each, up to 128 (kda_attn_rows.h).
//
// Split. Sequences differ in length and only the device knows it, so the steps
// of all (sequence, kv head, row tile)s are laid on one line and each of W
// workgroups takes an equal piece of it. A (sequence, kv head, row tile) that
// one workgroup covers is finished there; otherwise each piece leaves its
// maximum, sum and unnormalised output in the workspace, and a second kernel
// joins them in the order of the line, so results do not depend on timing.
//
// What bounds it: the cache's bytes. One token for each of 64 sequences of 1000 to 16000
// tokens, H = 32, Hk = 8, d = 128: a bf16 cache of 1.37 GB in 247 us (5.55 TB/s; a copy
// reaches 4.9), an e4m3 one of 0.69 GB in 140 us (4.93 TB/s), an fp32 one of 2.75 GB in 480 us
// (5.7 TB/s, though its kernel at d = 128 spills 6 registers). One sequence of 524288 tokens: 2.15
// GB in 366 us (5.86 TB/s), 9 us of them the join. 24 drafted tokens for each of 16 sequences of
// 500 to 20000 tokens: 125 us from bf16 (4.05 TB/s), 105 from e4m3 (2.45 TB/s, 450 TFLOP/s).
// Chunks of a prompt (2048 tokens over 30000): 1.05 ms from bf16 (990 TFLOP/s), 1.30 from e4m3.
// Every row tile of a sequence has as many steps on the line, also those that its causal rows do
// not see; with no tokens before a chunk that is half of them (2048 over 0: 81 and 105 us, 420
// and 330 TFLOP/s).
#include "kda_attn_stream.h"

namespace kda {
namespace {

// Sequence n's place on the line. One unit of the line is a step of a (sequence, kv head,
// row tile), or all of its steps where the line is not cut inside them (AttnArgs::whole).
struct Seq {
    int start, count;  // its new tokens
    int ctx, end;      // tokens before them (may be below 0), cached tokens within the page table
    int tiles, steps;  // row tiles; steps per row tile
    int per;           // units per row tile
    __device__ __forceinline__ int64_t units(int Hk) const { return static_cast<int64_t>(Hk) * tiles * per; }
};

// from the sequence's rows and cached length
template <int R, int STEP> __device__ __forceinline__ Seq seq_from(const AttnArgs &a, int start, int count, int len) {
    Seq s;
    s.start = start;
    s.count = count;
    len = max(len, 0);
    s.ctx = len - s.count;
    s.end = min(len, a.max_pages << a.page_shift);
    s.tiles = static_cast<int>((static_cast<int64_t>(s.count) * a.G + R - 1) / R);
    s.steps = max((s.end + STEP - 1) / STEP, 1);  // at least one, which writes the rows
    s.per = a.whole ? 1 : s.steps;
    return s;
}
template <int R, int STEP> __device__ __forceinline__ Seq seq_of(const AttnArgs &a, int n) {
    int start, count;
    seq_rows(a.cu, n, a.T, start, count);
    return seq_from<R, STEP>(a, start, count, ld_meta(a.lens, n));
}

// A workgroup takes at least kMinSteps steps where the line is short, so that a
// short cache is not cut into pieces that cost more to join than to read. With 1, 2 and
// 4: 11.6, 12.7 and 15.3 us for one token at 1000 tokens, 17.1, 16.7 and 17.7 for eight
// such sequences, 20.4, 17.1 and 17.8 for 16 tokens at 2000.
constexpr int kMinSteps = 2;
__device__ __forceinline__ int64_t line_workgroups(const AttnArgs &a, int64_t U) {
    const int64_t W = a.W, w = a.whole ? U : (U + kMinSteps - 1) / kMinSteps;
    return w < W ? max(w, static_cast<int64_t>(1)) : W;
}
__device__ __forceinline__ int64_t line_begin(int64_t w, int64_t U, int64_t W) { return w * U / W; }
__device__ __forceinline__ int64_t line_owner(int64_t u, int64_t U, int64_t W) { return ((u + 1) * W - 1) / U; }

__device__ __forceinline__ int64_t wave_scan(int64_t x, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int lo = __shfl_up(static_cast<int>(x & 0xFFFFFFFFll), d), hi = __shfl_up(static_cast<int>(x >> 32), d);
        if (lane >= d) x += (static_cast<int64_t>(hi) << 32) | static_cast<uint32_t>(lo);
    }
    return x;
}

// Workspace: prefix of the line [N + 1] int64, then 2 W partial tiles. A
// workgroup has at most two pieces that are not whole, its first and its last.
__host__ __device__ inline size_t part_floats(int R, int V) { return static_cast<size_t>(R) * (V + 2); }
__host__ __device__ inline size_t prefix_bytes(int N) { return (static_cast<size_t>(N) + 1) * 8 + 255 & ~static_cast<size_t>(255); }

// The line, as a wave sees it: 64 sequences at a time, one to a lane. Up to 64 sequences stay
// in the lanes, so that the sequences of a workgroup cost no further loads.
template <int R, int STEP> struct Line {
    int64_t total;
    int start, count, len;  // of sequence base + lane
    int64_t before, mine;   // units before it, its own
    int base;

    __device__ __forceinline__ void load(const AttnArgs &a, int n0, int64_t units_before, int lane) {
        base = n0;
        const int n = n0 + lane;
        start = count = len = 0;
        mine = 0;
        if (n < a.N) {
            start = clampi(a.cu[n], 0, a.T);
            count = clampi(a.cu[n + 1], start, a.T) - start;
            len = a.lens[n];
            mine = seq_from<R, STEP>(a, start, count, len).units(a.Hk);
        }
        before = wave_scan(mine, lane) - mine + units_before;
    }
    __device__ __forceinline__ int64_t end() const {  // units up to the last lane's
        const int64_t x = before + mine;
        return static_cast<int64_t>(__builtin_amdgcn_readlane(static_cast<int>(x >> 32), 63)) << 32 |
               static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x & 0xFFFFFFFFll), 63));
    }
    // prefix: the units before each sequence, and in all; written if not nullptr
    __device__ __forceinline__ void scan(const AttnArgs &a, int lane, int64_t *prefix) {
        int64_t units = 0;
        for (int n0 = 0; n0 < a.N; n0 += 64) {
            load(a, n0, units, lane);
            if (prefix && n0 + lane < a.N) prefix[n0 + lane] = before;
            units = end();
        }
        total = units;
        if (prefix && lane == 0) prefix[a.N] = units;
    }
    // the sequence that holds unit u < total: `n`, and the units before it
    __device__ __forceinline__ Seq find(const AttnArgs &a, int64_t u, int lane, int &n, int64_t &units_before) {
        if (a.N > 64) {
            int64_t units = 0;
            for (int n0 = 0;; n0 += 64) {
                load(a, n0, units, lane);
                units = end();
                if (u < units) break;
            }
        }
        return take(a, __builtin_ctzll(__ballot(before <= u && u < before + mine)), n, units_before);
    }
    // the next sequence after n that has units: there is one
    __device__ __forceinline__ Seq next(const AttnArgs &a, int lane, int &n, int64_t &units_before) {
        for (;;) {
            const int at = n - base + 1;
            const uint64_t some = __ballot(mine > 0) & (at < 64 ? ~0ull << at : 0);
            if (some) return take(a, __builtin_ctzll(some), n, units_before);
            load(a, base + 64, end(), lane);
            n = base - 1;
        }
    }
    __device__ __forceinline__ Seq take(const AttnArgs &a, int at, int &n, int64_t &units_before) const {
        n = base + at;
        units_before = static_cast<int64_t>(__builtin_amdgcn_readlane(static_cast<int>(before >> 32), at)) << 32 |
                       static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(before & 0xFFFFFFFFll), at));
        return seq_from<R, STEP>(a, __builtin_amdgcn_readlane(start, at), __builtin_amdgcn_readlane(count, at),
                                 __builtin_amdgcn_readlane(len, at));
    }
};

// A run of a sequence's page table in registers: lane i of `now` holds page first + i, and
// `next` the 64 after those. A scalar load would share its counter with the LDS reads and
// hold the first of them up at every step.
struct Pages {
    const int32_t *table;
    int first, max_pages, num_pages;
    int now, next;
    uint64_t there;  // bit i: page first + i exists

    __device__ __forceinline__ int load(int p, int lane) const {
        const int i = p + lane;
        return i < max_pages ? table[i] : -1;
    }
    __device__ __forceinline__ void check() {
        const bool ok = now >= 0 && now < num_pages;
        there = __ballot(ok);
        now = ok ? now : 0;  // a page that is not there is read as page 0, and masked
    }
    // runs start at a multiple of a step's pages, so a step never lies in two of them
    __device__ __forceinline__ void begin(const AttnArgs &a, int n, int pos, int lane) {
        table = a.table + static_cast<int64_t>(n) * a.max_pages;
        max_pages = a.max_pages;
        num_pages = a.num_pages;
        first = pos >> a.page_shift;
        now = load(first, lane);
        next = load(first + 64, lane);
        check();
    }
    // position pos of the next step (not below the last one)
    __device__ __forceinline__ void reach(const AttnArgs &a, int pos, int lane) {
        if ((pos >> a.page_shift) - first < 64) return;
        first += 64;
        now = next;
        next = load(first + 64, lane);
        check();
    }
    // cache row (of [pages, Hk, page]) of position pos
    __device__ __forceinline__ int64_t row(const AttnArgs &a, int kvh, int pos) const {
        const int id = __builtin_amdgcn_readlane(now, ((pos >> a.page_shift) - first) & 63);
        return ((static_cast<int64_t>(id) * a.Hk + kvh) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
    __device__ __forceinline__ bool exists(const AttnArgs &a, int pos) const {
        return (there >> (((pos >> a.page_shift) - first) & 63)) & 1u;
    }
};

// workgroups to a compute unit, as registers and LDS allow
constexpr int kPerCu = 2;

template <int K, int V, typename TC>
__global__ __launch_bounds__(64 * kWaves, kPerCu) void attn_cache_kernel(AttnArgs a) {
    using S = Stream<K, V, TC>;
    constexpr int R = S::R;
    __shared__ __align__(16) char lds[S::kLds];
    __shared__ float stat[2][kWaves][R];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    char *lk = lds + w * (S::KB + S::VB), *lv = lk + S::KB;

    Line<R, S::kStep> line;
    line.scan(a, lane, blockIdx.x == 0 && w == 0 && !a.whole ? static_cast<int64_t *>(a.ws) : nullptr);
    const int64_t U = line.total;
    if (U == 0) return;
    const int64_t W = line_workgroups(a, U);
    if (static_cast<int64_t>(blockIdx.x) >= W) return;
    int64_t u = line_begin(blockIdx.x, U, W);
    const int64_t u_end = line_begin(blockIdx.x + 1, U, W);
    if (u >= u_end) return;
    int n;
    int64_t before;
    Seq q = line.find(a, u, lane, n, before);
    bool first = true;

    S st;
    while (u < u_end) {
        if (u >= before + q.units(a.Hk)) q = line.next(a, lane, n, before);
        const int64_t in = u - before;
        const int item = static_cast<int>(in / q.per), t0 = static_cast<int>(in - static_cast<int64_t>(item) * q.per);
        const int t1 = a.whole ? q.steps : static_cast<int>(min(static_cast<int64_t>(q.steps), t0 + (u_end - u)));
        const int kvh = item / q.tiles, r0 = (item - kvh * q.tiles) * R;
        const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(q.count) * a.G - r0));
        const bool whole = t0 == 0 && t1 == q.steps;
        const int tok0 = r0 / a.G, tok1 = (r0 + rows - 1) / a.G;
        // tokens below `open` are seen by all rows, none from `last` on is seen by any
        const int open = min(q.end, a.mask ? q.ctx : q.ctx + tok0 + 1);
        const int last = min(q.end, a.mask ? q.end : q.ctx + tok1 + 1);

        st.reset();
        st.load_q(a, q.start, kvh, r0, rows, lane);
        Pages pages;
        pages.begin(a, n, t0 * S::kStep, lane);
        // this wave's steps: those with a token that some row sees
        const int te = min(t1, (last - w * S::kStepWave + S::kStep - 1) / S::kStep);
        auto load = [&](int t, typename S::Ahead &n) {
            pages.reach(a, t * S::kStep, lane);
            int64_t row[S::NB];
#pragma unroll
            for (int b = 0; b < S::NB; ++b) {
                const int pos = t * S::kStep + w * S::kStepWave + 16 * b;
                row[b] = pages.row(a, kvh, pos);
                n.here[b] = pages.exists(a, pos);
            }
            S::load_cache(n, a, row, lane);
        };
        // Loads past the last step read that step again, so that every step has as many behind it.
        auto step = [&](int t, typename S::Ahead &n) {
            const int p0 = t * S::kStep + w * S::kStepWave;
            const bool masked = p0 + S::kStepWave > open || !n.here[0] || !n.here[S::NB - 1];
            uint32_t kx[S::NB], vx[S::NB];  // this step's: the next one's are about to be loaded
#pragma unroll
            for (int b = 0; b < S::NB; ++b) {
                kx[b] = n.ke[b];
                vx[b] = n.ve[b];
            }
            uint32_t sees = 0;
            if (masked) sees = st.visible(a, q.start, r0, rows, p0, q.ctx, q.end, n.here, lane);
            const bool odd = S::stage(n, lk, lv, masked, p0, q.end, lane);
            load(min(t + 1, te - 1), n);
            __builtin_amdgcn_wave_barrier();
            st.step(lk, lv, a.c, masked, sees, odd, kx, vx, lane);
            __builtin_amdgcn_wave_barrier();
        };
        if (t0 < te) {
            load(t0, st.next);
            for (int t = t0; t < te; ++t) step(t, st.next);
        }
        __syncthreads();  // the join takes the waves' LDS
        if (whole) {
            st.join(lds, stat, w, lane, rows, [&](int row, int ch, float m, f32x4 x, float l) {
                store_out(a, q.start, kvh, r0 + row, ch, m, x, l);
            });
        } else {
            float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + prefix_bytes(a.N)) +
                          (2 * static_cast<size_t>(blockIdx.x) + (first ? 0 : 1)) * part_floats(R, V);
            st.join(lds, stat, w, lane, rows, [&](int row, int ch, float m, f32x4 x, float l) {
                *reinterpret_cast<f32x4 *>(part + row * V + ch) = x;
                if (ch == 0) {
                    part[R * V + row] = m;
                    part[R * V + R + row] = l;
                }
            });
        }
        first = false;
        u += a.whole ? 1 : t1 - t0;
    }
}

// Where the page tables reach no further than this, a (sequence, kv head, row tile) is one unit
// of the line, and there is nothing to join: one step more or less costs about a microsecond,
// joining about five (its launch and its reads). Whole against cut at 500 tokens: 11.4 and 12.6
// us for one token, 30 and 34 for one token of 64 sequences, 19.2 and 14.3 for 16 tokens of one
// sequence, 20.5 and 27.6 for 12 tokens of 16. At 1000 tokens: 16.6 and 12.7, 54 and 58, 31.8
// and 14.5. The lengths are the device's, so a short sequence in a table that reaches further is
// cut: whole calls of one token at 300 tokens take 12.8 us with tables of up to 512 tokens and
// 18.5 beyond, those of 64 such sequences 19.8 and 23.7.
constexpr int kWhole = 512;

// Joins the pieces of the (sequence, kv head, row tile)s that the line was cut inside: a
// workgroup takes up to 16 rows of one. Groups of V / 4 lanes take a row each; where there are
// more groups than rows, several share a row's pieces and are added in the end.
constexpr int kJoinThreads = 512, kJoinRows = 16;
template <int V, int R, int STEP>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a) {
    constexpr int LPR = V / 4, GR = kJoinThreads / LPR;  // lanes of a row, groups
    __shared__ __align__(16) f32x4 red[GR][LPR];
    __shared__ float red_l[GR];
    const int tid = threadIdx.x, gr = tid / LPR, c = tid % LPR;
    constexpr int PARTS = R / kJoinRows;
    const int part_of = blockIdx.x % PARTS, rest = blockIdx.x / PARTS, kvh = rest % a.Hk;
    const int64_t slot = rest / a.Hk;
    const int n = seq_of_slot(a.cu, a.N, a.T, a.G, R, slot, tid & 63);
    const int64_t *prefix = static_cast<const int64_t *>(a.ws);
    const int64_t U = prefix[a.N], before = prefix[n];  // on their way with what seq_of reads
    const Seq q = seq_of<R, STEP>(a, n);
    const int64_t tile = slot - static_cast<int64_t>(q.start) * a.G / R - n;
    if (tile < 0 || tile >= q.tiles) return;
    const int64_t r0 = tile * R + part_of * kJoinRows;
    const int rows = static_cast<int>(min(static_cast<int64_t>(kJoinRows), static_cast<int64_t>(q.count) * a.G - r0));
    if (rows <= 0) return;
    const int64_t W = line_workgroups(a, U);
    const int64_t s = before + (static_cast<int64_t>(kvh) * q.tiles + tile) * q.steps, e = s + q.steps;
    const int64_t w0 = line_owner(s, U, W), w1 = line_owner(e - 1, U, W);
    if (w0 == w1) return;
    // piece i of the tile: of workgroup w0 + i, whose first piece it is unless w0 had other work before
    const float *parts = reinterpret_cast<const float *>(static_cast<const char *>(a.ws) + prefix_bytes(a.N));
    const int pieces = static_cast<int>(w1 - w0) + 1;
    const bool other = line_begin(w0, U, W) < s;
    const float *p0 = parts + (2 * w0 + (other ? 1 : 0)) * part_floats(R, V), *p1 = parts + 2 * w0 * part_floats(R, V);
    auto piece = [&](int i) { return i == 0 ? p0 : p1 + 2 * i * part_floats(R, V); };

    int share = 1;  // groups to a row
    while (share * 2 * rows <= GR) share *= 2;
    const int per = GR / share;  // rows at a time
    for (int rb = 0; rb < rows; rb += per) {
        const int rr = rb + gr / share, sub = gr % share, row = part_of * kJoinRows + min(rr, rows - 1);
        float m = -INFINITY;
        for (int i = c; i < pieces; i += LPR) m = fmaxf(m, piece(i)[R * V + row]);
#pragma unroll
        for (int d = 1; d < LPR; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        float l = 0.f;
#pragma unroll 8
        for (int i = sub; i < pieces; i += share) {
            const float *p = piece(i);
            const float mi = p[R * V + row], f = mi == -INFINITY ? 0.f : exp2f(mi - m);
            x += *reinterpret_cast<const f32x4 *>(p + row * V + 4 * c) * f;
            l += p[R * V + R + row] * f;
        }
        if (share > 1) {
            red[gr][c] = x;
            if (c == 0) red_l[gr] = l;
            __syncthreads();
            for (int i = 1; i < share; ++i) {
                x += red[(gr + i) % GR][c];
                l += red_l[(gr + i) % GR];
            }
            __syncthreads();
        }
        if (sub == 0 && rr < rows) store_out(a, q.start, kvh, static_cast<int>(r0) + rr, 4 * c, m, x, l);
    }
}

// ---- more than 16 rows
//
// Four waves of 32 rows. A ring of two tiles as the cache holds them is copied to LDS ahead;
// e4m3 tiles are turned to bf16 with their scales by all four waves together, once, into a
// tile of their own (exactly: four bits of significand and a power of two), so that the
// products are the bf16 ones. Two workgroups share a compute unit, so that one's softmax and
// waits run under the other's products. 24 tokens of 4 heads to a kv head, 16 sequences of 8000
// tokens: 115 us from a bf16 cache (524 MB, 4.6 TB/s), 107 from e4m3 (270 MB, 2.5 TB/s), where
// the turn to bf16, the products and the softmax are what it waits for.
template <int K, int V, typename TC> struct Tiles {
    using X = Rows<K, V>;
    static constexpr int NW = 4, R = 32 * NW, ES = sizeof(TC);
    static constexpr bool kCodes = ES == 1;
    static constexpr int KR = kTile * K * ES, VR = kTile * V * ES;  // bytes of a tile in the cache's type
    static constexpr int XB = kCodes ? 256 : 0;  // exponents: 64 of keys, 64 of values, and those again
    static constexpr int kRaw = KR + VR + XB, kStages = 2;
    static constexpr int kLds = kStages * kRaw + (kCodes ? X::KB + X::VB : 0);
    static constexpr int NK = KR / (1024 * NW), NV = VR / (1024 * NW);
    static constexpr int kCopies = NK + NV + (kCodes ? 1 : 0);  // memory operations per wave and tile
    static_assert(NK >= 1 && NV >= 1, "a tile is at least one copy per wave");

    // tile at position p0 to LDS at dst
    static __device__ __forceinline__ void copy(const AttnArgs &a, const Pages &pages, uint32_t dst, int kvh, int p0, int w, int lane) {
#pragma unroll
        for (int i = 0; i < NK; ++i) rows<K, true>(a, pages, dst + (i * NW + w) * 1024, a.k, kvh, p0, i, w, lane);
#pragma unroll
        for (int i = 0; i < NV; ++i) rows<V, false>(a, pages, dst + KR + (i * NW + w) * 1024, a.v, kvh, p0, i, w, lane);
        if (kCodes) {
            // words 0-15: keys' exponents, 16-31: values', 32-63: again. Every wave writes the same
            // bytes, so that all have as many operations to await.
            const int pos = p0 + 4 * (lane & 15);
            const int id = __shfl(pages.now, ((pos >> a.page_shift) - pages.first) & 63);
            const int64_t r = ((static_cast<int64_t>(id) * a.Hk + kvh) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
            copy_word_to_lds(dst + KR + VR, (lane & 16 ? a.vexp : a.kexp) + r);
        }
    }
    // 1024 bytes: 64 chunks, all in one group of 16 tokens and so in one page. bf16 chunks go where
    // the products read them, codes as they lie.
    template <int D, bool KEYS>
    static __device__ __forceinline__ void rows(const AttnArgs &a, const Pages &pages, uint32_t dst, const void *cache, int kvh,
                                                int p0, int i, int w, int lane) {
        constexpr int C = D * ES / 16;
        const int t0 = (i * NW + w) * 64 / C, t = t0 + lane / C;
        const int c = (lane % C) ^ (kCodes ? 0 : KEYS ? X::swz_k(t) : X::swz_v(t));
        const char *base = static_cast<const char *>(cache) + pages.row(a, kvh, p0 + t0) * (D * ES);
        copy_to_lds(dst, base, (lane / C) * (D * ES) + 16 * c);
    }

    // codes of a tile to bf16, at the chunks that the products read. tid: of 256 threads.
    static __device__ __forceinline__ void convert(const char *raw, char *to, int tid) {
        part<K, true>(raw, raw + KR + VR, to, tid);
        part<V, false>(raw + KR, raw + KR + VR + kTile, to + X::KB, tid);
    }
    template <int D, bool KEYS> static __device__ __forceinline__ void part(const char *raw, const char *exps, char *to, int tid) {
        constexpr int C = D / 16;  // chunks of 16 codes to a row
#pragma unroll
        for (int i = 0; i < kTile * C / 256; ++i) {
            const int e = i * 256 + tid, t = e / C, c = e % C, sw = KEYS ? X::swz_k(t) : X::swz_v(t);
            const u32x4 w = *reinterpret_cast<const u32x4 *>(raw + 16 * e);
            // the conversion takes a scale's exponent bits
            const float scale = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint8_t *>(exps + t)) << 23);
            // which of the two is written first: the chunks of eight lanes then lie in different banks
            // (107 against 109 us for the trees above)
            const int f = (D == 128 ? (c >> 2) ^ (KEYS ? 0 : t) : t) & 1;
            const bf16x8 x = codes_to_bf16(f ? w[2] : w[0], f ? w[3] : w[1], scale);
            const bf16x8 y = codes_to_bf16(f ? w[0] : w[2], f ? w[1] : w[3], scale);
            *reinterpret_cast<bf16x8 *>(to + t * (2 * D) + 16 * ((2 * c + f) ^ sw)) = x;
            *reinterpret_cast<bf16x8 *>(to + t * (2 * D) + 16 * ((2 * c + 1 - f) ^ sw)) = y;
        }
    }
};

template <int K, int V, typename TC>
__global__ __launch_bounds__(256, 2) void attn_cache_rows_kernel(AttnArgs a) {
    using T = Tiles<K, V, TC>;
    using X = Rows<K, V>;
    constexpr int R = T::R;
    __shared__ __align__(1024) char lds[T::kLds];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);

    Line<R, kTile> line;
    line.scan(a, lane, blockIdx.x == 0 && w == 0 && !a.whole ? static_cast<int64_t *>(a.ws) : nullptr);
    const int64_t U = line.total;
    if (U == 0) return;
    const int64_t W = line_workgroups(a, U);
    if (static_cast<int64_t>(blockIdx.x) >= W) return;
    int64_t u = line_begin(blockIdx.x, U, W);
    const int64_t u_end = line_begin(blockIdx.x + 1, U, W);
    if (u >= u_end) return;
    int n;
    int64_t before;
    Seq q = line.find(a, u, lane, n, before);
    bool first = true;
    const uint32_t base = lds_address(lds);
    const float c = fabsf(a.c);

    X st;
    while (u < u_end) {
        if (u >= before + q.units(a.Hk)) q = line.next(a, lane, n, before);
        const int64_t in = u - before;
        const int item = static_cast<int>(in / q.per), t0 = static_cast<int>(in - static_cast<int64_t>(item) * q.per);
        const int t1 = a.whole ? q.steps : static_cast<int>(min(static_cast<int64_t>(q.steps), t0 + (u_end - u)));
        const int kvh = item / q.tiles, r0 = (item - kvh * q.tiles) * R;
        const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(q.count) * a.G - r0));
        const bool whole = t0 == 0 && t1 == q.steps;
        const int tok0 = r0 / a.G, tok1 = (r0 + rows - 1) / a.G;
        // tokens below `open` are seen by all rows, none from `last` on is seen by any
        const int open = min(q.end, a.mask ? q.ctx : q.ctx + tok0 + 1);
        const int last = min(q.end, a.mask ? q.end : q.ctx + tok1 + 1);
        const int te = min(t1, (max(last, 0) + kTile - 1) / kTile);  // tiles that hold something

        // this lane's row; rows past the last repeat it and are not stored
        const bool some = 32 * w < rows;
        const int r = r0 + min(32 * w + (lane & 31), rows - 1), tok = r / a.G, h = kvh * a.G + (r - tok * a.G);
        const uint64_t bits = a.mask ? a.mask[q.start + tok] : 0;
        st.reset();
        st.load_q(static_cast<const bf16_t *>(a.q) + static_cast<int64_t>(q.start + tok) * a.qs + h * K, a.c < 0.f, lane);

        Pages pages;
        pages.begin(a, n, t0 * kTile, lane);
        uint32_t here = 0;  // which groups of 16 tokens of the tiles on their way exist, the next one's lowest
        auto copy = [&](int t) {
            pages.reach(a, t * kTile, lane);
            T::copy(a, pages, base + (t & 1) * T::kRaw, kvh, t * kTile, w, lane);
            uint32_t v = 0;
#pragma unroll
            for (int g = 0; g < 4; ++g) v |= (pages.exists(a, t * kTile + 16 * g) ? 1u : 0u) << g;
            return v;
        };
        phase_barrier();  // all are done with the ring
        if (t0 < te) here = copy(t0);
        if (T::kCodes && t0 + 1 < te) here |= copy(t0 + 1) << 4;
        // Makes tile t ready for all waves, once all are done with the one before, and says which of
        // its groups exist. Copies of bf16 tiles: t + 1 is issued here. Codes: t + 1 is on its
        // way, and t + 2 follows once t has been turned to bf16.
        auto turn = [&](int t) {
            if (T::kCodes && t + 1 < te) wait_copies<T::kCopies>();
            else wait_copies();
            phase_barrier();
            const uint32_t there = here & 15u;
            here >>= 4;
            if (T::kCodes) {
                T::convert(lds + (t & 1) * T::kRaw, lds + T::kStages * T::kRaw, tid);
                phase_barrier();
                if (t + 2 < te) here |= copy(t + 2) << 4;
            } else if (t + 1 < te) {
                here |= copy(t + 1);
            }
            return there;
        };
        auto tile = [&](int t) { return lds + (T::kCodes ? T::kStages * T::kRaw : (t & 1) * T::kRaw); };
        int t = t0;
        uint32_t there = 0;
        // tiles that all rows see whole, then from the first other one on
        for (; t < te; ++t) {
            there = turn(t);
            if ((t + 1) * kTile > open || there != 15u) break;
            if (!some) continue;
            const char *lk = tile(t), *lv = lk + X::KB;
            st.scores(lk, lane);
            X::template interleave<false>();
            st.template softmax<false>(c, 0);
            st.values(lv, lane);
            X::template interleave<true, false>();
        }
        for (; t < te; ++t, there = t < te ? turn(t) : 0) {
            if (!some) continue;
            const uint32_t sees = X::of_lane(seen_tokens(a.mask != nullptr, bits, t * kTile, q.ctx, q.ctx + tok, q.end, there), lane);
            const char *lk = tile(t), *lv = lk + X::KB;
            st.scores(lk, lane);
            st.template softmax<true>(c, sees);
            st.values_masked(lv, sees, lane);
        }
        if (32 * w + (lane & 31) < rows) {
            const float l = swap32_sum(st.l);
            if (whole) {
                st.each(lane, [&](int ch, f32x4 x) { store_out(a, q.start, kvh, r, ch, st.m, x, l); });
            } else {
                float *part = reinterpret_cast<float *>(static_cast<char *>(a.ws) + prefix_bytes(a.N)) +
                              (2 * static_cast<size_t>(blockIdx.x) + (first ? 0 : 1)) * part_floats(R, V);
                const int row = r - r0;
                st.each(lane, [&](int ch, f32x4 x) { *reinterpret_cast<f32x4 *>(part + row * V + ch) = x; });
                if (lane < 32) {
                    part[R * V + row] = st.m;
                    part[R * V + R + row] = l;
                }
            }
        }
        first = false;
        u += a.whole ? 1 : t1 - t0;
    }
}

// Rows of a tile: 16 where the mean rows of a (sequence, kv head) fit them, else 128. Tiles of 16
// against 128 rows, 16 sequences of 8000 tokens, us: 16 rows 107 and 110 from bf16, 62 and 94
// from e4m3; 20 and 32 rows 164 and 110, 92 and 94; 48 rows 274 and 113, 137 and 101; 96 rows
// 481 and 120, 245 and 115. (From e4m3, 32 rows are even closer: 64 sequences of 6000 tokens 294
// and 240, one of 100000 64 and 78.)
// The counts are the device's, and the mean stands for them. One chunk among single tokens (chunk
// @ tokens before it + others, each @ its own), 16 against 128 rows, bf16 and e4m3: mean of 8 rows,
// 500 @ 2000 + 500 @ 2000 815 and 892, 438 and 830; 100 @ 1000 + 200 @ 1000 176 and 228, 106 and
// 217; 64 @ 4000 + 64 @ 4000 204 and 226, 116 and 208. Of 24, 500 @ 2000 + 100 @ 2000 286 and 209,
// but 154 and 206. Of 44, 2000 @ 20000 + 200 @ 2000 6623 and 1061, 3497 and 1231; of 68, 512 @
// 8000 + 32 @ 4000 717 and 189, 377 and 202; of 132, 2048 @ 0 + 64 @ 4000 420 and 281, 322 and 301.
// fp32 has the 16-row form alone: 24 tokens of 4 heads, 16 sequences of 500 to 20000 tokens take
// 919 us against a floor of 310 (its products).
int tile_rows(int64_t T, int64_t N, int64_t G, bool f32) { return f32 || (T + N - 1) / N * G <= 16 ? 16 : 128; }

template <int V, int R, int STEP> hipError_t launch_join(const AttnArgs &a, hipStream_t st) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole) return e;
    const int64_t slots = static_cast<int64_t>(a.T) * a.G / R + a.N;
    hipLaunchKernelGGL((attn_join_kernel<V, R, STEP>), dim3(static_cast<unsigned>(slots * a.Hk * (R / kJoinRows))),
                       dim3(kJoinThreads), 0, st, a);
    return hipGetLastError();
}
template <int K, int V, typename TC> hipError_t launch_stream(const AttnArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((attn_cache_kernel<K, V, TC>), dim3(a.W), dim3(64 * kWaves), 0, st, a);
    return launch_join<V, 16, Stream<K, V, TC>::kStep>(a, st);
}
template <int K, int V, typename TC> hipError_t launch_rows(const AttnArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((attn_cache_rows_kernel<K, V, TC>), dim3(a.W), dim3(256), 0, st, a);
    return launch_join<V, Tiles<K, V, TC>::R, kTile>(a, st);
}

template <int K, int V> hipError_t launch_dims(const AttnArgs &a, hipStream_t st) {
    const bool one = tile_rows(a.T, a.N, a.G, a.in_dtype == KDA_F32) == 16;
    if (a.kv_dtype == KDA_KV_F32) return launch_stream<K, V, float>(a, st);
    if (a.kv_dtype == KDA_KV_BF16) return one ? launch_stream<K, V, bf16_t>(a, st) : launch_rows<K, V, bf16_t>(a, st);
    return one ? launch_stream<K, V, e4m3_t>(a, st) : launch_rows<K, V, e4m3_t>(a, st);
}

}  // namespace

int32_t attn_cache_workgroups() { return kPerCu * compute_units(); }

size_t attn_cache_workspace(int32_t N, int32_t T, int32_t H, int32_t Hk, int32_t V, int32_t max_tokens, kda_dtype_t in_dtype) {
    if (max_tokens <= kWhole) return 0;
    const int R = tile_rows(T, N, H / Hk, in_dtype == KDA_F32);
    return prefix_bytes(N) + 2 * static_cast<size_t>(attn_cache_workgroups()) * part_floats(R, V) * sizeof(float);
}

hipError_t launch_attn_cache(const AttnArgs &args, hipStream_t st) {
    AttnArgs a = args;
    a.W = attn_cache_workgroups();
    a.whole = (a.max_pages << a.page_shift) <= kWhole;
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

}  // namespace kda
