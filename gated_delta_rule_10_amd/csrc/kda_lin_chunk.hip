// Linear attention with one decay per head over packed prompts (kda_lin_chunk_fwd).
//
// A workgroup walks a segment of a sequence for one value head, chunk by chunk,
// with the state in registers (kda_lin_bf16.h, kda_lin_f32.h). A sequence is one segment where
// there are enough sequences and heads to fill the card; otherwise it is cut, and
// two more launches come before: one walks all segments but each sequence's last
// from a state of zeros (the first from the initial state) to their ends, without
// outputs, and one joins these, a segment's state being the one before it times
// e^(its sum of g), plus its own. They read k and v a second time, and are worth
// it where a few sequences would leave the card empty.
//
// What bounds it (H = 32, 128 channels, bf16): 131072 tokens are 4.37 GB, 930 us at the
// rate of a large copy (4.7 TB/s), and take 1550 to 1600 by the card's state: 1090 to
// 1210 for the outputs (4.5 GB, 3.7 to 4.1 TB/s, matrix cores 36 % and vector instructions
// 46 % busy: a chunk's steps hardly overlap), 440 to 460 for the ends, which are bound
// by the walk of the heads that forget slowly (128 chunks at 3.4 us, two workgroups to
// a compute unit; the others stop early, so that 1.3 GB are read). The same in pieces of
// 8192 to 65536 tokens, whose k and v the Infinity Cache could hold for the second
// walk, is slower (6 to 47 %): the launches drain the card between them. Few prompts
// are bound by the walk: one workgroup alone takes 3.5 us a chunk of 64 tokens.
#include "kda_attn_internal.h"
#include "kda_lin_bf16.h"
#include "kda_lin_device.h"
#include "kda_lin_f32.h"

namespace kda {
namespace {

constexpr double kLog2e = 1.4426950408889634;

// A segmented call's workspace, as the registers of a workgroup hold states: those at the starts of
// segments from a sequence's second on, the initial states of sequences that are cut (the final ones may
// take their place in memory), and the sums of log2 e^g over segments. Segment g of a sequence from token
// t on has piece t / R + g, the same for no other but one's first and another's last; only sequences of
// more than R tokens are cut, so that two of them do not begin in one piece.
struct Segments {
    float *state, *first;
    double *sum;
};

// What a workgroup works on: segment `seg` of `segs` of sequence n, `tokens` of them from t0 on. Segments
// are found by their piece, if they are not their sequence's last (then no other such segment has it, and no
// later sequence begins in it or before), or by their place, which is piece + n.
struct Span {
    int n, seg, segs, t0, tokens;
    __device__ __forceinline__ void set(const LinArgs &a, int R, int piece) {
        int start, count;
        seq_rows(a.cu, n, a.T, start, count);
        seg = piece - start / R;
        segs = (count - 1) / R + 1;  // one of no tokens, too
        t0 = start + seg * R;
        tokens = min(R, count - seg * R);
    }
    __device__ __forceinline__ void at_place(const LinArgs &a, int R, int place, int lane) {
        n = seq_of_slot(a.cu, a.N, a.T, 1, R, place, lane);
        set(a, R, place - n);
    }
    __device__ __forceinline__ void at_piece(const LinArgs &a, int R, int piece, int lane) {
        n = wave_last_upto(a.N, piece, lane, [&](int i) { return static_cast<int64_t>(clampi(a.cu[i], 0, a.T)) / R; });
        set(a, R, piece);
    }
};

// The place whose turn it is, in the order of the grid, where there are more workgroups than the card
// holds: up to 64 places go by their tokens, most first, so that a long one is not left over at the end (16
// prompts of 259 to 3509 tokens, the longest last, H = 32: 216 us, and 277 as they come, before later steps). A place to
// a lane. More than 64 go as they come, and have less to lose (80 prompts of 50 to 1912 tokens, H = 32: 499 us the
// longest first, 511 mixed, 523 the longest last).
__device__ __forceinline__ int place_of(const LinArgs &a, int R, int turn, int places, int lane) {
    int start, count, first = 0, of = 0, rank = 0;
    seq_rows(a.cu, min(lane, a.N - 1), a.T, start, count);
    start = start / R + lane;
    for (int n = 0; n < a.N; ++n) {
        const int f = __builtin_amdgcn_readlane(start, n), c = __builtin_amdgcn_readlane(count, n);
        if (f <= lane) first = f, of = c;
    }
    const int64_t left = of - static_cast<int64_t>(lane - first) * R;
    const int tokens = static_cast<int>(min(max(left, static_cast<int64_t>(0)), static_cast<int64_t>(R)));
    for (int i = 0; i < places; ++i) {
        const int other = __builtin_amdgcn_readlane(tokens, i);
        rank += other > tokens || (other == tokens && i < lane);
    }
    return __ffsll(static_cast<unsigned long long>(__ballot(lane < places && rank == turn))) - 1;
}

// x of the lane that a DPP control names, 0 where there is none (or its row is masked)
template <int CTRL, int ROWS> __device__ __forceinline__ double from_dpp(double x) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xF, true);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Inclusive sums over a chunk of log2 e^g, one token to a lane, and their total: shifts within rows of
// 16 lanes, then each row's last lane to the rows behind it.
__device__ __forceinline__ double sums(float g, double &all) {
    double x = static_cast<double>(g) * kLog2e;
    x += from_dpp<0x111, 0xF>(x);
    x += from_dpp<0x112, 0xF>(x);
    x += from_dpp<0x114, 0xF>(x);
    x += from_dpp<0x118, 0xF>(x);
    x += from_dpp<0x142, 0xA>(x);  // lane 15 to row 1, lane 47 to row 3
    x += from_dpp<0x143, 0xC>(x);  // lane 31 to rows 2 and 3
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 63), hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 63);
    all = __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
    return x;
}

// The states at the ends of all segments but each sequence's last, from zeros (the first: from the
// initial state). Chunk by chunk from the end: a token's value is weighed with all the decay between
// it and the segment's end, the state itself is not decayed step by step, and the walk ends where all
// further weights are 0 in fp32. (Heads that forget fast look at a few chunks only.)
template <typename W, int K, int V>
__global__ __launch_bounds__(W::NT, W::kWavesPerSimd) void lin_ends_kernel(LinArgs a, Segments ws, int R) {
    using T = typename W::T;
    constexpr int C = W::C;
    constexpr double kNothing = -160.0;  // 2^-150 is 0 in fp32
    __shared__ __align__(16) char lds[2][W::kTiles];
    __shared__ __align__(16) float left[2][C];
    __shared__ int over[2];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t piece = blockIdx.x;
    const int g0 = blockIdx.x / a.H, h = blockIdx.x - g0 * a.H, hk = h / (a.H / a.Hk);
    Span x;
    x.at_piece(a, R, g0, lane);
    if (x.seg < 0 || x.seg >= x.segs - 1) return;
    const int chunks = R / C;  // all whole
    const T *kp = static_cast<const T *>(a.k) + (x.t0 + R - C) * a.ks + hk * K, *vp = static_cast<const T *>(a.v) + (x.t0 + R - C) * a.vs + h * V;
    W s;
    s.clear();
    double sum = 0.0;  // from the chunk's end to the segment's
    auto decay = [&](int i) { return lane < C ? a.g[(x.t0 + R - (i + 1) * C + lane) * a.gs + h] : 0.f; };
    auto tabulate = [&](float g, int b) {
        double all;
        const double y = sums(log_decay(g), all);  // (g was on its way until here)
        if (lane < C) left[b][lane] = __builtin_amdgcn_exp2f(static_cast<float>(sum + (all - y)));
        if (lane == 0) over[b] = sum < kNothing;
        sum += all;
    };
    auto load = [&] {
        s.load(nullptr, kp, vp, a, C, tid);
        kp -= C * a.ks, vp -= C * a.vs;
    };
    float g = 0.f;
    if (w == W::NW - 1) {
        tabulate(decay(0), 0);
        g = chunks > 1 ? decay(1) : 0.f;
    }
    load();
    s.to_lds(lds[0], tid);
    if (chunks > 1) load();
#pragma unroll 1
    for (int i = 0; i < chunks; ++i) {
        const int b = i & 1;
        __syncthreads();
        if (over[b]) break;
        if (w == W::NW - 1 && i + 1 < chunks) {
            tabulate(g, b ^ 1);
            if (i + 2 < chunks) g = decay(i + 2);
        }
        s.template update<false>(lds[b], {nullptr, nullptr, nullptr, left[b]}, w, lane);
        if (i + 1 < chunks) s.to_lds(lds[b ^ 1], tid);
        if (i + 2 < chunks) load();
    }
    if (x.seg == 0) {
        // the last wave has the sum
        __shared__ float whole;
        if (tid == W::NT - 1) whole = __builtin_amdgcn_exp2f(static_cast<float>(sum));
        __syncthreads();
        const float e = whole;
        const int slot = slot_of(a, x.n);
        const float *s0 = a.s0 + (static_cast<int64_t>(slot) * a.H + h) * (K * V);
        W first;
        first.clear();
        if (a.s0 && slot >= 0) first.take(s0, w, lane);
        first.put(ws.first + piece * (K * V), w, lane);
        s.add(first, e);
    } else if (tid == W::NT - 1) {
        ws.sum[piece] = sum;
    }
    s.put(ws.state + (piece + a.H) * (K * V), w, lane);  // the next segment's
}

// All outputs, and the states at the sequences' ends.
template <typename W, typename TOut, int K, int V>
__global__ __launch_bounds__(W::NT, W::kWavesPerSimd) void lin_segments_kernel(LinArgs a, Segments ws, int R, int sorted) {
    using T = typename W::T;
    constexpr int C = W::C;
    __shared__ __align__(16) char tiles[W::kTiles];
    __shared__ __align__(16) char scores[W::kScores];
    __shared__ __align__(16) char outs[W::kOuts];
    __shared__ __align__(16) float table[2][4][C];
    __shared__ int strange[2];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int turn = blockIdx.x / a.H, h = blockIdx.x - turn * a.H, hk = h / (a.H / a.Hk);
    const int place = sorted ? place_of(a, R, turn, sorted, lane) : turn;
    Span x;
    x.at_place(a, R, place, lane);
    if (x.seg < 0 || x.seg >= x.segs) return;
    const int t0 = x.t0, tokens = x.tokens, chunks = (tokens + C - 1) / C, slot = slot_of(a, x.n);
    const int64_t held = (static_cast<int64_t>(slot) * a.H + h) * (K * V);

    W s;
    s.clear();
    W::prepare(scores, tid);
    if (x.segs > 1)
        s.get((x.seg ? ws.state : ws.first) + (static_cast<int64_t>(place - x.n) * a.H + h) * (K * V), w, lane);
    else if (a.s0 && slot >= 0)
        s.take(a.s0 + held, w, lane);

    const T *qp = static_cast<const T *>(a.q) + t0 * a.qs + hk * K, *kp = static_cast<const T *>(a.k) + t0 * a.ks + hk * K;
    const T *vp = static_cast<const T *>(a.v) + t0 * a.vs + h * V;
    const int64_t os = static_cast<int64_t>(a.H) * V * sizeof(TOut);
    char *op = static_cast<char *>(a.o) + t0 * os + static_cast<int64_t>(h) * V * sizeof(TOut);
    const bool summing = w == W::NW - 1;  // the last wave sums the decays, a chunk ahead
    auto decay = [&](int c) { return lane < min(C, tokens - c * C) ? a.g[(t0 + c * C + lane) * a.gs + h] : 0.f; };
    auto tabulate = [&](float g, int b, int rows) {
        double all;
        const double y = sums(log_decay(g), all);  // (g was on its way until here)
        if (lane < C) {
            const float hi = static_cast<float>(y);
            table[b][0][lane] = hi;
            table[b][1][lane] = static_cast<float>(y - static_cast<double>(hi));
            table[b][2][lane] = __builtin_amdgcn_exp2f(hi);
            table[b][3][lane] = lane < rows ? __builtin_amdgcn_exp2f(static_cast<float>(all - y)) : 0.f;
        }
        if (lane == 0) strange[b] = 0;
    };
    auto load = [&](int c) {
        s.load(qp, kp, vp, a, min(C, tokens - c * C), tid);
        qp += C * a.qs, kp += C * a.ks, vp += C * a.vs;
    };
    auto store = [&](int c) {
        W::store(op, os, outs, min(C, tokens - c * C), tid);
        op += C * os;
    };
    float g = 0.f;
    if (chunks > 0) load(0);
    if (summing && chunks > 0) {
        tabulate(decay(0), 0, tokens);
        if (chunks > 1) g = decay(1);
    }
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        const int b = c & 1;
        const Decays d = {table[b][0], table[b][1], table[b][2], table[b][3]};
        __syncthreads();  // all have read the chunk before
        if (s.to_lds(tiles, tid)) strange[b] = 1;
        __syncthreads();
        if (summing && c + 1 < chunks) {
            tabulate(g, b ^ 1, tokens - (c + 1) * C);
            if (c + 2 < chunks) g = decay(c + 2);
        }
        // Whole rows, a chunk late, past the caches, before the next chunk's loads. (8 x 2000 tokens,
        // 135 us when scores had one part, 157 now: behind the scores 1.5 more, behind the loads 12, through
        // the caches 1.5; the waves' own columns, 32 bytes of a row, 5, and those past the caches 14.)
        if (c > 0) store(c - 1);
        W::scores(scores, tiles, d, a.scale, w, lane);
        if (c + 1 < chunks) load(c + 1);
        s.from_state(tiles, d, a.scale, lane);
        __syncthreads();
        s.from_chunk(scores, tiles, __builtin_amdgcn_readfirstlane(strange[b]) != 0, w, lane);
        s.stage(outs, w, lane);
        s.advance(tiles, d, w, lane);
    }
    __syncthreads();
    if (chunks > 0) store(chunks - 1);
    if (x.seg == x.segs - 1 && a.sT && slot >= 0) s.give(a.sT + held, w, lane);
}

// The states at the starts of each sequence's segments from the third on: that of the one before,
// decayed over it, added to what it wrote itself. Four elements of the state to a thread.
template <int KV> __global__ __launch_bounds__(256) void lin_join_kernel(LinArgs a, Segments ws, int R) {
    constexpr int PER = KV / 4 / 256;
    const int e = (blockIdx.x % PER) * 256 + threadIdx.x, lane = threadIdx.x & 63;
    const int at = blockIdx.x / PER, h = at % a.H;
    // the sequence: of those that have three segments, number at / H
    int start, count, before = at / a.H, n = -1;
    for (int first = 0; first < a.N && n < 0; first += 64) {
        seq_rows(a.cu, min(first + lane, a.N - 1), a.T, start, count);
        uint64_t m = __ballot(first + lane < a.N && count - R > R);
        for (; m && before > 0; --before) m &= m - 1;
        if (m) n = first + __ffsll(static_cast<unsigned long long>(m)) - 1;
    }
    if (n < 0) return;
    seq_rows(a.cu, n, a.T, start, count);
    const int segs = (count - 1) / R + 1;
    const int64_t piece = static_cast<int64_t>(start / R) * a.H + h;
    f32x4 *p = reinterpret_cast<f32x4 *>(ws.state + piece * KV) + e;
    const int64_t step = static_cast<int64_t>(a.H) * (KV / 4);
    f32x4 x = p[step];
    for (int g = 2; g < segs; ++g) {
        const float d = __builtin_amdgcn_exp2f(static_cast<float>(ws.sum[piece + static_cast<int64_t>(g - 1) * a.H]));
        const f32x4 own = p[g * step];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaf(d, x[i], own[i]);
        p[g * step] = x;
    }
}

// Tokens to a segment, and an upper bound of the segments: sequence n's begin at place
// cu[n] / R + n, so a place finds its sequence from cu alone.
struct Plan {
    int R;
    int64_t places;
    bool cut;
};

// Workgroups that the card holds: a compute unit, one of 8 waves (d_v = 128) or two of 4.
int64_t room_of(int32_t V) { return compute_units() * (V == 64 ? 2 : 1); }

// The host knows the number of tokens and sequences, not the lengths.
//
// Where sequences and heads alone fill the card, only a sequence of more than four times the mean length is cut
// (16 of 217 to 3448, H = 32: 214 us, 4 less without the two launches that find nothing to do; cutting those of
// twice the mean was a third slower).
//
// Else segments are as long as lets all of them run at once (1 x 4000, H = 32: 63 chunks uncut 192 us, 8 to a
// segment 60, 4 in two rounds 72, 16 on half of the card 90). From 128 chunks on, two rounds of half as many end
// more evenly (H = 32, halved and not: 1 x 131072 1590 and 1616 us, 1 x 80000 982 and 992, 1 x 66000 820 and
// 821; halved from 64 on, 1 x 60000 753 and 750).
//
// Sequences of the mean length are cut where that is faster (H = 32, cut and uncut: 1 x 400 26.5 and 29.7 us, 1 x
// 300 24 and 23; d = 64, 1 x 500 18.6 and 21.4, 1 x 300 18.6 and 14.6; fp32, 1 x 200 43 and 46). Where it is not,
// only longer ones are, if one that had all the tokens would gain 100 us or more: one of 40000 among 31 of 30, H = 4:
// 130 us, uncut 2212; 16 of 214 to 3509, H = 8: 86 and 197; 8 of 30 and 2000, H = 8, below that line, 41 and 118. A
// batch of equal ones pays 4 us for the launches that find nothing (16 x 512, H = 8: 39.6 and 35.9).
Plan plan_of(int32_t N, int32_t T, int32_t H, int32_t V, kda_dtype_t in_dtype) {
    const int64_t room = room_of(V), rows = static_cast<int64_t>(N) * H;
    const int64_t mean = (static_cast<int64_t>(T) + 64 * static_cast<int64_t>(N) - 1) / (64 * static_cast<int64_t>(N));  // chunks of 64
    int64_t L = max(static_cast<int64_t>(2), ((static_cast<int64_t>(T) / 64 + N) * H + room - 1) / room);
    if (L >= 128) L = (L + 1) / 2;
    // tenths of us: a chunk's walk, and with both walks of a sequence that is cut; launches
    const bool f32 = in_dtype == KDA_F32, narrow = V == 64;
    const int64_t walk = f32 ? (narrow ? 49 : 118) : narrow ? 22 : 35, both = f32 ? (narrow ? 70 : 146) : narrow ? 30 : 55;
    const int64_t launches = 100, gain = 1000;
    if (rows >= room) {
        L = max(L, 4 * mean);
    } else if (launches + both * L >= walk * mean) {
        L = max(L, mean);
        if (launches + both * L + gain > walk * (T / 64)) L = T;
    }
    if (64 * L >= T) return {(T + 63) / 64 * 64 + 64, N, false};
    return {static_cast<int>(64 * L), T / (64 * L) + N, true};
}

size_t pieces_of(const Plan &p, int32_t T, int32_t H) { return static_cast<size_t>(T / p.R + 1) * H; }
size_t sums_bytes(size_t pieces) { return (pieces * sizeof(double) + 255) / 256 * 256; }

template <typename Ends, typename All, typename TOut, int K, int V> hipError_t launch(const LinArgs &a, hipStream_t st) {
    const Plan p = plan_of(a.N, a.T, a.H, V, a.in_dtype);
    Segments ws{};
    const dim3 block(All::NT);
    if (p.cut) {
        const size_t pieces = pieces_of(p, a.T, a.H);
        ws.sum = static_cast<double *>(a.ws);
        ws.state = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sums_bytes(pieces));
        ws.first = ws.state + pieces * (K * V);
        // at most T / R segments are not their sequence's last, and at most T / 2R sequences have three
        const int ends = a.T / p.R, seqs = min(a.N, a.T / p.R / 2);
        hipLaunchKernelGGL((lin_ends_kernel<Ends, K, V>), dim3(ends * a.H), block, 0, st, a, ws, p.R);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        if (seqs > 0) {
            hipLaunchKernelGGL((lin_join_kernel<K * V>), dim3(seqs * a.H * (K * V / 1024)), dim3(256), 0, st, a, ws, p.R);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    const bool sorted = a.N > 1 && p.places <= 64 && p.places * a.H > room_of(V);
    hipLaunchKernelGGL((lin_segments_kernel<All, TOut, K, V>), dim3(static_cast<unsigned>(p.places * a.H)), block, 0, st, a, ws, p.R,
                       sorted ? static_cast<int>(p.places) : 0);
    return hipGetLastError();
}

template <int K, int V> hipError_t launch_dims(const LinArgs &a, hipStream_t st) {
    if (a.in_dtype == KDA_F32) return launch<LinF32<K, V, false>, LinF32<K, V, true>, float, K, V>(a, st);
    if (a.out_dtype == KDA_BF16) return launch<LinBf16<K, V, void>, LinBf16<K, V, bf16_t>, bf16_t, K, V>(a, st);
    return launch<LinBf16<K, V, void>, LinBf16<K, V, float>, float, K, V>(a, st);
}

}  // namespace

hipError_t launch_lin_chunk(const LinArgs &a, hipStream_t st) {
    if (a.K == 128) return a.V == 128 ? launch_dims<128, 128>(a, st) : launch_dims<128, 64>(a, st);
    return a.V == 128 ? launch_dims<64, 128>(a, st) : launch_dims<64, 64>(a, st);
}

size_t lin_chunk_workspace(int32_t N, int32_t T, int32_t H, int32_t K, int32_t V, kda_dtype_t in_dtype) {
    const Plan p = plan_of(N, T, H, V, in_dtype);
    if (!p.cut) return 0;
    const size_t pieces = pieces_of(p, T, H);
    return sums_bytes(pieces) + 2 * pieces * K * V * sizeof(float);
}

}  // namespace kda
