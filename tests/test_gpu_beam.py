"""kda_beam_select and kda_state_reorder: choices have to be equal to the definition's in 64 bits, states to be
moved bit for bit; and whole steps of a beam search over both kinds of recurrent layer."""

import numpy as np
import pytest
import torch

from gated_delta_rule_10_amd import beam, kda, lin
from tests import lin_common as lc

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def definition(logits, scores, K, done=None, done_token=0):
    """Per request: (scores [K], parent [K], token [K]) in 64 bits, and the least gap between candidates of
    different beams next to each other among the first K + 1 (which fp32's e^x could turn round)."""
    x = logits.double().cpu().numpy()
    N, W, V = x.shape
    sc = scores.double().cpu().numpy()
    out = np.full((N, K), -INF), np.full((N, K), -1), np.full((N, K), -1)
    gap = INF
    for n in range(N):
        cand = []
        for w in range(W):
            if done is not None and done[n, w]:
                cand.append((sc[n, w], w, done_token))
                continue
            row = x[n, w]
            if np.isnan(row).any() or (row == INF).any() or not (row > -INF).any():
                continue
            top = row.max()
            c = row - (top + np.log(np.exp(row - top).sum())) + sc[n, w]
            for t in np.lexsort((np.arange(V), -row))[:K + 1]:
                cand.append((c[t], w, int(t)))
        cand = [c for c in cand if c[0] > -INF]
        cand.sort(key=lambda c: (-c[0], c[1], c[2]))
        for a, b in zip(cand[:K], cand[1:K + 1]):
            if a[1] != b[1] and a[0] != b[0]:
                gap = min(gap, a[0] - b[0])
        for i, c in enumerate(cand[:K]):
            out[0][n, i], out[1][n, i], out[2][n, i] = c
    return out, gap


def check(logits, scores, K, done=None, done_token=0, **kw):
    (ref, parent, token), gap = definition(logits, scores, K, done, done_token)
    assert gap > 1e-6, "the inputs leave two beams' candidates too near to each other"
    d = None if done is None else torch.from_numpy(np.asarray(done)).cuda()
    s, p, t = beam.kda_beam_select(logits, scores, K, done=d, done_token=done_token, **kw)
    torch.cuda.synchronize()
    assert np.array_equal(p.cpu().numpy(), parent) and np.array_equal(t.cpu().numpy(), token)
    got = s.double().cpu().numpy()
    fine = ref > -INF
    assert np.array_equal(got > -INF, fine)
    # the row's logarithm to 2^-22 (sums of e^x, each right to 2^-22), and one rounding
    lim = 2.0 ** -22 + 2.0 ** -24 * np.abs(ref[fine])
    worst = float((np.abs(got[fine] - ref[fine]) / lim).max()) if fine.any() else 0.0
    print(f"  worst error / bound = {worst:.3f}", flush=True)
    assert worst <= 1.0
    return s, p, t


def normal(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).cuda()


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N,W,V,K", [(1, 1, 1, 1), (1, 1, 7, 4), (2, 3, 9, 5), (1, 4, 100, 8), (3, 5, 1001, 10), (2, 8, 4099, 16),
                                     (1, 4, 32000, 4), (1, 64, 500, 64), (2, 2, 20011, 64), (5, 1, 65536, 3), (1, 2, 200003, 7)])
def test_select(dt, N, W, V, K):
    x = (3 * normal(N + W + V + K, N, W, V)).to(dt)
    scores = -10 + 3 * normal(V, N, W)
    check(x, scores, K)


@pytest.mark.parametrize("dt", [F32, BF])
def test_equal_candidates_go_by_index(dt):
    """Constant rows, rows of few values, equal beams: the lowest beam and token first."""
    x = torch.zeros((2, 4, 3001), device="cuda")
    scores = torch.zeros((2, 4), device="cuda")
    s, p, t = check(x.to(dt), scores, 12)
    assert (p == 0).all() and torch.equal(t.cpu(), torch.arange(12, dtype=torch.int32).expand(2, 12))
    x = torch.round(normal(1, 2, 1, 3001)).expand(2, 4, 3001).contiguous()
    check(x.to(dt), scores, 64)
    x = torch.round(2 * normal(2, 1, 1, 5000))
    check(x.to(dt), torch.zeros((1, 1), device="cuda"), 50)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_sorted_rows(dt, order):
    x = torch.linspace(-20, 20, 70000, device="cuda").to(dt)
    x = (x if order == "rising" else x.flip(0)).expand(1, 2, -1).contiguous()
    check(x, torch.tensor([[0.0, -0.013]], device="cuda"), 32)


@pytest.mark.parametrize("dt", [F32, BF])
def test_what_is_no_candidate(dt):
    """Masked tokens, whole rows of them, NaN, +infinity, beams that hold nothing; fewer than K are left."""
    x = (2 * normal(3, 3, 6, 300)).to(dt)
    x[0, :, 2:] = -INF                                  # two tokens are allowed
    x[0, 1] = -INF                                      # none
    x[0, 2, 7] = float("nan")
    x[0, 3, 299] = INF
    x[1, :, ::2] = -INF
    scores = -5 + normal(4, 3, 6)
    scores[0, 4] = -INF
    scores[1, 1:] = -INF                                # the first step: one beam
    scores[2] = -INF
    s, p, t = check(x, scores, 16)
    assert (p[0, 4:] == -1).all() and (t[0, 4:] == -1).all() and (s[0, 4:] == -INF).all()
    assert (p[1] == 0).all() and (t[1] % 2 == 1).all() and (p[2] == -1).all()
    low = torch.finfo(dt).min                           # the type's lowest value is a candidate, behind all others
    x = torch.full((1, 2, 40), low, device="cuda").to(dt)
    x[0, 0, 5] = 0.0
    s, p, t = beam.kda_beam_select(x, torch.zeros((1, 2), device="cuda"), 64)
    assert p[0, 0] == 1 and t[0, 40] == 5 or (p[0, 0], t[0, 0]) == (0, 5)


@pytest.mark.parametrize("kind", [np.uint8, np.bool_])
def test_ended_beams(kind):
    x = 2 * normal(5, 4, 5, 1000)
    scores = -4 + normal(6, 4, 5)
    done = np.zeros((4, 5), kind)
    done[0, 2] = done[1, [0, 4]] = 1
    done[2] = 1
    x[0, 2] = float("nan")                              # not read
    scores[1, 4] = -INF                                 # ended, but holds nothing
    s, p, t = check(x, scores, 10, done, 999)
    assert (t[2, :5] == 999).all() and (p[2, 5:] == -1).all()


def test_rows_of_a_wider_tensor():
    """Rows apart by an odd stride: any alignment; what lies between and around them is not used."""
    wide = torch.full((2, 3, 1237), 1e30, dtype=BF, device="cuda")
    x = (2 * normal(7, 2, 3, 1001)).to(BF)
    wide[:, :, 8:1009] = x
    s, p, t = check(wide[:, :, 8:1009], -3 + normal(8, 2, 3), 9)
    ref = beam.kda_beam_select(x, -3 + normal(8, 2, 3), 9)
    for a, b in zip((s, p, t), ref):
        assert torch.equal(a, b)
    with pytest.raises(ValueError):
        beam.kda_beam_select(wide[:, :2, 8:1009], torch.zeros((2, 2), device="cuda"), 3)  # not evenly apart
    with pytest.raises(ValueError):
        beam.kda_beam_select(x.transpose(1, 2), torch.zeros((2, 1001), device="cuda"), 3)


def test_select_on_streams_in_graphs_and_guarded():
    x, scores = (2 * normal(9, 3, 4, 30011)).to(BF), -3 + normal(10, 3, 4)
    ref = check(x, scores, 8)
    need = beam.kda_beam_select_workspace_size(3, 4, 30011, 8)
    band = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tuple(torch.empty_like(r) for r in ref)
    got = beam.kda_beam_select(x, scores, 8, out=out, workspace=band[4096:4096 + need], stream=side)
    side.synchronize()
    assert all(a is b and torch.equal(a, r) for a, b, r in zip(got, out, ref))
    assert (band[:4096] == 0xA5).all() and (band[4096 + need:] == 0xA5).all()
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        beam.kda_beam_select(x, scores, 8, out=out, workspace=ws)
    for i in range(4):
        [o.zero_() for o in out]
        ws.fill_(255)
        x.copy_((2 * normal(20 + i, 3, 4, 30011)).to(BF))
        g.replay()
        torch.cuda.synchronize()
        for a, r in zip(out, check(x, scores, 8)):
            assert torch.equal(a, r)


# ---- states


def moved(states, slots, parent):
    """The definition: (states, slots) afterwards, on the host."""
    states, old = states.clone(), states.clone()
    out = slots.clone()
    inside = lambda i: 0 <= i < states.shape[1]  # noqa: E731
    for n in range(slots.shape[0]):
        W = slots.shape[1]
        row = [int(p) if 0 <= p < W else -1 for p in parent[n]]
        free = [w for w in range(W) if w not in row]
        for j, p in enumerate(row):
            if p >= 0 and p not in row[:j]:
                out[n, j] = slots[n, p]
                continue
            out[n, j] = slots[n, free.pop(0)]
            a, b = (int(slots[n, p]) if p >= 0 else -1), int(out[n, j])
            if inside(a) and inside(b):
                states[:, b] = old[:, a]
    return states, out


def reorder_case(seed, L, N, W, slots, shape, dtype=F32):
    r = np.random.default_rng(seed)
    states = torch.from_numpy(r.integers(-2 ** 31, 2 ** 31, (L, slots) + shape, dtype=np.int64).astype(np.int32)).view(dtype)
    s = torch.from_numpy(r.permutation(slots)[:N * W].astype(np.int32).reshape(N, W))
    p = torch.from_numpy(r.integers(0, W, (N, W)).astype(np.int32))
    return states, s, p


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("L,N,W,shape", [(1, 1, 1, (4,)), (1, 1, 2, (4,)), (2, 3, 4, (2, 64, 64)), (3, 5, 8, (1, 128, 64)),
                                         (1, 2, 64, (20,)), (2, 7, 5, (1028,)), (1, 1, 4, (3, 128, 128)), (5, 40, 3, (36,))])
def test_reorder(L, N, W, shape):
    states, slots, parent = reorder_case(L + N + W, L, N, W, N * W + 3, shape)
    want, wslots = moved(states, slots, parent)
    x = states.cuda()
    out = beam.kda_state_reorder(x, slots.cuda(), parent.cuda())
    assert torch.equal(out.cpu(), wslots) and same_bits(x.cpu(), want)
    assert torch.equal(out.cpu().sort(1).values, slots.sort(1).values)


@pytest.mark.parametrize("parents", ["same", "all one", "rotated", "none", "outside"])
def test_reorder_kinds_of_parents(parents):
    states, slots, parent = reorder_case(3, 2, 4, 6, 30, (64, 64))
    parent[:] = {"same": torch.arange(6), "all one": torch.full((6,), 2), "rotated": torch.tensor([5, 0, 1, 2, 3, 4]),
                 "none": torch.full((6,), -1), "outside": torch.tensor([3, 6, -2, 3, 2 ** 31 - 1, 0])}[parents].int()
    want, wslots = moved(states, slots, parent)
    x = states.cuda()
    out = beam.kda_state_reorder(x, slots.cuda(), parent.cuda())
    assert torch.equal(out.cpu(), wslots) and same_bits(x.cpu(), want)
    if parents in ("same", "rotated", "none"):
        assert same_bits(x.cpu(), states)


def test_reorder_slots_outside_and_layers_apart():
    states, slots, parent = reorder_case(4, 3, 5, 4, 24, (2, 32, 16))
    slots[0, 1], slots[2, 0], slots[3, 3] = -1, 24, 2 ** 31 - 1
    want, wslots = moved(states, slots, parent)
    wide = torch.full((3, 26, 2, 32, 16), 1.5, device="cuda")
    wide[:, 1:25] = states.cuda()
    x = wide[:, 1:25]
    out = beam.kda_state_reorder(x, slots.cuda(), parent.cuda())
    assert torch.equal(out.cpu(), wslots) and same_bits(x.cpu(), want) and (wide[:, [0, 25]] == 1.5).all()


def test_reorder_other_types_streams_and_graphs():
    states, slots, parent = reorder_case(5, 2, 3, 4, 15, (4, 64), torch.int32)
    x, s, p = states.view(BF).cuda(), slots.cuda(), parent.cuda()
    want, wslots = moved(states, slots, parent)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = beam.kda_state_reorder(x, s, p, stream=side)
    side.synchronize()
    assert same_bits(x.cpu(), want) and torch.equal(out.cpu(), wslots)
    out = torch.empty_like(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        beam.kda_state_reorder(x, s, p, slots_out=out)
    for i in range(4):
        states, slots, parent = reorder_case(6 + i, 2, 3, 4, 15, (4, 64), torch.int32)
        x.copy_(states.view(BF)), s.copy_(slots), p.copy_(parent), out.zero_()
        g.replay()
        torch.cuda.synchronize()
        want, wslots = moved(states, slots, parent)
        assert same_bits(x.cpu(), want) and torch.equal(out.cpu(), wslots)
    with pytest.raises(kda.KDAError):
        beam.kda_state_reorder(x, s, p, slots_out=s)
    with pytest.raises(ValueError):
        beam.kda_state_reorder(x, s, p[:2])
    with pytest.raises(kda.KDAError):
        beam.kda_state_reorder(torch.zeros((1, 12, 3), device="cuda"), s, p)  # rows of 12 bytes


# ---- together


@pytest.mark.parametrize("layer", ["linear", "kda"])
def test_a_beam_search(layer):
    """Prompts, then steps of a beam search with one layer and a vocabulary: every beam's state, kept in slots
    that are reordered, equals the state of its whole line of tokens run from the prompt."""
    N, W, H, d, V, steps = 3, 4, 2, 64, 211, 6
    r = torch.Generator(device="cuda").manual_seed(11)

    def rnd(*shape):
        return torch.randn(shape, generator=r, device="cuda")

    emb = {c: rnd(V, H, d) for c in "qkv"}
    emb["k"] /= d ** 0.5 * 1.5
    gate = -0.2 * torch.rand((V, H), generator=r, device="cuda")
    head = 0.2 * rnd(H * d, V)

    def tokens(ids):
        ids = ids.long()
        return tuple(emb[c][ids].contiguous() for c in "qkv") + (gate[ids].contiguous(),)

    def prompt(ids, cu, cache, slots):
        q, k, v, g = tokens(ids)
        if layer == "linear":
            return lin.kda_lin_chunk_fwd(q, k, v, g, cu, initial_state=cache, state_slots=slots)[0]
        beta = torch.full((len(ids), H), 0.5, device="cuda")
        return kda.kda_chunk_fwd_ex(q, k, v, cu, log_alpha=g[..., None].expand(-1, -1, d).contiguous(), beta=beta,
                                    initial_state=cache, state_slots=slots)[0]

    def step(ids, cache, slots):
        q, k, v, g = tokens(ids)
        if layer == "linear":
            return lin.kda_lin_decode_step(q, k, v, g, cache, slots)
        beta = torch.full((len(ids), H), 0.5, device="cuda")
        return kda.kda_decode_step(q, k, v, g[..., None].expand(-1, -1, d).contiguous(), beta, cache, slots)

    lens = [70, 1, 33]
    ids = torch.randint(V, (sum(lens),), generator=r, device="cuda")
    cache = torch.zeros((N * W + 2, H, d, d), device="cuda")
    slots = torch.arange(N * W, dtype=torch.int32, device="cuda").view(N, W) + 1
    o = prompt(ids, lc.offsets(lens), cache, slots[:, 0].contiguous())
    last = o[torch.tensor(lens).cumsum(0).cuda() - 1].reshape(N, 1, -1)
    logits = (last.expand(N, W, -1) @ head)
    scores = torch.full((N, W), -INF, device="cuda")
    scores[:, 0] = 0.0
    lines = [[list(ids[sum(lens[:n]):sum(lens[:n + 1])].tolist()) for _ in range(W)] for n in range(N)]
    for i in range(steps):
        scores, parent, token = beam.kda_beam_select(logits.contiguous(), scores, W)
        slots = beam.kda_state_reorder(cache[None], slots, parent)
        assert (parent >= 0).all()
        p, t = parent.tolist(), token.tolist()
        lines = [[lines[n][p[n][w]] + [t[n][w]] for w in range(W)] for n in range(N)]
        o = step(token.view(-1), cache, slots.view(-1))
        logits = (o.reshape(N, W, -1) @ head)
    every = [line for row in lines for line in row]
    check_cache = torch.zeros((N * W, H, d, d), device="cuda")
    prompt(torch.tensor(sum(every, []), device="cuda"), lc.offsets([len(x) for x in every]), check_cache,
           torch.arange(N * W, dtype=torch.int32, device="cuda"))
    got = cache[slots.view(-1).long()]
    # two orders of fp32 sums over at most 80 tokens: far below 1e-4 of the states' size
    assert (got - check_cache).abs().max() <= 1e-4 * check_cache.abs().max()
    assert len({tuple(x) for x in every}) == N * W  # every beam is a line of its own
