"""kda_lin_chunk_fwd and kda_lin_decode_step against the definition in 64 bits (tests/lin_common.py, which
derives the bounds)."""

import pytest
import torch

from gated_delta_rule_10_amd import kda, lin
from tests import lin_common as lc

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = [("bf16", BF), ("bf16", F32), ("f32", F32)]


def run(x, **kw):
    o, s = lin.kda_lin_chunk_fwd(*x.args(), **kw)
    torch.cuda.synchronize()
    return o, s


@pytest.mark.parametrize("dt,out", TYPES)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("H,Hk", [(3, 3), (4, 2), (5, 1)])
def test_packed_prompts(dt, out, dk, dv, H, Hk):
    lens = [1, 0, 63, 64, 65, 2, 130, 0, 31, 33, 200]
    x = lc.Inputs(dk + dv + H, lens, H, Hk, dk, dv, dt)
    o, s = run(x, initial_state=x.s0, scale=0.7, out_dtype=out)
    x.check(o, s, x.s0, 0.7)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [16], [17], [63], [64], [65], [127], [128], [129], [191], [0], [0, 0, 5]])
def test_lengths_from_zeros(dt, lens):
    x = lc.Inputs(3, lens, 2, 2, 128, 128, dt)
    o, s = run(x)
    x.check(o, s, None, 1.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("lens", [[2500], [700, 1500, 1, 300], [1024, 1024]])
@pytest.mark.parametrize("rate", [1e-3, 2.0])
def test_long_sequences(dt, dk, dv, lens, rate):
    """Lengths that are cut into segments where few heads leave the card empty."""
    x = lc.Inputs(sum(lens) + dk, lens, 2, 1, dk, dv, dt, rate=rate)
    o, s = run(x, initial_state=x.s0)
    x.check(o, s, x.s0, 1.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_segments_and_the_state_in_place(dt):
    """The final state over the initial one, in segments: the same bits as into another tensor."""
    x = lc.Inputs(8, [3000, 40, 999], 2, 2, 128, 64, dt)
    o, s = run(x, initial_state=x.s0)
    buf = x.s0.clone()
    for _ in range(3):
        buf.copy_(x.s0)
        o2, s2 = run(x, initial_state=buf, final_state=buf)
        assert s2.data_ptr() == buf.data_ptr() and torch.equal(o2, o) and torch.equal(buf, s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [70, 2500])
def test_one_decay_per_head(dt, n):
    x = lc.Inputs(5, [n, 20], 4, 2, 64, 128, dt, decay="heads")
    o, s = run(x, initial_state=x.s0)
    x.check(o, s, x.s0, 1.0)
    wide = x.g.expand(x.T, 4).contiguous()
    o2, s2 = lin.kda_lin_chunk_fwd(x.q, x.k, x.v, wide, x.cu, initial_state=x.s0)
    assert torch.equal(o, o2) and torch.equal(s, s2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "strong", "resets", "all resets", "one in ten"])
@pytest.mark.parametrize("n", [150, 2000])
def test_decays_of_every_size(dt, kind, n):
    x = lc.Inputs(6, [n], 3, 3, 128, 64, dt)
    g = torch.zeros_like(x.g)
    if kind == "strong":
        g = x.g * 100
    if kind == "resets":
        g = x.g.clone()
        g[[0, 5, 63, 64, n - 7]] = -float("inf")
    if kind == "all resets":
        g = torch.full_like(g, -float("inf"))
    if kind == "one in ten":
        g[::10] = -40.0
    x.g = g
    o, s = run(x, initial_state=x.s0)
    x.check(o, s, x.s0, 1.0, kind)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slots(dt):
    """States in a cache: each sequence's slot, and no other, changes; a slot outside the cache is padding."""
    lens = [70, 5, 0, 129, 64]
    x = lc.Inputs(7, lens, 4, 2, 64, 128, dt)
    r = torch.Generator(device="cuda").manual_seed(1)
    cache = torch.randn((9, 4, 64, 128), generator=r, device="cuda")
    slots = torch.tensor([7, -1, 2, 0, 9], dtype=torch.int32, device="cuda")
    S0 = torch.zeros((5, 4, 64, 128), device="cuda")
    for n, i in enumerate([7, None, 2, 0, None]):
        if i is not None:
            S0[n] = cache[i]
    before = cache.clone()
    o, s = run(x, initial_state=cache, state_slots=slots)
    assert s.data_ptr() == cache.data_ptr()
    state = S0.clone()
    ref = x.reference(S0, 1.0)
    for n, i in enumerate([7, None, 2, 0, None]):
        state[n] = cache[i] if i is not None else torch.from_numpy(ref[n][2]).float().cuda()
    x.check(o, state, S0, 1.0)
    for i in (1, 3, 4, 5, 6, 8):
        assert torch.equal(cache[i], before[i])
    assert torch.equal(cache[2], before[2])  # no tokens: as it was
    # another cache for the final states
    other = torch.full_like(before, 5.0)
    o2, _ = run(x, initial_state=before, final_state=other, state_slots=slots)
    assert torch.equal(o2, o) and torch.equal(other[[7, 2, 0]], cache[[7, 2, 0]]) and (other[[1, 3, 4, 5, 6, 8]] == 5).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [100, 2500])
def test_rows_of_a_fused_projection(dt, n):
    """q, k and v as parts of one wider row, decays as a column of another tensor, rows behind the last
    sequence: none of it changes a bit, and rows outside the sequences stay as they were."""
    x = lc.Inputs(9, [n, 33], 4, 2, 128, 64, dt, spare=17)
    fused = torch.full((x.T, 2 * 2 * 128 + 4 * 64 + 24), float("nan"), dtype=x.q.dtype, device="cuda")
    q, k, v = fused[:, 8:264].unflatten(1, (2, 128)), fused[:, 264:520].unflatten(1, (2, 128)), fused[:, 520:776].unflatten(1, (4, 64))
    q.copy_(x.q), k.copy_(x.k), v.copy_(x.v)
    g = torch.full((x.T, 20), float("nan"), device="cuda")
    g[:, 8:12] = x.g
    o = torch.full((x.T, 4, 64), 3.0, dtype=x.q.dtype, device="cuda")
    lin.kda_lin_chunk_fwd(q, k, v, g[:, 8:12], x.cu, o=o, initial_state=x.s0)
    ref, _ = run(x, initial_state=x.s0)
    used = n + 33
    assert torch.equal(o[:used], ref[:used]) and (o[used:] == 3).all()


@pytest.mark.parametrize("dt,out", TYPES)
@pytest.mark.parametrize("where", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite_reaches_no_earlier_token(dt, out, where, bad):
    x = lc.Inputs(10, [150, 90], 4, 2, 128, 128, dt)
    clean, cs = run(x, initial_state=x.s0, out_dtype=out)
    t, h = 70, 1  # of the first sequence
    getattr(x, where)[t, h, 3] = bad
    o, s = run(x, initial_state=x.s0, out_dtype=out)
    hit = [h] if where == "v" else [2 * h, 2 * h + 1]
    rest = [i for i in range(4) if i not in hit]
    assert torch.equal(o[:, rest], clean[:, rest]) and torch.equal(s[:, rest], cs[:, rest])
    assert torch.equal(o[:t], clean[:t]) and torch.equal(o[150:], clean[150:]) and torch.equal(s[1], cs[1])
    assert not torch.isfinite(o[t, hit]).all()
    if where == "q":
        assert torch.equal(o[t + 1:], clean[t + 1:]) and torch.equal(s, cs)
    else:
        assert not torch.isfinite(s[0, hit]).all()
    if where == "v":  # columns of the state are apart
        cols = [i for i in range(128) if i != 3]
        assert torch.equal(o[:, :, cols], clean[:, :, cols]) and torch.equal(s[..., cols], cs[..., cols])


def test_offsets_that_break_the_rules_stay_inside():
    """Offsets below 0 and behind the last row are clamped; what lies around the arrays is not touched."""
    x = lc.Inputs(11, [40, 60], 2, 2, 64, 64, "bf16")
    big = torch.full((100 + 64, 2, 64), 7.0, dtype=BF, device="cuda")
    cu = torch.tensor([-50, 40, 1000], dtype=torch.int32, device="cuda")
    lin.kda_lin_chunk_fwd(x.q, x.k, x.v, x.g, cu, initial_state=x.s0, o=big[32:132])
    ref, _ = run(x, initial_state=x.s0)
    assert torch.equal(big[32:132], ref) and (big[:32] == 7).all() and (big[132:] == 7).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_guard_bands(dt):
    """Outputs, states and workspace between bands of a sentinel."""
    x = lc.Inputs(12, [2000, 77], 2, 2, 128, 128, dt)
    ref, rs = run(x, initial_state=x.s0)
    need = lin.kda_lin_chunk_fwd_workspace_size(2, x.T, 2, 128, 128, x.q.dtype)

    def banded(nbytes):
        b = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return b, b[4096:4096 + nbytes]

    bo, o = banded(ref.numel() * ref.element_size())
    bs, s = banded(rs.numel() * 4)
    bw, w = banded(max(need, 16))
    o, s = o.view(ref.dtype).view(ref.shape), s.view(F32).view(rs.shape)
    lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, o=o, final_state=s, workspace=w)
    assert torch.equal(o, ref) and torch.equal(s, rs)
    for b, inner in ((bo, o), (bs, s), (bw, w)):
        n = inner.numel() * inner.element_size()
        assert (b[:4096] == 0xA5).all() and (b[4096 + n:] == 0xA5).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_same_bits_every_time_on_streams_and_in_graphs(dt):
    x = lc.Inputs(13, [1800, 3, 500], 3, 3, 128, 128, dt)
    ref, rs = run(x, initial_state=x.s0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        o, s = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, stream=side)
        side.synchronize()
        assert torch.equal(o, ref) and torch.equal(s, rs)
    o, s = torch.empty_like(ref), torch.empty_like(rs)
    need = max(16, lin.kda_lin_chunk_fwd_workspace_size(3, x.T, 3, 128, 128, x.q.dtype))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, o=o, final_state=s, workspace=ws)
    for i in range(4):
        o.zero_(), s.zero_(), ws.fill_(255)
        x.q.mul_(-1)  # new inputs in the same places (the matrix cores' sums need not be symmetric in sign)
        g.replay()
        torch.cuda.synchronize()
        now, _ = run(x, initial_state=x.s0)
        assert torch.equal(o, now) and torch.equal(s, rs) and (i % 2 == 0 or torch.equal(o, ref))


def test_a_sequence_alone_and_in_pieces():
    """A prompt in two calls, the state handed over, and one token at a time."""
    x = lc.Inputs(14, [300], 4, 2, 128, 64, "bf16")
    cut = 171
    cu1, cu2 = lc.offsets([cut]), lc.offsets([300 - cut])
    o1, s1 = lin.kda_lin_chunk_fwd(x.q[:cut], x.k[:cut], x.v[:cut], x.g[:cut], cu1, initial_state=x.s0)
    o2, s2 = lin.kda_lin_chunk_fwd(x.q[cut:], x.k[cut:], x.v[cut:], x.g[cut:], cu2, initial_state=s1)
    x.check(torch.cat([o1, o2]), s2, x.s0, 1.0, "two calls")
    cache = x.s0.clone()
    steps = [lin.kda_lin_decode_step(x.q[t:t + 1], x.k[t:t + 1], x.v[t:t + 1], x.g[t:t + 1], cache) for t in range(300)]
    x.check(torch.cat(steps), cache, x.s0, 1.0, "single tokens")


@pytest.mark.parametrize("dt,out", TYPES)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("H,Hk,B", [(1, 1, 1), (6, 2, 5), (5, 5, 33)])
def test_decode_step(dt, out, dk, dv, H, Hk, B):
    x = lc.Inputs(15 + B, [1] * B, H, Hk, dk, dv, dt, rate=3.0)
    cache = torch.randn((B + 4, H, dk, dv), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    idx = torch.randperm(B + 4, generator=torch.Generator().manual_seed(3))[:B].int().cuda()
    S0, before = cache[idx.long()].clone(), cache.clone()
    o = lin.kda_lin_decode_step(x.q, x.k, x.v, x.g, cache, idx, scale=1.5, out_dtype=out)
    # single tokens: fp32 whatever the inputs' type
    for n, (ro, ao, rs, as_) in enumerate(x.reference(S0, 1.5)):
        lc.check(f"o {n}", o[n:n + 1], ro, ao, lc.e32(1, dk), out == BF)
        lc.check(f"state {n}", cache[idx[n].long()], rs, as_, lc.e32(1, dk))
    rest = torch.ones(B + 4, dtype=torch.bool, device="cuda")
    rest[idx.long()] = False
    assert torch.equal(cache[rest], before[rest])


def test_decode_step_padding_strides_and_decays():
    x = lc.Inputs(20, [1] * 4, 4, 2, 64, 64, "bf16", decay="heads")
    cache = torch.randn((4, 4, 64, 64), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    before = cache.clone()
    idx = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    fused = torch.zeros((4, 2 * 2 * 64 + 4 * 64 + 8), dtype=BF, device="cuda")
    q, k, v = fused[:, :128].unflatten(1, (2, 64)), fused[:, 128:256].unflatten(1, (2, 64)), fused[:, 264:].unflatten(1, (4, 64))
    q.copy_(x.q), k.copy_(x.k), v.copy_(x.v)
    o = lin.kda_lin_decode_step(q, k, v, x.g, cache, idx)
    S0 = torch.stack([before[2], torch.zeros_like(before[0]), torch.zeros_like(before[0]), before[0]])
    for n, (ro, ao, rs, as_) in enumerate(x.reference(S0, 1.0)):
        lc.check(f"o {n}", o[n:n + 1], ro, ao, lc.e32(1, 64), True)
        if n in (0, 3):
            lc.check(f"state {n}", cache[idx[n].long()], rs, as_, lc.e32(1, 64))
    assert torch.equal(cache[[1, 3]], before[[1, 3]])
    x.g[:] = -float("inf")  # forgets everything
    o = lin.kda_lin_decode_step(q, k, v, x.g, cache, idx)
    want = torch.einsum("bhi,bhi->bh", x.q.double(), x.k.double()).repeat_interleave(2, 1)[..., None] * x.v.double()
    assert torch.allclose(o.double(), want, rtol=2.0 ** -7, atol=1e-5)


def test_binding_refuses():
    x = lc.Inputs(21, [10], 4, 2, 64, 64, "bf16")
    with pytest.raises(ValueError):
        lin.kda_lin_chunk_fwd(x.q, x.k, x.v[:9], x.g, x.cu)
    with pytest.raises(ValueError):
        lin.kda_lin_chunk_fwd(x.q, x.k.float(), x.v, x.g, x.cu)
    with pytest.raises(ValueError):
        lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0[:, :2])
    with pytest.raises(ValueError):
        lin.kda_lin_chunk_fwd(*x.args(), state_slots=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        lin.kda_lin_chunk_fwd(*x.args(), o=torch.empty((10, 4, 64), device="cuda"))
    with pytest.raises(ValueError):
        lin.kda_lin_chunk_fwd(x.q, x.k, x.v, x.g, x.cu.cpu())
    with pytest.raises(kda.KDAError):
        lin.kda_lin_chunk_fwd(*x.args(), scale=float("nan"))
    with pytest.raises(ValueError):
        lin.kda_lin_decode_step(x.q, x.k, x.v, x.g, x.s0.half())
    with pytest.raises(kda.KDAError):
        lin.kda_lin_decode_step(x.q, x.k, x.v, x.g, x.s0)  # ten tokens, one slot
