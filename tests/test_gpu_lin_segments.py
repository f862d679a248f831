"""kda_lin_chunk_fwd where sequences are cut into segments: each test asserts that its batch is (such a call has a
workspace), so that a change of the rule that decides it cannot leave the test without its subject."""

import numpy as np
import pytest
import torch

from gated_delta_rule_10_amd import lin
from tests import lin_common as lc

pytestmark = pytest.mark.gpu
F32 = torch.float32


def cut(x, N, H, dk, dv):
    need = lin.kda_lin_chunk_fwd_workspace_size(N, x.T, H, dk, dv, x.q.dtype)
    assert need > 0, "this batch is not cut"
    return need


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_long_sequences_among_more_than_64(dt, dk, dv):
    """Cut sequences, two segments and many, before, between and behind more than 64 short and empty ones."""
    lens = [2] * 3 + [900] + [0] * 66 + [1500] + [1] * 69 + [1250, 0, 258, 5, 640] + [3] * 60 + [777]
    x = lc.Inputs(40, lens, 1, 1, dk, dv, dt, rate=0.01)
    cut(x, len(lens), 1, dk, dv)
    o, s = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
    x.check(o, s, x.s0, 1.0)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("lens,H", [([5, 64, 3000, 130, 0, 300, 65, 1], 40), ([5, 64, 700, 130, 0, 300, 65, 1], 40), ([200, 5, 130, 64], 80)])
def test_order_where_the_card_is_full(dt, order, lens, H):
    """Workgroups in the order of their tokens, more than the card holds: each sequence has the bits that it has in
    another order. One sequence is cut, none is long enough, and (four sequences) none can be."""
    dk, dv, N = 64, 128, len(lens)
    x = lc.Inputs(4, lens, H, H // 5, dk, dv, dt)
    assert N * H > torch.cuda.get_device_properties(0).multi_processor_count
    assert (lin.kda_lin_chunk_fwd_workspace_size(N, x.T, H, dk, dv, x.q.dtype) > 0) == (N == 8)
    ref, rs = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
    x.check(ref, rs, x.s0, 1.0)
    to = {"rising": np.argsort(lens, kind="stable"), "falling": np.argsort(lens, kind="stable")[::-1],
          "mixed": np.random.default_rng(1).permutation(N)}[order]
    at = np.concatenate([[0], np.cumsum(lens)])
    rows = torch.from_numpy(np.concatenate([np.arange(at[n], at[n + 1]) for n in to])).cuda()
    seqs = torch.from_numpy(to.copy()).cuda()
    o, s = lin.kda_lin_chunk_fwd(x.q[rows], x.k[rows], x.v[rows], x.g[rows], lc.offsets([lens[n] for n in to]),
                                 initial_state=x.s0[seqs])
    assert torch.equal(o, ref[rows]) and torch.equal(s, rs[seqs])


@pytest.mark.parametrize("dt,out", [("bf16", torch.bfloat16), ("bf16", F32), ("f32", F32)])
@pytest.mark.parametrize("where", ["q", "k", "v", "g"])
@pytest.mark.parametrize("t", [70, 1111, 1999])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_what_is_not_finite_reaches_no_earlier_token(dt, out, where, t, bad):
    """In the first, a middle and the last segment of the second sequence."""
    lens = [700, 2000, 300]
    x = lc.Inputs(10, lens, 4, 2, 128, 128, dt, rate=1e-3)
    cut(x, 3, 4, 128, 128)
    clean, cs = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, out_dtype=out)
    h, row = 1, 700 + t
    if where == "g":
        x.g[row, h] = bad
    else:
        getattr(x, where)[row, h, 3] = bad
    o, s = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, out_dtype=out)
    hit = [h] if where in "vg" else [2 * h, 2 * h + 1]
    rest = [i for i in range(4) if i not in hit]
    assert torch.equal(o[:, rest], clean[:, rest]) and torch.equal(s[:, rest], cs[:, rest])
    assert torch.equal(o[:row], clean[:row]) and torch.equal(o[2700:], clean[2700:])
    assert torch.equal(s[[0, 2]], cs[[0, 2]])
    assert not torch.isfinite(o[row, hit]).all()
    if where == "q":
        assert torch.equal(o[row + 1:], clean[row + 1:]) and torch.equal(s, cs)
    else:  # heads that forget slowly: it has not decayed
        assert not torch.isfinite(s[1, hit]).all() and not torch.isfinite(o[2699, hit]).all()
    if where == "v":
        cols = [i for i in range(128) if i != 3]
        assert torch.equal(o[:, :, cols], clean[:, :, cols]) and torch.equal(s[..., cols], cs[..., cols])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_slots(dt):
    """A cut sequence's state in a slot, in no slot (padding), and the final states over the initial ones."""
    lens, dk, dv = [1300, 900, 70, 1100], 64, 128
    x = lc.Inputs(7, lens, 2, 2, dk, dv, dt, rate=0.01)
    cut(x, 4, 2, dk, dv)
    cache = torch.randn((6, 2, dk, dv), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    slots = torch.tensor([4, -1, 6, 0], dtype=torch.int32, device="cuda")
    before = cache.clone()
    S0 = torch.zeros((4, 2, dk, dv), device="cuda")
    S0[0], S0[3] = cache[4], cache[0]
    o, s = lin.kda_lin_chunk_fwd(*x.args(), initial_state=cache, state_slots=slots)
    ref, rs = lin.kda_lin_chunk_fwd(*x.args(), initial_state=S0)
    x.check(ref, rs, S0, 1.0)
    assert s.data_ptr() == cache.data_ptr()
    assert torch.equal(o, ref) and torch.equal(cache[[4, 0]], rs[[0, 3]]) and torch.equal(cache[[1, 2, 3, 5]], before[[1, 2, 3, 5]])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offsets_that_break_the_rules_stay_inside(dt):
    """Offsets below 0 and behind the last row are clamped, sequences that would end before they begin have no tokens;
    what lies around the outputs, the states and the workspace is not touched."""
    x = lc.Inputs(11, [1500, 900], 2, 2, 64, 64, dt, rate=0.01)
    need = cut(x, 2, 2, 64, 64)
    ref, rs = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)

    def banded(like, nbytes):
        b = torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        return b, b[4096:4096 + nbytes] if like is None else b[4096:4096 + nbytes].view(like.dtype).view(like.shape)

    for cu in ([-50, 1500, 10 ** 6], [-2 ** 31, 1500, 2 ** 31 - 1], [2400, 1500, 0], [1500, 1500, 2400], [900, 2400, 1500]):
        (bo, o), (bs, s), (bw, w) = banded(ref, ref.numel() * ref.element_size()), banded(rs, rs.numel() * 4), banded(None, need)
        lin.kda_lin_chunk_fwd(x.q, x.k, x.v, x.g, torch.tensor(cu, dtype=torch.int32, device="cuda"), initial_state=x.s0, o=o,
                              final_state=s, workspace=w)
        if cu[1] == 1500 and cu[0] < 0:
            assert torch.equal(o, ref) and torch.equal(s, rs)
        for b, inner in ((bo, o), (bs, s), (bw, w)):
            n = inner.numel() * inner.element_size()
            assert (b[:4096] == 0xA5).all() and (b[4096 + n:] == 0xA5).all()


def test_rows_far_apart():
    """The largest token stride, 2^24 elements, over a cut sequence; decays too."""
    lens, H, stride = [620, 300], 2, 1 << 24
    x = lc.Inputs(30, lens, H, 1, 64, 64, "bf16", rate=0.05)
    need = cut(x, 2, H, 64, 64)
    wide = torch.empty(((x.T - 1) * stride + 512,), dtype=torch.bfloat16, device="cuda")

    def part(at, heads, d):
        return wide.as_strided((x.T, heads, d), (stride, d, 1), at)

    q, k, v = part(0, 1, 64), part(64, 1, 64), part(128, H, 64)
    q.copy_(x.q), k.copy_(x.k), v.copy_(x.v)
    g = torch.empty(((x.T - 1) * stride + 8,), device="cuda").as_strided((x.T, H), (stride, 1))
    g.copy_(x.g)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    ref, rs = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
    o, s = lin.kda_lin_chunk_fwd(q, k, v, g, x.cu, initial_state=x.s0, workspace=ws)
    assert torch.equal(o, ref) and torch.equal(s, rs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_a_graph(dt):
    """A skewed batch, captured and replayed, with other inputs and a workspace that holds anything."""
    lens = [30] * 5 + [4000] + [30] * 18
    x = lc.Inputs(12, lens, 4, 2, 128, 128, dt, rate=0.05)
    ws = torch.empty(cut(x, len(lens), 4, 128, 128), dtype=torch.uint8, device="cuda")
    ref, rs = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
    o, s = torch.empty_like(ref), torch.empty_like(rs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, o=o, final_state=s, workspace=ws)
    for i in range(4):
        o.zero_(), s.zero_(), ws.fill_(255 if i % 2 else 0)
        x.v.mul_(-0.5)
        g.replay()
        torch.cuda.synchronize()
        now, ns = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
        assert torch.equal(o, now) and torch.equal(s, ns)
