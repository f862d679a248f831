"""kda_beam_select over beams whose tokens are masked by large finite numbers: all V tokens of a beam at one value
have probability 1 / V each, whatever the value, so that such a beam's tokens get score - ln V and not score."""

import numpy as np
import pytest
import torch

from gated_delta_rule_10_amd import beam

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def definition(logits, scores, K):
    """Per request (scores, parent, token), [K] each, in 64 bits: (x - top) - ln sum e^(x - top) + score, in which
    nothing small is added to something large; -inf, -1 and -1 where there are fewer than K."""
    x, sc = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    N, W, V = x.shape
    out = np.full((N, K), -np.inf), np.full((N, K), -1), np.full((N, K), -1)
    for n in range(N):
        cand = []
        for w in range(W):
            d = x[n, w] - x[n, w].max()
            c = d - np.log(np.exp(d).sum()) + sc[n, w]
            cand += [(c[t], w, int(t)) for t in np.lexsort((np.arange(V), -d))[:K]]
        cand.sort(key=lambda c: (-c[0], c[1], c[2]))
        for a, b in zip(cand[:K], cand[1:K + 1]):
            assert a[1] == b[1] or a[0] == b[0] or a[0] - b[0] > 1e-6, "two beams' candidates are too near to each other"
        for i, c in enumerate(cand[:K]):
            out[0][n, i], out[1][n, i], out[2][n, i] = c
    return out


def check(logits, scores, K):
    ref, parent, token = definition(logits, scores, K)
    s, p, t = beam.kda_beam_select(logits, scores, K)
    assert np.array_equal(p.cpu().numpy(), parent) and np.array_equal(t.cpu().numpy(), token)
    # the row's logarithm to 2^-22, and one rounding of the score
    got, fine = s.double().cpu().numpy(), ref > -np.inf
    assert np.array_equal(got > -np.inf, fine)
    lim = 2.0 ** -22 + 2.0 ** -24 * np.abs(ref[fine])
    worst = float((np.abs(got[fine] - ref[fine]) / lim).max())
    print(f"  worst error / bound = {worst:.3f}", flush=True)
    assert worst <= 1.0
    return s, p, t


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("mask", ["lowest", -1e30, 1e30])
@pytest.mark.parametrize("V,K", [(40, 64), (5000, 8), (5000, 64), (30011, 16)])
def test_a_beam_without_allowed_tokens(dt, mask, V, K):
    """Beam 0 allows one token, beam 1 none: its tokens have 1 / V each, behind beam 0's one, before its masked ones."""
    low = torch.finfo(dt).min if mask == "lowest" else mask
    x = torch.full((2, 2, V), low, device="cuda").to(dt)
    if low < 0:
        x[:, 0, 5] = 0.0
    s, p, t = check(x, torch.zeros((2, 2), device="cuda"), K)
    if low < 0:
        assert (p[:, 0] == 0).all() and (t[:, 0] == 5).all()
        n = min(K, V + 1)
        assert (p[:, 1:n] == 1).all() and torch.equal(t[0, 1:n].cpu(), torch.arange(n - 1, dtype=torch.int32))
        assert (s[:, 1] + np.log(V)).abs().max() < 1e-5


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("mask", ["lowest", -1e30])
@pytest.mark.parametrize("V", [700, 9001])
def test_live_and_dead_beams(dt, mask, V):
    """Beams that allow all, some and no tokens; the dead ones' scores are better."""
    low = torch.finfo(dt).min if mask == "lowest" else mask
    r = np.random.default_rng(V)
    x = torch.from_numpy(3 * r.standard_normal((3, 6, V))).to("cuda", dt)
    x[:, 1, 20:] = low
    x[:, 2, :-7] = low
    x[:, 3] = low
    x[:, 4, ::2] = low
    scores = torch.from_numpy(-4 + r.standard_normal((3, 6)).astype(np.float32)).cuda()
    scores[:, 3] += 4
    check(x, scores, 32)
