"""Packed sequences that do not begin at the packed axis's first row (a part of a longer table of offsets), for every
operator that finds a row's sequence by its offsets, and offsets that break the rules."""

import pytest
import torch

from gated_delta_rule_10_amd import attn, lin
from tests import attn_common as ac
from tests import lin_common as lc

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def offsets(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("skip,lens", [(7, [3, 40]), (700, [300, 0, 65, 1]), (1000, [5] * 70 + [600] + [1] * 60)])
def test_prompt_attention_from_a_later_row(dt, skip, lens):
    T = skip + sum(lens)
    q, k, v = (ac.normal(i, T, h, 64).to(DT[dt]).cuda() for i, h in ((1, 4), (2, 2), (3, 2)))
    cu = [skip]
    for n in lens:
        cu.append(cu[-1] + n)
    o = torch.full_like(q, 7.0)
    attn.kda_attn_fwd(q, k, v, offsets(cu), o=o)
    ref = attn.kda_attn_fwd(q[skip:], k[skip:], v[skip:], offsets([x - skip for x in cu]))
    torch.cuda.synchronize()
    assert torch.equal(o[skip:], ref) and (o[:skip] == 7).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("skip,new", [(5, [1, 3]), (130, [1, 70, 0, 3, 33]), (300, [2] * 80 + [90])])
def test_cache_from_a_later_row(kv, skip, new):
    """Written, read and attended to: rows before the first sequence are left as they were."""
    c = ac.Cache([n + 40 for n in new], 2, 64, 64, 16, kv, seed=1)
    d = ac.Cache([n + 40 for n in new], 2, 64, 64, 16, kv, seed=1)
    T = skip + sum(new)
    k, v, q = (ac.normal(i, T, h, 64).bfloat16().cuda() for i, h in ((1, 2), (2, 2), (3, 4)))
    cu, cu0 = [skip], [0]
    for n in new:
        cu.append(cu[-1] + n)
        cu0.append(cu0[-1] + n)
    cu, cu0 = offsets(cu), offsets(cu0)
    for x, a, b, at in ((c, k, v, cu), (d, k[skip:], v[skip:], cu0)):
        for t in (x.k, x.v) + ((x.k_exp, x.v_exp) if kv == "e4m3" else ()):
            t.view(torch.uint8).zero_()
        attn.kda_kv_write(a, b, at, *x.args(), **x.exps())
    torch.cuda.synchronize()
    for a, b in ((c.k, d.k), (c.v, d.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    rk, rv = attn.kda_kv_read(T, cu, *c.args(), **c.exps(), out_dtype=torch.bfloat16)
    sk, sv = attn.kda_kv_read(T - skip, cu0, *d.args(), **d.exps(), out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(rk[skip:], sk) and torch.equal(rv[skip:], sv)
    o = torch.full_like(q, 7.0)
    attn.kda_attn_cache_fwd(q, cu, *c.args(), **c.exps(), o=o)
    ref = attn.kda_attn_cache_fwd(q[skip:], cu0, *d.args(), **d.exps())
    torch.cuda.synchronize()
    # The work is cut by the call's rows, so sums may be joined at other places: on each side weights are off by up to
    # 2^-8 (and sums by far less), and the output is rounded by 2^-8 of itself.
    far = (o[skip:].float() - ref.float()).abs()
    assert (o[:skip] == 7).all() and (far <= 2.0 ** -6 * v.float().abs().max() + 2.0 ** -7 * ref.float().abs()).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("skip,lens", [(7, [3, 40]), (700, [2000, 0, 65, 1])])
def test_linear_attention_from_a_later_row(dt, skip, lens):
    x = lc.Inputs(3, [skip] + lens, 2, 1, 64, 64, dt, rate=0.02)
    cu = x.cu[1:].clone()
    T = x.T
    o = torch.full((T, 2, 64), 7.0, dtype=DT[dt], device="cuda")
    _, s = lin.kda_lin_chunk_fwd(x.q, x.k, x.v, x.g, cu, initial_state=x.s0[1:], o=o)
    torch.cuda.synchronize()
    assert (o[:skip] == 7).all()
    at = skip
    for n, (L, (ro, ao, rs, as_)) in enumerate(list(zip(x.lens, x.reference(x.s0, 1.0)))[1:]):
        lc.check(f"o {n}", o[at:at + L], ro, ao, x.bound(L, 64, dt == "bf16"), dt == "bf16")
        lc.check(f"state {n}", s[n], rs, as_, lc.e32(L, 64))
        at += L


@pytest.mark.parametrize("cu", [[600, 300, 0], [300, 300, 100], [-5, 10 ** 6, 2 ** 31 - 1], [600, 600, 600], [2 ** 31 - 1, -2 ** 31, 0]])
def test_offsets_that_break_the_rules_stay_inside(cu):
    """Falling and far ones: nothing around the outputs is touched."""
    T = 600
    q, k, v = (ac.normal(i, T, h, 64).bfloat16().cuda() for i, h in ((1, 4), (2, 2), (3, 2)))
    c = ac.Cache([400, 500], 2, 64, 64, 16, "bf16", seed=1)

    def banded():
        b = torch.full((T + 128, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        return b, b[64:64 + T]

    at = offsets(cu)
    for call in (lambda o: attn.kda_attn_fwd(q, k, v, at, o=o), lambda o: attn.kda_attn_cache_fwd(q, at, *c.args(), o=o)):
        b, o = banded()
        call(o)
        torch.cuda.synchronize()
        assert (b[:64] == 7).all() and (b[64 + T:] == 7).all()
    attn.kda_kv_write(k, v, at, *c.args())
    attn.kda_kv_read(T, at, *c.args())
    torch.cuda.synchronize()
