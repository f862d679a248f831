"""kda_kv_write and kda_kv_read against the plain 64-bit form (tests/attn_common.py).
Codes and exponents have to be equal: the only rounding is to the nearest code."""

import numpy as np
import pytest
import torch

from gated_delta_rule_10_amd import attn
from tests import attn_common as ac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def wanted(k, kv):
    """What a cache of kind kv holds for k, 64 bits on the CPU."""
    if kv != "e4m3":
        return k.double().cpu()
    codes, e = ac.to_codes(k.double().cpu().numpy())
    return torch.from_numpy(codes * np.exp2(e.astype(np.float64))[..., None])


def same(a, b):
    return torch.equal(torch.nan_to_num(a, 12345.0), torch.nan_to_num(b, 12345.0)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("dt,kv", [("bf16", "e4m3"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_write_and_read(dt, kv, dk, dv, page):
    new, ctx, Hk = [1, 70, 0, 3, 33], [0, 30, 9, 255, 17], 3
    c = ac.Cache([a + b for a, b in zip(new, ctx)], Hk, dk, dv, page, kv, seed=page)
    before = [getattr(c, x).view(torch.uint8).clone() for x in ("k", "v")]
    T = sum(new)
    k, v = ac.normal(1, T, Hk, dk).to(DT[dt]).cuda(), (100 * ac.normal(2, T, Hk, dv)).to(DT[dt]).cuda()
    cu = ac.offsets(new)
    attn.kda_kv_write(k, v, cu, *c.args(), **c.exps())
    rk, rv = attn.kda_kv_read(T, cu, *c.args(), **c.exps(), out_dtype=torch.float32)
    assert same(rk.double().cpu(), wanted(k, kv)) and same(rv.double().cpu(), wanted(v, kv))
    back = attn.kda_kv_read(T, cu, *c.args(), **c.exps(), out_dtype=DT[dt])
    assert torch.equal(back[0].float(), rk) and torch.equal(back[1].float(), rv)  # exact in bf16 too
    # every other place of the cache is as it was
    at = 0
    held = torch.zeros(c.k.shape[0], c.page, dtype=torch.bool)
    for n, L in enumerate(new):
        page_, off = c.place(n, np.arange(ctx[n], ctx[n] + L))
        held[torch.from_numpy(page_).long(), torch.from_numpy(off).long()] = True
        at += L
    for x, b in zip(("k", "v"), before):
        now = getattr(c, x).view(torch.uint8)
        rest = ~held[:, None, :, None].expand(now.shape).cuda()
        assert torch.equal(now[rest], b[rest])
        if kv == "e4m3":
            e = getattr(c, x + "_exp")
            assert (e[~held[:, None].expand(e.shape).cuda()] == 0xFF).all()


def test_codes_of_every_kind_of_row():
    """Rows of zeros, one element, the largest and the smallest bf16 numbers, powers of two, numbers at
    7/8 of a power of two and next to it, ties, infinities, NaN."""
    d, rows = 64, []

    def row(*x):
        r = torch.zeros(d)
        r[:len(x)] = torch.tensor(x)
        rows.append(r)

    row(0.0)
    row(-0.0, 1.0)
    row(448.0, 1.0, -3.3)
    row(449.0)
    row(450.0, 17.0, 19.0, 1.0625)       # bf16 450: past 448, the exponent is one more
    row(446.0, 17.0, 19.0, 21.0)
    row(3.0 * 2.0 ** 120, 1.0)
    row(2.0 ** 127, -2.0 ** 127)
    row(2.0 ** -133, 2.0 ** -130)        # bf16 denormals
    row(2.0 ** -126 * 1.5, 2.0 ** -133)
    row(0.875, 0.876953125, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11)
    row(1.0, 2.0 ** -20)
    row(float("inf"), 5.0, -2.0)
    row(float("nan"), -float("inf"), 0.25)
    row(float("nan"))
    for s in range(40):
        rows.append(ac.normal(s, d) * 10.0 ** (s - 20))
    k = torch.stack(rows)[:, None].to(torch.bfloat16).cuda()
    T = k.shape[0]
    c = ac.Cache([T], 1, d, d, 32, "e4m3")
    cu = ac.offsets([T])
    attn.kda_kv_write(k, -k, cu, *c.args(), **c.exps())
    page, off = (torch.from_numpy(x).long() for x in c.place(0, np.arange(T)))
    codes, e = ac.to_codes(k.double().cpu().numpy())
    assert torch.equal(c.k_exp.cpu()[page, :, off].long(), torch.from_numpy(e + 127))
    got = c.k.cpu().view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).double()
    assert same(got, torch.from_numpy(codes))
    rk, rv = attn.kda_kv_read(T, cu, *c.args(), **c.exps(), out_dtype=torch.float32)
    ref = torch.from_numpy(codes * np.exp2(e.astype(np.float64))[..., None]).to(torch.float32)
    assert same(rk.cpu(), ref) and same(rv.cpu(), -ref)
    rk, _ = attn.kda_kv_read(T, cu, *c.args(), **c.exps(), out_dtype=torch.bfloat16)
    assert same(rk.cpu().float(), ref.to(torch.bfloat16).float())
    # what was read is written again as it is
    again = ac.Cache([T], 1, d, d, 32, "e4m3")
    fine = torch.isfinite(rk).all(-1).all(-1) & (rk.abs().amax((-1, -2)) < 1e38) & (rk.abs().amax((-1, -2)) > 1e-30)
    attn.kda_kv_write(rk, rv.bfloat16(), cu, *again.args(), **again.exps())
    r2, _ = attn.kda_kv_read(T, cu, *again.args(), **again.exps())
    assert torch.equal(r2[fine], rk[fine])


def test_parts_of_wider_rows():
    x = ac.normal(3, 40, 6, 64).bfloat16().cuda()
    k, v = x[:, 2:4], x[:, 4:]
    c, e = ac.Cache([40], 2, 64, 64, 16, "bf16"), ac.Cache([40], 2, 64, 64, 16, "e4m3")
    cu = ac.offsets([40])
    for cache in (c, e):
        attn.kda_kv_write(k, v, cu, *cache.args(), **cache.exps())
        rk, rv = attn.kda_kv_read(40, cu, *cache.args(), **cache.exps(), out_dtype=torch.float32)
        assert same(rk.double().cpu(), wanted(k, cache.kv)) and same(rv.double().cpu(), wanted(v, cache.kv))


@pytest.mark.parametrize("kv", ["e4m3", "bf16"])
def test_places_that_are_not_there(kv):
    """Tokens with a negative position, on a page that the table does not have, past the table, and rows
    behind the last sequence: nothing is written for them, and zeros (nothing at all behind the last
    sequence) are read."""
    c = ac.Cache([40, 40, 40], 2, 64, 64, 16, kv, max_pages=3)
    table = c.table.clone()
    table[0, 1] = -1
    table[1, 1] = c.k.shape[0]          # one past the last page
    lens = torch.tensor([40, 40, 100], dtype=torch.int32, device="cuda")  # sequence 2: places 60 .. 99 of 48
    lens[0] = 30                        # its 40 new tokens: places -10 .. 29
    new, T = [40, 40, 40], 125
    k, v = ac.normal(4, T, 2, 64).bfloat16().cuda(), ac.normal(5, T, 2, 64).bfloat16().cuda()
    cu = ac.offsets(new)
    was = c.k.view(torch.uint8).clone()
    args = (lens, table, c.k, c.v)
    attn.kda_kv_write(k, v, cu, *args, **c.exps())
    o = [torch.full((T, 2, 64), 3.0, dtype=torch.float32, device="cuda") for _ in "kv"]
    rk, rv = attn.kda_kv_read(T, cu, *args, **c.exps(), out_dtype=torch.float32, k=o[0], v=o[1])
    torch.cuda.synchronize()
    there = torch.zeros(T, dtype=torch.bool)
    there[10:26] = True                 # sequence 0: places 0 .. 15; 16 .. 29 lie on the missing page
    there[40:56] = True                 # sequence 1: places 0 .. 15, then the bad page
    there[72:80] = True                 # and 32 .. 39
    for got, x in ((rk, k), (rv, v)):
        got = got.double().cpu()
        assert same(got[there], wanted(x, kv)[there])
        assert (got[:120][~there[:120]] == 0).all() and (got[120:] == 3).all()
    changed = (c.k.view(torch.uint8) != was).any(-1).any(1)  # [pages, offset]
    assert int(changed.sum()) <= int(there.sum())


def test_one_token_for_many_sequences():
    N = 600
    c = ac.Cache([1 + n % 40 for n in range(N)], 1, 64, 64, 16, "e4m3")
    k, v = ac.normal(6, N, 1, 64).bfloat16().cuda(), ac.normal(7, N, 1, 64).bfloat16().cuda()
    cu = ac.offsets([1] * N)
    attn.kda_kv_write(k, v, cu, *c.args(), **c.exps())
    rk, rv = attn.kda_kv_read(N, cu, *c.args(), **c.exps(), out_dtype=torch.float32)
    assert same(rk.double().cpu(), wanted(k, "e4m3")) and same(rv.double().cpu(), wanted(v, "e4m3"))


@pytest.mark.parametrize("lens", [[0] * 100 + [3] + [0] * 90 + [200, 0, 1], [1, 0] * 80, [130]])
def test_sequences_without_tokens_between_others(lens):
    """The place of a token is found whatever number of empty sequences lies before it."""
    c = ac.Cache([x + 5 for x in lens], 3, 64, 64, 16, "bf16")
    T = sum(lens)
    k, v = ac.normal(8, T, 3, 64).bfloat16().cuda(), ac.normal(9, T, 3, 64).bfloat16().cuda()
    cu = ac.offsets(lens)
    attn.kda_kv_write(k, v, cu, *c.args())
    rk, rv = attn.kda_kv_read(T, cu, *c.args())
    assert torch.equal(rk, k) and torch.equal(rv, v)
    at = 0
    for n, L in enumerate(lens):
        held = c.values(n, L + 5)
        assert torch.equal(held[0][5:], k[at:at + L].double().cpu()) and torch.equal(held[1][5:], v[at:at + L].double().cpu())
        at += L


def test_another_stream_and_capture():
    c, e = (ac.Cache([9, 40], 2, 64, 64, 16, "e4m3") for _ in "ce")
    k, v = ac.normal(10, 12, 2, 64).bfloat16().cuda(), ac.normal(11, 12, 2, 64).bfloat16().cuda()
    cu = ac.offsets([2, 10])
    attn.kda_kv_write(k, v, cu, *c.args(), **c.exps())
    want = attn.kda_kv_read(12, cu, *c.args(), **c.exps())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    attn.kda_kv_write(k, v, cu, *e.args(), **e.exps(), stream=s)
    got = attn.kda_kv_read(12, cu, *e.args(), **e.exps(), stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.zeros_like(x) for x in want]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        attn.kda_kv_write(k, v, cu, *e.args(), **e.exps())
        attn.kda_kv_read(12, cu, *e.args(), **e.exps(), k=out[0], v=out[1])
    for step in range(3):
        k.copy_(ac.normal(20 + step, *k.shape))
        graph.replay()
        got = out[0].clone()
        attn.kda_kv_write(k, v, cu, *c.args(), **c.exps())
        want = attn.kda_kv_read(12, cu, *c.args(), **c.exps())
        torch.cuda.synchronize()
        assert torch.equal(got, want[0]) and torch.equal(out[1], want[1])


def test_refused_on_the_gpu():
    c = ac.Cache([4], 1, 64, 64, 16, "e4m3")
    k = torch.zeros((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    cu = ac.offsets([4])
    with pytest.raises(ValueError):
        attn.kda_kv_write(k, k, cu, *c.args())                                  # no exponents
    with pytest.raises(ValueError):
        attn.kda_kv_write(k, k[:3], cu, *c.args(), **c.exps())
    with pytest.raises(ValueError):
        attn.kda_kv_write(k, k, cu, c.lens, c.table.expand(1, 4), c.k, c.v, **c.exps())
    with pytest.raises(ValueError):
        attn.kda_kv_write(k.expand(4, 2, 64), k.expand(4, 2, 64), cu, *c.args(), **c.exps())
    with pytest.raises(RuntimeError):
        attn.kda_kv_write(k.float(), k.float(), cu, *c.args(), **c.exps())      # fp32 into codes
    with pytest.raises(TypeError):
        attn.kda_kv_read(4, cu, c.lens, c.table, c.k.view(torch.uint8), c.v.view(torch.uint8))
    with pytest.raises(ValueError):
        attn.kda_kv_read(4, cu, *c.args(), **c.exps(), k=torch.empty((4, 1, 32), dtype=torch.bfloat16, device="cuda"))
