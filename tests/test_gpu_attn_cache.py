"""kda_attn_cache_fwd against the plain 64-bit form (tests/attn_common.py), and the
attention operators together as a model's layer uses them."""

import pytest
import torch

from gated_delta_rule_10_amd import attn
from tests import attn_common as ac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
KINDS = [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")]


def filled(seed, lens, Hk, dk, dv, page, kv, **kw):
    c = ac.Cache(lens, Hk, dk, dv, page, kv, seed=seed, **kw)
    for n, L in enumerate(lens):
        c.put(n, ac.normal(seed + 10 * n + 1, L, Hk, dk).to(torch.bfloat16).float(),
              ac.normal(seed + 10 * n + 2, L, Hk, dv).to(torch.bfloat16).float())
    return c


def run(seed, new, ctx, H, Hk, dk, dv, page, dt, kv, masks=None, out=None, scale=None, **kw):
    c = filled(seed, [a + b for a, b in zip(new, ctx)], Hk, dk, dv, page, kv, **kw)
    q = ac.normal(seed, sum(new), H, dk).to(DT[dt]).cuda()
    scale = dk ** -0.5 if scale is None else scale
    got = call(q, new, c, masks, scale, out or dt)
    ref, lim = ac.cache_reference(q, c, new, masks, scale, dt == "bf16", (out or dt) == "bf16")
    ac.check(f"o {dt}/{kv} new {new[:6]} ctx {ctx[:6]}", got, ref, lim)
    return q, c, got


def call(q, new, c, masks, scale, out, **kw):
    return attn.kda_attn_cache_fwd(q, ac.offsets(new), *c.args(), **c.exps(), scale=scale, out_dtype=DT[out],
                                   tree_mask=None if masks is None else ac.mask_tensor(masks), **kw)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_dims(dt, kv, dk, dv):
    run(1, [1, 3, 1], [70, 0, 200], 4, 2, dk, dv, 32, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(dt, kv, page):
    run(2, [1, 1, 1, 1], [0, 15, 16, 300], 8, 2, 128, 128, page, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("H,Hk", [(1, 1), (7, 1), (8, 8), (12, 3), (32, 2), (40, 1)])
def test_heads(dt, kv, H, Hk):
    run(3, [1, 2], [129, 33], H, Hk, 64, 64, 16, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 31, 32, 33, 127, 128, 255, 256, 1023])
def test_one_token(dt, kv, ctx):
    run(4, [1], [ctx], 4, 1, 128, 128, 64, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("new", [[2], [5, 0, 1], [16], [33], [64, 7], [65], [100], [200, 1, 30]])
def test_several_tokens(dt, kv, new):
    """More than 64 new tokens are fine without a mask."""
    run(5, new, [17 * (i + 1) for i in range(len(new))], 4, 1, 64, 64, 32, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_several_tokens_dims_and_pages(dt, kv, dk, dv, page):
    """More than 16 rows for a kv head: 9 and 20 tokens for 3 query heads each; the second has none before it."""
    run(28, [9, 0, 20], [150, 7, 0], 6, 2, dk, dv, page, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
def test_more_rows_than_a_tile(dt, kv):
    """64 drafted tokens for 9 query heads: 576 rows; and 300 tokens in a row."""
    new = [64]
    run(29, new, [100], 9, 1, 64, 64, 32, dt, kv, masks=ac.tree_masks(new, 29))
    run(30, [300], [77], 2, 2, 64, 64, 32, dt, kv)


@pytest.mark.parametrize("dt,kv", KINDS)
def test_several_tokens_over_a_long_cache(dt, kv):
    """Rows of several tokens whose cache is split over workgroups, with a mask."""
    new = [12, 5, 33]
    run(31, new, [2500, 40, 900], 4, 1, 64, 64, 64, dt, kv, masks=ac.tree_masks(new, 31))


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("new", [[1], [2, 9], [24, 3], [63], [64, 64], [5, 0, 31]])
def test_trees(dt, kv, new):
    run(6, new, [50, 3, 0][:len(new)], 8, 2, 64, 128, 16, dt, kv, masks=ac.tree_masks(new, 6))


@pytest.mark.parametrize("dt,kv", KINDS)
def test_long_cache_split_over_workgroups(dt, kv):
    run(7, [1], [5000], 4, 1, 64, 64, 64, dt, kv)
    run(8, [1, 4, 1], [3001, 100, 777], 8, 4, 128, 128, 64, dt, kv)


def test_fp32_out_from_bf16():
    run(9, [1, 5], [90, 400], 8, 2, 128, 128, 32, "bf16", "e4m3", out="f32")


def test_large_scores():
    run(10, [1, 3], [300, 40], 4, 2, 64, 64, 16, "bf16", "e4m3", scale=4.0)
    run(10, [1, 3], [300, 40], 4, 2, 64, 64, 16, "f32", "f32", scale=-2.0)


def test_magnitudes():
    """Tokens whose keys and values differ by many orders of magnitude, each with its own scale."""
    for L, ctx in ((1, 150), (9, 150)):
        c = ac.Cache([ctx + L], 2, 64, 64, 16, "e4m3", seed=33)
        k, v = ac.normal(33, ctx + L, 2, 64), ac.normal(34, ctx + L, 2, 64)
        f = 10.0 ** (6 * torch.rand(ctx + L, 2, 1, generator=torch.Generator().manual_seed(1)) - 6)
        g = 10.0 ** (50 * torch.rand(ctx + L, 2, 1, generator=torch.Generator().manual_seed(2)) - 30)
        c.put(0, (k * f).bfloat16().float(), (v * g).bfloat16().float())
        q = ac.normal(35, L, 8, 64).bfloat16().cuda()
        ref, lim = ac.cache_reference(q, c, [L], None, 0.125, True, True)
        ac.check(f"{L} new", call(q, [L], c, None, 0.125, "bf16"), ref, lim)


def test_many_sequences():
    """More sequences than a workgroup looks over at once, some of them without new tokens."""
    new = [1, 0, 2, 1] * 150
    run(11, new, [(37 * n) % 90 for n in range(600)], 2, 1, 64, 64, 16, "bf16", "e4m3")


@pytest.mark.parametrize("new", [1, 5])
def test_many_sequences_and_a_long_one(new):
    """The work is shared out over 64 sequences at a time, here with pieces that start behind sequences
    without new tokens, and with a whole run of 64 that has none."""
    count = [0 if 70 <= n < 140 else new if n % 3 else 0 for n in range(200)]
    ctx = [(53 * n) % 300 if n != 150 else 3000 for n in range(200)]
    run(26, count, ctx, 6, 1, 64, 64, 16, "bf16", "e4m3")
    run(27, count, ctx, 6, 2, 64, 64, 16, "bf16", "bf16")


def test_page_table_far_longer_than_the_sequences():
    run(12, [1, 1], [20, 150], 4, 2, 64, 64, 16, "bf16", "bf16", max_pages=5000)


@pytest.mark.parametrize("dt,kv", KINDS)
def test_rows_that_see_nothing(dt, kv):
    """An empty mask without context: zeros. With context: the context alone."""
    new, masks = [3, 2], [0, 0b010, 0b001, 0, 0b10]
    _, _, got = run(13, new, [0, 20], 4, 2, 64, 64, 16, dt, kv, masks=masks)
    assert (got[0] == 0).all()


def test_mask_bits_of_tokens_that_are_not_there():
    """Bits past a sequence's new tokens see nothing, and the 65th new token is seen by none."""
    new = [3, 66]
    masks = [-1 & (2 ** 64 - 1)] * 69
    run(14, new, [4, 0], 2, 1, 64, 64, 16, "bf16", "bf16", masks=masks)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("H", [4, 20])
def test_tokens_not_seen_have_no_influence(dt, kv, which, H):
    """A drafted token that holds NaN: rows that do not see it are right, rows that do are NaN. What no
    sequence holds is NaN throughout (ac.Cache fills it so). 10 and 50 rows for a kv head."""
    new, ctx = [5], [45]
    masks = [0b00001, 0b00011, 0b00101, 0b01001, 0b10001]  # token 2 is seen by itself alone
    c = filled(15, [50], 2, 64, 64, 16, kv)
    q = ac.normal(15, 5, H, 64).to(DT[dt]).cuda()
    ref, lim = ac.cache_reference(q, c, new, masks, 0.125, dt == "bf16", dt == "bf16")
    page, off = c.place(0, [ctx[0] + 2])
    getattr(c, which).view(torch.uint8)[int(page[0]), :, int(off[0])] = 0xFF
    got = call(q, new, c, masks, 0.125, dt)
    keep = [0, 1, 3, 4]
    ac.check("rows that do not see it", got[keep], ref[keep], lim[keep])
    assert torch.isnan(got[2]).all()


def test_lengths_and_pages_that_break_the_rules():
    """New tokens with negative positions, a length past the page table, missing and bad pages: nothing
    outside is touched, and what is there is seen."""
    c = filled(16, [40, 40, 48], 1, 64, 64, 16, "bf16", max_pages=3)
    q = ac.normal(16, 6, 2, 64).bfloat16().cuda()
    new = [2, 2, 2]
    lens = torch.tensor([1, 40, 1000], dtype=torch.int32, device="cuda")
    table = c.table.clone()
    table[1, 1] = 10 ** 9
    o = attn.kda_attn_cache_fwd(q, ac.offsets(new), lens, table, c.k, c.v, scale=0.125)
    torch.cuda.synchronize()
    assert (o[0] == 0).all()                              # position -1 sees nothing
    k, v = c.values(0, 1)
    assert torch.equal(o[1].cpu(), v[0].expand(2, 64).bfloat16())
    k, v = (torch.cat([x[:16], x[32:40]]) for x in c.values(1, 40))
    for i in (0, 1):
        sees = torch.ones((1, 24), dtype=torch.bool)
        sees[0, 23] = i == 1                              # position 39 is the second new token
        for h in range(2):
            r = ac.attend(q[2 + i:3 + i, h].cpu(), k[:, 0], v[:, 0], sees, 0.125)
            ac.check("past a bad page", o[2 + i, h][None], r[0], ac.bound(*r, 64, True, True))
    k, v = c.values(2, 48)
    for h in range(2):
        r = ac.attend(q[4:5, h].cpu(), k[:, 0], v[:, 0], torch.ones((1, 48), dtype=torch.bool), 0.125)
        ac.check("past the table", o[4, h][None], r[0], ac.bound(*r, 64, True, True))


def test_lengths_of_zero_write_zeros():
    c = filled(17, [10], 1, 64, 64, 16, "bf16")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = torch.full((2, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    q = ac.normal(17, 2, 2, 64).bfloat16().cuda()
    attn.kda_attn_cache_fwd(q, ac.offsets([1]), lens, c.table, c.k, c.v, o=o)
    assert (o[0] == 0).all() and (o[1] == 5).all()       # and the row behind the last sequence stays


def test_q_of_a_wider_row():
    c = filled(18, [60, 9], 2, 64, 64, 16, "e4m3")
    x = ac.normal(18, 3, 8, 64).bfloat16().cuda()
    q = x[:, :4]
    ref, lim = ac.cache_reference(q, c, [1, 2], None, 0.125, True, True)
    ac.check("o", call(q, [1, 2], c, None, 0.125, "bf16"), ref, lim)


@pytest.mark.parametrize("L", [1, 9])
def test_offsets_past_32_bits(L):
    """A cache of more than 2^32 bytes whose used pages lie at its end, for single and several tokens."""
    pages, page, Hk, d = 2 ** 18 + 40, 64, 1, 128
    k = torch.zeros((pages, Hk, page, d), dtype=torch.bfloat16, device="cuda")
    assert k.numel() * 2 > 2 ** 32
    c = filled(19, [130], Hk, d, d, page, "bf16")
    v = torch.zeros_like(k)
    base = pages - c.k.shape[0]
    k[base:], v[base:] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + base, c.table)
    q = ac.normal(19, L, 4, d).bfloat16().cuda()
    got = attn.kda_attn_cache_fwd(q, ac.offsets([L]), c.lens, table, k, v, scale=0.09)
    ref, lim = ac.cache_reference(q, c, [L], None, 0.09, True, True)
    ac.check("o", got, ref, lim)
    new = ac.normal(20, 1, Hk, d).bfloat16().cuda()
    attn.kda_kv_write(new, new, ac.offsets([1]), c.lens, table, k, v)
    rk, rv = attn.kda_kv_read(1, ac.offsets([1]), c.lens, table, k, v)
    assert torch.equal(rk, new) and torch.equal(rv, new)


def test_same_call_same_bits_whatever_the_workspace_held():
    q, c, a = run(21, [1, 1], [2500, 700], 8, 2, 64, 64, 64, "bf16", "e4m3")
    n = attn.kda_attn_cache_fwd_workspace_size(2, 2, 8, 2, 64, 64, c.table.shape[1] * 64, torch.bfloat16)
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(call(q, [1, 1], c, None, 64 ** -0.5, "bf16", workspace=ws), a)


def test_writes_nothing_outside():
    c = filled(22, [2600, 30], 2, 64, 128, 64, "bf16")
    q = ac.normal(22, 2, 4, 64).bfloat16().cuda()
    n = attn.kda_attn_cache_fwd_workspace_size(2, 2, 4, 2, 64, 128, c.table.shape[1] * 64, torch.bfloat16)
    bufs = []

    def guarded(nbytes):
        bufs.append(torch.full((nbytes + 8192,), 0xA5, dtype=torch.uint8, device="cuda"))
        return bufs[-1][4096:4096 + nbytes]

    o = guarded(2 * 4 * 128 * 2).view(torch.bfloat16).view(2, 4, 128)
    got = call(q, [1, 1], c, None, 0.125, "bf16", o=o, workspace=guarded(n))
    assert torch.equal(got, call(q, [1, 1], c, None, 0.125, "bf16"))
    for b in bufs:
        assert (b[:4096] == 0xA5).all() and (b[-4096:] == 0xA5).all()


def test_another_stream():
    q, c, a = run(23, [1, 2], [1500, 90], 4, 2, 64, 64, 64, "bf16", "e4m3")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [call(q, [1, 2], c, None, 64 ** -0.5, "bf16", stream=s) for _ in range(5)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(o, a) for o in outs)


def test_captured_and_replayed():
    """A layer's decode step in a graph: write, attend. Replays with eager calls between them, new tokens,
    lengths and pages' contents changing under the graph, checked against eager calls each time."""
    N, Hk, H, d, page = 3, 2, 8, 64, 16
    start = [5, 100, 31]
    steps = 6
    c = filled(24, [s + steps for s in start], Hk, d, d, page, "e4m3")
    lens = torch.tensor(start, dtype=torch.int32, device="cuda")
    cu = ac.offsets([1] * N)
    q, k, v = (torch.zeros((N, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk))
    o = torch.zeros_like(q)
    ws = torch.empty(attn.kda_attn_cache_fwd_workspace_size(N, N, H, Hk, d, d, c.table.shape[1] * page, torch.bfloat16) + 16,
                     dtype=torch.uint8, device="cuda")

    def layer(out, work):
        attn.kda_kv_write(k, v, cu, lens, c.table, c.k, c.v, **c.exps())
        attn.kda_attn_cache_fwd(q, cu, lens, c.table, c.k, c.v, **c.exps(), o=out, workspace=work)

    lens += 1
    layer(o, ws)
    lens -= 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(o, ws)
    for step in range(steps):
        lens += 1
        for i, x in enumerate((q, k, v)):
            x.copy_(ac.normal(1000 + 10 * step + i, *x.shape))
        graph.replay()
        got = o.clone()
        eager = torch.empty_like(o)
        layer(eager, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert torch.equal(got, eager), f"replay {step}"
        c.host_lens = [int(x) for x in lens.cpu()]
        ref, lim = ac.cache_reference(q, c, [1] * N, None, d ** -0.5, True, True)
        ac.check(f"replay {step}", got, ref, lim)


def test_captured_tree_over_a_split_cache():
    """Drafted tokens over a cache that is split over workgroups, in two graphs with workspaces of their own,
    replayed in turn with eager calls of other inputs between them."""
    new, H, Hk, d = [6, 11], 8, 2, 64
    c = filled(32, [1500, 700], Hk, d, d, 64, "e4m3")
    T, masks = sum(new), [ac.mask_tensor(ac.tree_masks(new, s)) for s in (1, 2)]
    cu = ac.offsets(new)
    n = attn.kda_attn_cache_fwd_workspace_size(2, T, H, Hk, d, d, c.table.shape[1] * 64, torch.bfloat16)
    assert n > 0
    q = [torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda") for _ in masks]
    o = [torch.zeros_like(x) for x in q]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in masks]

    def layer(i, out, work):
        attn.kda_attn_cache_fwd(q[i], cu, *c.args(), **c.exps(), tree_mask=masks[i], o=out, workspace=work)

    graphs = []
    for i in range(2):
        layer(i, o[i], ws[i])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer(i, o[i], ws[i])
    for step in range(4):
        for i in range(2):
            q[i].copy_(ac.normal(2000 + 10 * step + i, T, H, d))
        graphs[0].replay()
        graphs[1].replay()
        got = [x.clone() for x in o]
        for i in range(2):
            eager = torch.empty_like(o[i])
            layer(i, eager, torch.empty_like(ws[i]))
            torch.cuda.synchronize()
            assert torch.equal(got[i], eager), f"replay {step} of graph {i}"


def test_prompt_then_decode_equals_one_prompt():
    """The operators together: prompts through kda_attn_fwd and into the cache; then single tokens and a tree
    of drafted tokens over it. Over a bf16 cache every token's output is that of one whole prompt."""
    H, Hk, d, page = 8, 2, 128, 16
    whole, prompt = [90, 37], [70, 20]
    T = sum(whole)
    q, k, v = (ac.normal(30 + i, T, h, d).bfloat16().cuda() for i, h in enumerate((H, Hk, Hk)))
    ref, lim = ac.prompt_reference(q, k, v, whole, d ** -0.5, True, True)
    c = ac.Cache(whole, Hk, d, d, page, "bf16")
    rows = [list(range(0, 70)), list(range(90, 110))]
    at = torch.tensor(sum(rows, []), device="cuda")
    cu, lens = ac.offsets(prompt), torch.tensor(prompt, dtype=torch.int32, device="cuda")
    o = attn.kda_attn_fwd(q[at], k[at], v[at], cu)
    ac.check("prompt", o, ref[at.cpu()], lim[at.cpu()])
    attn.kda_kv_write(k[at], v[at], cu, lens, c.table, c.k, c.v)
    rk, rv = attn.kda_kv_read(90, cu, lens, c.table, c.k, c.v)
    assert torch.equal(rk, k[at]) and torch.equal(rv, v[at])
    cu1 = ac.offsets([1, 1])
    for step in range(12):
        at = torch.tensor([70 + step, 110 + step], device="cuda")
        lens += 1
        attn.kda_kv_write(k[at], v[at], cu1, lens, c.table, c.k, c.v)
        o = attn.kda_attn_cache_fwd(q[at], cu1, lens, c.table, c.k, c.v)
        ac.check(f"token {step}", o, ref[at.cpu()], lim[at.cpu()])
    # a chain as a tree: 8 and 5 drafted tokens
    at = torch.tensor(list(range(82, 90)) + list(range(122, 127)), device="cuda")
    cu2 = ac.offsets([8, 5])
    lens += torch.tensor([8, 5], dtype=torch.int32, device="cuda")
    attn.kda_kv_write(k[at], v[at], cu2, lens, c.table, c.k, c.v)
    chain = [(2 << i) - 1 for i in range(8)] + [(2 << i) - 1 for i in range(5)]
    o = attn.kda_attn_cache_fwd(q[at], cu2, lens, c.table, c.k, c.v, tree_mask=ac.mask_tensor(chain))
    ac.check("chain of drafts", o, ref[at.cpu()], lim[at.cpu()])


def test_refused_on_the_gpu():
    c = filled(31, [20], 2, 64, 64, 16, "e4m3", max_pages=40)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    cu = ac.offsets([1])
    with pytest.raises(ValueError):
        attn.kda_attn_cache_fwd(q, cu, *c.args())                                             # no exponents
    with pytest.raises(ValueError):
        attn.kda_attn_cache_fwd(torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda"), cu, *c.args(), **c.exps())
    with pytest.raises(ValueError):
        attn.kda_attn_cache_fwd(q, cu, *c.args(), **c.exps(), tree_mask=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(RuntimeError):
        attn.kda_attn_cache_fwd(q.float(), cu, *c.args(), **c.exps())
    with pytest.raises(RuntimeError):
        attn.kda_attn_cache_fwd(torch.zeros((1, 3, 64), dtype=torch.bfloat16, device="cuda"), cu, *c.args(), **c.exps())
    with pytest.raises(RuntimeError):
        attn.kda_attn_cache_fwd(q, cu, *c.args(), **c.exps(), workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
