"""The attention entry points at values and layouts where one kernel form could differ from the others,
against the plain 64-bit form (tests/attn_common.py)."""

import pytest
import torch

from gated_delta_rule_10_amd import attn
from tests import attn_common as ac
from tests.test_gpu_attn_cache import call, run

pytestmark = pytest.mark.gpu

# 10 query heads share a kv head: two tokens and more are more than 16 rows for it, which take tiles of 128 rows
H, HK = 20, 2


def held(seed, lens, k, v, page, kv):
    """A cache that holds k, v [sum(lens), HK, d] for sequences of `lens` tokens."""
    c = ac.Cache(lens, k.shape[1], k.shape[2], v.shape[2], page, kv, seed=seed)
    at = 0
    for n, L in enumerate(lens):
        c.put(n, k[at:at + L].bfloat16().float(), v[at:at + L].bfloat16().float())
        at += L
    return c


def compare(name, q, c, new, scale, masks=None):
    ref, lim = ac.cache_reference(q, c, new, masks, scale, True, True)
    ac.check(name, call(q, new, c, masks, scale, "bf16"), ref, lim)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
@pytest.mark.parametrize("ctx", [400, 1700])
def test_scales_with_many_rows(kv, scale, ctx):
    run(40, [5, 3], [ctx, 250], H, HK, 64, 64, 64, "bf16", kv, scale=scale)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("d", [64, 128])
def test_rising_and_falling_scores_with_many_rows(kv, sign, d):
    """Scores that grow (fall) along the cache by far more than the fp32 exponent reaches."""
    L, ctx = 5, 700
    k, v = torch.zeros(ctx + L, HK, d), ac.normal(41, ctx + L, HK, d)
    k[:, :, 0] = sign * 1.5 * torch.arange(ctx + L)[:, None]
    q = torch.zeros(L, H, d)
    q[:, :, 0] = 1
    compare(f"{sign} {kv}", q.bfloat16().cuda(), held(41, [ctx + L], k, v, 64, kv), [L], 1.0)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("d,dv", [(64, 64), (128, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("ctx", [400, 1700])
def test_scores_whose_sums_cancel_late(kv, sign, d, dv, ctx):
    """All but the last 16 channels add up to hundreds, which the last 16 take away again: a maximum of sums
    that are not complete would be off by more than the exponent's reach."""
    L, big = 3, 6.0
    k, v = 0.5 * ac.normal(42, ctx + L, HK, d), ac.normal(43, ctx + L, HK, dv)
    k[:, :, :d - 16] += sign * big
    k[:, :, d - 16:] -= sign * big * (d - 16) / 16
    q = (1 + 0.25 * ac.normal(44, L, H, d)).bfloat16().cuda()
    compare(f"{sign} {kv} {d}", q, held(42, [ctx + L], k, v, 64, kv), [L], 1.0)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,T", [(4, 2, 300), (128, 32, 600)])
def test_scores_whose_sums_cancel_late_in_prompts(sign, d, heads, kv_heads, T):
    big = 6.0
    k, v = 0.5 * ac.normal(45, T, kv_heads, d), ac.normal(46, T, kv_heads, d)
    k[:, :, :d - 16] += sign * big
    k[:, :, d - 16:] -= sign * big * (d - 16) / 16
    q, k, v = (x.bfloat16().cuda() for x in (1 + 0.25 * ac.normal(47, T, heads, d), k, v))
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=1.0)
    h = torch.tensor([0, heads - 1], device="cuda")
    g = h // (heads // kv_heads)
    ref, lim = ac.prompt_reference(q[:, h].contiguous(), k[:, g].contiguous(), v[:, g].contiguous(), [T], 1.0, True, True)
    ac.check(f"{sign} {d}", got[:, h], ref, lim)


def check_values(name, got, ref, lim):
    """ac.check, and every infinity and NaN in its place."""
    g = got.double().cpu()
    odd = ~torch.isfinite(ref)
    assert torch.equal(torch.nan_to_num(g[odd], nan=1.0), torch.nan_to_num(ref[odd], nan=1.0)), f"{name}: other infinities or NaN"
    ac.check(name, got, ref, lim)


def infinities(v, at, other):
    """Infinities of both signs in some channels of token `at` of v [T, heads, d], and of token `other`."""
    inf = float("inf")
    v[at, :, 3], v[at, :, 20], v[at, 0, 41:44] = inf, -inf, inf
    v[other, :, 20], v[other, 1, 50] = inf, -inf      # channel 20: NaN for the rows that see both


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [4, 20])
@pytest.mark.parametrize("ctx", [100, 1500])
def test_infinite_values_that_a_row_sees(dt, heads, ctx):
    """Infinities in v reach the rows that see them as infinities, early in the cache and among the new tokens,
    with 4 and 20 rows for a kv head."""
    bf, dtype = dt == "bf16", torch.bfloat16 if dt == "bf16" else torch.float32
    q = ac.normal(50, 2, heads, 64).to(dtype).cuda()
    for at, other in ((0, ctx + 1), (37, 5), (ctx // 2, ctx // 2 + 20), (ctx - 1, 2), (ctx + 1, 64)):
        k, v = ac.normal(51, ctx + 2, 2, 64), ac.normal(52, ctx + 2, 2, 64)
        infinities(v, at, other)
        c = held(53, [ctx + 2], k, v, 64, dt)
        ref, lim = ac.cache_reference(q, c, [2], None, 0.125, bf, bf)
        check_values(f"{dt} {ctx} {at}", call(q, [2], c, None, 0.125, dt), ref, lim)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads,T", [(4, 2, 300), (128, 32, 600)])
@pytest.mark.parametrize("at,other", [(0, 299), (130, 30), (200, 199)])
def test_infinite_values_that_a_row_sees_in_prompts(dt, heads, kv_heads, T, at, other):
    bf, dtype = dt == "bf16", torch.bfloat16 if dt == "bf16" else torch.float32
    v = ac.normal(56, T, kv_heads, 64)
    infinities(v, at, other)
    q, k, v = (x.to(dtype).cuda() for x in (ac.normal(54, T, heads, 64), ac.normal(55, T, kv_heads, 64), v))
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=0.125)
    h = torch.tensor([0, heads // kv_heads, heads - 1], device="cuda")
    g = h // (heads // kv_heads)
    ref, lim = ac.prompt_reference(q[:, h].contiguous(), k[:, g].contiguous(), v[:, g].contiguous(), [T], 0.125, bf, bf)
    check_values(f"{dt} {at}", got[:, h], ref, lim)


@pytest.mark.parametrize("dt,kv", [("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
@pytest.mark.parametrize("heads", [4, 20])
@pytest.mark.parametrize("ctx", [6, 300, 1700])
@pytest.mark.parametrize("size", ["large", "small"])
def test_values_at_the_ends_of_the_range(dt, kv, heads, ctx, size):
    """Values of one sign just below 2^120 / tokens, and about 2^-100, under scores that rise slowly, so that
    weights reach 2^8 of the reference that they are taken from."""
    bf, T = dt == "bf16", ctx + 2
    f = 2.0 ** 119 / T if size == "large" else 2.0 ** -100
    k, v = 0.1 * ac.normal(60, T, 2, 64), f * (1 + 0.5 * torch.rand(T, 2, 64, generator=torch.Generator().manual_seed(60)))
    k[:, :, 0] = 0.011 * torch.arange(T)[:, None]
    q = 0.1 * ac.normal(61, 2, heads, 64)
    q[:, :, 0] = 1
    c = ac.Cache([T], 2, 64, 64, 64, kv, seed=62)
    c.put(0, k, v)
    q = q.to(torch.bfloat16 if bf else torch.float32).cuda()
    ref, lim = ac.cache_reference(q, c, [2], None, 1.0, bf, bf)
    assert torch.isfinite(ref).all()
    ac.check(f"{size} {dt}/{kv} {heads} {ctx}", call(q, [2], c, None, 1.0, dt), ref, lim)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads,T", [(4, 2, 300), (128, 32, 600)])
@pytest.mark.parametrize("size", ["large", "small"])
def test_values_at_the_ends_of_the_range_in_prompts(dt, heads, kv_heads, T, size):
    bf, dtype = dt == "bf16", torch.bfloat16 if dt == "bf16" else torch.float32
    f = 2.0 ** 119 / T if size == "large" else 2.0 ** -100
    k, v = 0.1 * ac.normal(63, T, kv_heads, 64), f * (1 + 0.5 * torch.rand(T, kv_heads, 64, generator=torch.Generator().manual_seed(63)))
    k[:, :, 0] = 0.03 * torch.arange(T)[:, None]
    q = 0.1 * ac.normal(64, T, heads, 64)
    q[:, :, 0] = 1
    q, k, v = (x.to(dtype).cuda() for x in (q, k, v))
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=1.0)
    h = torch.tensor([0, heads - 1], device="cuda")
    g = h // (heads // kv_heads)
    ref, lim = ac.prompt_reference(q[:, h].contiguous(), k[:, g].contiguous(), v[:, g].contiguous(), [T], 1.0, bf, bf)
    ac.check(f"{size} {dt}", got[:, h], ref, lim)


def infinite_keys(T, kv_heads, heads, seed, which):
    """q, k, v where the tokens of `which` have a score of -infinity for all queries."""
    q, k, v = (ac.normal(seed + i, n, h, 64) for i, (n, h) in enumerate(((T, heads), (T, kv_heads), (T, kv_heads))))
    q[:, :, 0] = 1 + q[:, :, 0].abs()
    k[which, :, 0] = -float("inf")
    return q, k, v


def expected(q, k, v, sees, scale, bf):
    """A head's (o, bound): tokens with a score of -infinity weigh nothing; NaN where there is no other."""
    q, k, v = q.cpu(), k.cpu(), v.cpu()
    there = torch.isfinite(k).all(1)
    o = ac.attend(q, torch.nan_to_num(k, neginf=0.0), v, sees & there, scale)
    lim = ac.bound(*o, 64, bf, bf)
    return torch.where((sees.any(1) & ~(sees & there).any(1))[:, None], torch.nan, o[0]), lim


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [4, 20])
@pytest.mark.parametrize("ctx", [10, 100, 1500])
def test_scores_of_minus_infinity(dt, heads, ctx):
    """Some tokens weigh nothing; a row all of whose tokens do is NaN, one that sees no token is 0."""
    bf, dtype, T = dt == "bf16", torch.bfloat16 if dt == "bf16" else torch.float32, ctx + 3
    for name, which, ctx_, masks in (("some", slice(0, T - 5), ctx, None), ("all", slice(0, T), ctx, None),
                                     ("the new ones", slice(ctx, T), ctx, None), ("no context", slice(0, 3), 0, [0, 2, 6])):
        q, k, v = infinite_keys(ctx_ + 3, 2, heads, 70, which)
        q = q[-3:].to(dtype).cuda()
        c = held(73, [ctx_ + 3], k, v, 64, dt)
        got = call(q, [3], c, masks, 0.125, dt)
        kk, vv = c.values(0, ctx_ + 3)
        sees = torch.ones(3, ctx_ + 3, dtype=torch.bool).tril(ctx_)
        if masks:
            sees = torch.tensor([[bool(m >> b & 1) for b in range(3)] for m in masks])
        for h in range(heads):
            g = h // (heads // 2)
            check_values(f"{name} {dt} {ctx}", got[:, h], *expected(q[:, h], kk[:, g], vv[:, g], sees, 0.125, bf))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads,T", [(4, 2, 300), (128, 32, 600)])
def test_scores_of_minus_infinity_in_prompts(dt, heads, kv_heads, T):
    """The first 150 tokens: their rows are NaN, later ones as if they were not there."""
    bf, dtype = dt == "bf16", torch.bfloat16 if dt == "bf16" else torch.float32
    q, k, v = (x.to(dtype).cuda() for x in infinite_keys(T, kv_heads, heads, 74, slice(0, 150)))
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=0.125)
    for h in (0, heads - 1):
        g = h // (heads // kv_heads)
        check_values(dt, got[:, h], *expected(q[:, h], k[:, g], v[:, g], torch.ones(T, T, dtype=torch.bool).tril(), 0.125, bf))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_scores_times_a_scale_of_zero(dt, sign):
    """0 times infinity: NaN in the rows that see the token, whatever the form, and nowhere else."""
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    for heads, kv_heads, T, at in ((4, 2, 300, 200), (128, 32, 600, 550)):
        q, k, v = infinite_keys(T, kv_heads, heads, 77, slice(at, at + 1))
        q, k, v = (x.to(dtype).cuda() for x in (q, sign * k, v))
        got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=0.0)
        assert torch.isfinite(got[:at]).all() and got[at:].isnan().all()
    for heads in (4, 20):
        for ctx, at in ((100, 30), (100, 101), (1500, 40)):
            q, k, v = infinite_keys(ctx + 3, 2, heads, 80, slice(at, at + 1))
            got = call(q[-3:].to(dtype).cuda(), [3], held(83, [ctx + 3], sign * k, v, 64, dt), None, 0.0, dt)
            sees = max(at - ctx, 0)
            assert torch.isfinite(got[:sees]).all() and got[sees:].isnan().all()


def wide(T, heads, kv_heads, dtype):
    """q, k, v [T, heads, 64] as parts of rows of 2^24 elements, the longest allowed: the last lie past 2^31."""
    step = 2 ** 24
    x = torch.empty(T * step, dtype=dtype, device="cuda")
    at, out = 0, []
    for i, h in enumerate((heads, kv_heads, kv_heads)):
        y = x.as_strided((T, h, 64), (step, 64, 1), at)
        y.copy_(ac.normal(90 + i, T, h, 64))
        out.append(y)
        at += h * 64
    assert (T - 1) * step > 2 ** 31
    return out


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,kv_heads", [(4, 2), (512, 128)])
def test_rows_past_32_bits(dt, heads, kv_heads):
    """Prompts (both tile forms), cache writes and cache attention of tokens whose offsets pass 2^31 elements."""
    T, bf = 200, dt == "bf16"
    q, k, v = wide(T, heads, kv_heads, torch.bfloat16 if bf else torch.float32)
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=0.125)
    for h in (0, heads - 1):
        g = h // (heads // kv_heads)
        ref, lim = ac.prompt_reference(q[:, h:h + 1].contiguous(), k[:, g:g + 1].contiguous(), v[:, g:g + 1].contiguous(), [T],
                                       0.125, bf, bf)
        ac.check(f"prompt {dt} head {h}", got[:, h:h + 1], ref, lim)
    if heads > 4:
        return
    c = ac.Cache([T], kv_heads, 64, 64, 64, dt)
    attn.kda_kv_write(k, v, ac.offsets([T]), *c.args())
    held_k, held_v = c.values(0, T)
    assert torch.equal(held_k, k.double().cpu()) and torch.equal(held_v, v.double().cpu())
    # the whole sequence as new tokens: what the prompt gives, from rows of the same width
    got = attn.kda_attn_cache_fwd(q, ac.offsets([T]), *c.args(), scale=0.125)
    ref, lim = ac.prompt_reference(q.contiguous(), k.contiguous(), v.contiguous(), [T], 0.125, bf, bf)
    ac.check(f"over the cache {dt}", got, ref, lim)


@pytest.mark.parametrize("dt,T,heads", [("bf16", 20000, 4), ("bf16", 9001, 32), ("f32", 6000, 4)])
def test_long_prompts(dt, T, heads):
    """Rows throughout one long prompt (the larger one's tiles are 256 rows), some at tiles' edges."""
    bf, dtype = dt == "bf16", torch.bfloat16 if dt == "bf16" else torch.float32
    q, k, v = (ac.normal(100 + i, T, h, 64).to(dtype).cuda() for i, h in enumerate((heads, heads // 4, heads // 4)))
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([T]), scale=0.125)
    rows = torch.tensor([0, 1, 63, 64, 1023, T // 2, T // 2 + 1, T - 65, T - 2, T - 1])
    sees = torch.arange(T)[None] <= rows[:, None]
    for h in (0, heads - 1):
        r = ac.attend(q[rows.cuda(), h].cpu(), k[:, h // 4].cpu(), v[:, h // 4].cpu(), sees, 0.125)
        ac.check(f"{dt} {T} head {h}", got[rows.cuda(), h], r[0], ac.bound(*r, 64, bf, bf))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,ctx", [(700, 0), (700, 1500)])
def test_chunks_of_prompts_over_the_cache(kv, new, ctx):
    """A prompt's chunk of many new tokens, beside a single token of another sequence."""
    T = ctx + new
    c = held(110, [T, 40], ac.normal(111, T + 40, 2, 64), ac.normal(112, T + 40, 2, 64), 64, kv)
    q = ac.normal(113, new + 1, 8, 64).bfloat16().cuda()
    got = call(q, [new, 1], c, None, 0.125, "bf16")
    rows = torch.tensor([0, 1, 31, 32, 63, 64, 300, new - 2, new - 1])
    for n, at, count, total in ((0, rows, new, T), (1, torch.tensor([new]), 1, 40)):
        k, v = c.values(n, total)
        sees = torch.arange(total)[None] <= (at - (0 if n == 0 else new))[:, None] + total - count
        for h in (0, 7):
            r = ac.attend(q[at.cuda(), h].cpu(), k[:, h // 4], v[:, h // 4], sees, 0.125)
            ac.check(f"{kv} sequence {n} head {h}", got[at.cuda(), h], r[0], ac.bound(*r, 64, True, True))
