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
