"""kda_attn_fwd against the plain 64-bit form (tests/attn_common.py)."""

import pytest
import torch

from gated_delta_rule_10_amd import attn
from tests import attn_common as ac

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(seed, T, H, Hk, dk, dv, dt):
    return tuple(ac.normal(seed + i, T, h, d).to(DT[dt]).cuda() for i, (h, d) in enumerate(((H, dk), (Hk, dk), (Hk, dv))))


def run(q, k, v, lens, scale, dt, out=None, **kw):
    out = out or dt
    got = attn.kda_attn_fwd(q, k, v, ac.offsets(lens), scale=scale, out_dtype=DT[out], **kw)
    ref, lim = ac.prompt_reference(q, k, v, lens, scale, dt == "bf16", out == "bf16")
    ac.check(f"o {dt}->{out} {lens}", got[:sum(lens)], ref[:sum(lens)], lim[:sum(lens)])
    return got


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
def test_dims(dt, dk, dv):
    lens = [65, 1, 0, 200]
    run(*make(1, sum(lens), 4, 2, dk, dv, dt), lens, dk ** -0.5, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (7, 1), (12, 4), (16, 2), (33, 1)])
def test_heads(dt, H, Hk):
    lens = [37, 130]
    run(*make(2, sum(lens), H, Hk, 64, 64, dt), lens, 0.125, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [32], [33], [63], [64], [127], [128], [129], [255], [257],
                                  [1] * 70, [0, 0, 5, 0], [3, 64, 0, 128, 1, 300]])
def test_lengths(dt, lens):
    run(*make(3, sum(lens), 4, 1, 128, 128, dt), lens, 0.09, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_longer(dt):
    lens = [700, 1111]
    run(*make(4, sum(lens), 2, 1, 128, 128, dt), lens, 0.09, dt)


def test_fp32_out_from_bf16():
    lens = [150, 33]
    run(*make(5, sum(lens), 8, 2, 128, 128, "bf16"), lens, 0.09, "bf16", out="f32")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
def test_scales(scale):
    """Scale 4 makes scores of hundreds: one weight takes all, and the running maximum moves often."""
    run(*make(6, 200, 2, 1, 64, 64, "f32"), [200], scale, "f32")
    run(*make(6, 200, 2, 1, 64, 64, "bf16"), [200], scale, "bf16")


def test_rising_and_falling_scores():
    """Scores that grow (fall) along the sequence by far more than the fp32 exponent reaches."""
    for sign in (1, -1):
        q, k, v = make(7, 300, 1, 1, 64, 64, "f32")
        q[:], k[:] = 0, 0
        q[:, :, 0] = 1
        k[:, 0, 0] = sign * torch.arange(300).cuda() * 1.5
        run(q, k, v, [300], 1.0, "f32")
        run(q.bfloat16(), k.bfloat16(), v.bfloat16(), [300], 1.0, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_parts_of_wider_rows(dt):
    """q, k, v as parts of one projection's rows, and a length of one with any stride."""
    H, Hk, d = 6, 2, 64
    x = ac.normal(8, 90, H + 2 * Hk, d).to(DT[dt]).cuda()
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    assert not k.is_contiguous()
    run(q, k, v, [50, 40], 0.125, dt)
    run(q[5:6], k[5:6], v[5:6], [1], 0.125, dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_tokens_not_seen_have_no_influence(dt, bad):
    """Infinities and NaN in k and v of the last token of the first sequence: only that token's
    row changes; the rows before it and the sequence behind it are bit for bit the same."""
    lens = [100, 60]
    q, k, v = make(9, 160, 4, 2, 128, 128, dt)
    clean = run(q, k, v, lens, 0.09, dt)
    for spoil in (lambda: k[99].fill_(bad), lambda: v[99].fill_(bad)):
        spoil()
        got = attn.kda_attn_fwd(q, k, v, ac.offsets(lens), scale=0.09)
        torch.cuda.synchronize()
        # a token's value is added alone where a value near it is not finite: another order of the sum
        ref, lim = ac.prompt_reference(q[:99], k[:99], v[:99], [99], 0.09, dt == "bf16", dt == "bf16")
        ac.check("rows before", got[:99], ref, lim)
        assert torch.equal(got[100:], clean[100:])
        assert not torch.isfinite(got[99]).any()


def test_nan_in_q_stays_in_its_row():
    q, k, v = make(10, 80, 4, 2, 64, 64, "bf16")
    clean = run(q, k, v, [80], 0.125, "bf16")
    q[40, 1] = float("nan")
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([80]), scale=0.125)
    assert torch.isnan(got[40, 1]).all()
    got[40, 1] = clean[40, 1]
    assert torch.equal(got, clean)


def test_rows_behind_the_last_sequence_stay():
    q, k, v = make(11, 50, 4, 2, 64, 64, "bf16")
    o = torch.full((50, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    k[30:], v[30:], q[30:] = float("nan"), float("nan"), float("nan")
    got = attn.kda_attn_fwd(q, k, v, ac.offsets([20, 10]), scale=0.125, o=o)
    ref, lim = ac.prompt_reference(q[:30], k[:30], v[:30], [20, 10], 0.125, True, True)
    ac.check("o", got[:30], ref, lim)
    assert (o[30:] == 7).all()


def test_same_call_same_bits_and_default_scale():
    q, k, v = make(12, 500, 8, 2, 128, 128, "bf16")
    a = attn.kda_attn_fwd(q, k, v, ac.offsets([500]))
    b = attn.kda_attn_fwd(q, k, v, ac.offsets([500]), scale=128 ** -0.5)
    assert torch.equal(a, b)


def test_offsets_that_break_the_rules_stay_inside():
    """Decreasing, negative and too large offsets are clamped: no access outside the arrays, and the
    sequences that they leave are right."""
    q, k, v = make(13, 40, 2, 1, 64, 64, "f32")
    cu = torch.tensor([-5, 20, 10, 1000], dtype=torch.int32, device="cuda")
    o = torch.zeros((40, 2, 64), device="cuda")
    attn.kda_attn_fwd(q, k, v, cu, scale=0.125, o=o)
    ref, lim = ac.prompt_reference(q[:20], k[:20], v[:20], [20], 0.125, False, False)
    torch.cuda.synchronize()
    ac.check("the first sequence", o[:10], ref[:10], lim[:10])


def test_refused_on_the_gpu():
    q, k, v = make(14, 8, 2, 1, 64, 64, "bf16")
    cu = ac.offsets([8])
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(q, k, v.float(), cu)
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(q, k[:7], v, cu)
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(q, k, v, cu.long())
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(q, k, v, cu, o=torch.empty((8, 2, 32), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        attn.kda_attn_fwd(q.half(), k.half(), v.half(), cu)
    with pytest.raises(ValueError):
        attn.kda_attn_fwd(q, k, v, cu.cpu())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_writes_nothing_outside(dt):
    q, k, v = make(15, 131, 4, 2, 64, 128, dt)
    size = 131 * 4 * 128 * q.element_size()
    buf = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    o = buf[4096:4096 + size].view(q.dtype).view(131, 4, 128)
    attn.kda_attn_fwd(q, k, v, ac.offsets([100, 31]), o=o)
    assert (buf[:4096] == 0xA5).all() and (buf[-4096:] == 0xA5).all()
    assert torch.equal(o, attn.kda_attn_fwd(q, k, v, ac.offsets([100, 31])))


# Calls with enough rows for all compute units take larger tiles of rows; the small calls above share a
# tile's keys between two halves of a workgroup. Some of the heads are compared.
FULL = 600  # tokens that fill the card at 128 heads


def some_heads(q, k, v, cut=None):
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    h = torch.tensor(sorted({0, 1, H // 2 + 1, H - 1}), device="cuda")
    return tuple(x[:cut].contiguous() for x in (q[:, h], k[:, h // G], v[:, h // G])) + (h,)


def run_some(q, k, v, lens, scale, out="bf16"):
    got = attn.kda_attn_fwd(q, k, v, ac.offsets(lens), scale=scale, out_dtype=DT[out])
    *ref, h = some_heads(q, k, v)
    o, lim = ac.prompt_reference(*ref, lens, scale, True, out == "bf16")
    ac.check(f"o bf16->{out} {lens}", got[:, h], o, lim)
    return got


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("H,Hk", [(128, 32), (128, 128), (129, 3)])
def test_full_card(dk, dv, H, Hk):
    lens = [65, 1, 0, 64, 63, 129, 17, FULL - 339]
    assert sum(lens) == FULL
    run_some(*make(21, FULL, H, Hk, dk, dv, "bf16"), lens, dk ** -0.5)


def test_full_card_one_sequence_fp32_out():
    run_some(*make(22, FULL, 128, 16, 128, 128, "bf16"), [FULL], 0.09, out="f32")


@pytest.mark.parametrize("T", [1030, 1537, 2047])
def test_few_long_sequences(T):
    run_some(*make(23, T, 32, 8, 128, 128, "bf16"), [T], 0.09)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_full_card_scales(scale):
    run_some(*make(24, FULL, 128, 16, 64, 64, "bf16"), [200, FULL - 200], scale)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_full_card_tokens_not_seen_have_no_influence(bad):
    lens = [100, 60, FULL - 160]
    q, k, v = make(25, FULL, 128, 32, 128, 128, "bf16")
    clean = run_some(q, k, v, lens, 0.09)
    for spoil in (lambda: k[99].fill_(bad), lambda: v[99].fill_(bad)):
        spoil()
        got = attn.kda_attn_fwd(q, k, v, ac.offsets(lens), scale=0.09)
        torch.cuda.synchronize()
        *ref, h = some_heads(q, k, v, 99)
        o, lim = ac.prompt_reference(*ref, [99], 0.09, True, True)
        ac.check("rows before", got[:99, h], o, lim)
        assert torch.equal(got[100:], clean[100:])
        assert not torch.isfinite(got[99]).any()


@pytest.mark.parametrize("H,Hk", [(4, 2), (128, 32)])
def test_parts_of_wider_rows_at_the_end_of_memory(H, Hk):
    """k and v end with the tensor's last token: nothing behind it is read (strided rows, all lengths of a
    last tile's beginning)."""
    T = FULL + 128 if H == 128 else 300
    x = ac.normal(26, T, H + 2 * Hk, 64).bfloat16().cuda()
    for end in (T, T - 63, T - 65, T - 128):
        y = x[:end]
        run_some(y[:, :H], y[:, H:H + Hk], y[:, H + Hk:], [end // 3, end - end // 3], 0.125)


def test_nan_meets_both_halves():
    """A NaN in one half's keys reaches every row that sees it, and no other."""
    q, k, v = make(27, 300, 4, 2, 128, 128, "bf16")
    clean = run(q, k, v, [300], 0.09, "bf16")
    for at in (10, 70, 130, 200):
        k2 = k.clone()
        k2[at] = float("nan")
        got = attn.kda_attn_fwd(q, k2, v, ac.offsets([300]), scale=0.09)
        torch.cuda.synchronize()
        ref, lim = ac.prompt_reference(q[:at], k[:at], v[:at], [at], 0.09, True, True)
        ac.check("rows before", got[:at], ref, lim)
        assert torch.isnan(got[at:]).all()
    assert torch.equal(attn.kda_attn_fwd(q, k, v, ac.offsets([300]), scale=0.09), clean)


@pytest.mark.parametrize("H,Hk,T", [(4, 2, 300), (128, 32, FULL)])
def test_another_stream_and_capture(H, Hk, T):
    """The same bits on another stream, and from a graph replayed between eager calls with other inputs."""
    cu = ac.offsets([T // 3, T - T // 3])
    sets = [make(31 + 3 * i, T, H, Hk, 128, 128, "bf16") for i in range(3)]
    eager = [attn.kda_attn_fwd(*s, cu, scale=0.09) for s in sets]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = attn.kda_attn_fwd(*sets[0], cu, scale=0.09, stream=stream)
    stream.synchronize()
    assert torch.equal(got, eager[0])
    held = tuple(x.clone() for x in sets[0])
    with torch.cuda.stream(stream):
        attn.kda_attn_fwd(*held, cu, scale=0.09)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = attn.kda_attn_fwd(*held, cu, scale=0.09)
        for i in (1, 2, 0, 1):
            for to, x in zip(held, sets[i]):
                to.copy_(x)
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, eager[i])
            assert torch.equal(attn.kda_attn_fwd(*sets[i], cu, scale=0.09), eager[i])
            stream.synchronize()
