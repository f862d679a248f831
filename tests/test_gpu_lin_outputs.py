"""bf16 outputs of kda_lin_chunk_fwd are rounded once: before that they are as right as fp32 outputs.

Scores and the state that q reads are held in two bf16 numbers, whatever the outputs' type, so an output is the
definition's to 2^-16 of each term beside the fp32 errors (tests/lin_common.py), rounded by half a step of bf16
(2^-8 of itself). One bf16 number would be off by 2^-8 of each term, which is seen where terms cancel."""

import pytest
import torch

from gated_delta_rule_10_amd import lin
from tests import lin_common as lc

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("lens,H,Hk", [([200, 65, 1, 0, 64], 4, 2), ([2500], 2, 1)])
@pytest.mark.parametrize("rate", [1e-3, 0.5])
def test_bf16_outputs_are_rounded_once(dk, dv, lens, H, Hk, rate):
    x = lc.Inputs(dk + 2 * dv + len(lens), lens, H, Hk, dk, dv, "bf16", rate=rate)
    o, s = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, scale=0.7)
    assert o.dtype == BF
    at = 0
    for n, (L, (ro, ao, rs, as_)) in enumerate(zip(lens, x.reference(x.s0, 0.7))):
        lc.check(f"o {n} ({L})", o[at:at + L], ro, ao, lc.e32(L, dk) + 2.0 ** -16, True)
        lc.check(f"state {n} ({L})", s[n], rs, as_, lc.e32(L, dk))
        at += L


def test_bf16_outputs_are_the_fp32_outputs_rounded():
    """The same sums in both forms: only the last step differs."""
    x = lc.Inputs(5, [300, 40], 3, 3, 128, 128, "bf16")
    half, _ = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
    full, _ = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0, out_dtype=torch.float32)
    assert torch.equal(half, full.to(BF))
