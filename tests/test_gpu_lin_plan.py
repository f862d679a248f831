"""Which batches kda_lin_chunk_fwd cuts into segments: one long sequence among short ones is, also where sequences and
heads do not fill the card (uncut, a few workgroups would walk it chunk by chunk while the others stand empty)."""

import pytest
import torch

from gated_delta_rule_10_amd import lin
from tests import lin_common as lc

pytestmark = pytest.mark.gpu
ws = lin.kda_lin_chunk_fwd_workspace_size


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,T,H", [(32, 40930, 4), (64, 11150, 2), (16, 20450, 8), (100, 60000, 1)])
def test_skewed_batches_are_cut(dt, N, T, H):
    assert ws(N, T, H, 128, 128, dt) > 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("where", [0, 9, 23])
def test_one_long_sequence_on_an_empty_card(dt, where):
    lens = [30] * 23
    lens.insert(where, 4000)
    x = lc.Inputs(where, lens, 4, 2, 128, 128, dt, rate=0.05)
    assert ws(len(lens), x.T, 4, 128, 128, x.q.dtype) > 0
    o, s = lin.kda_lin_chunk_fwd(*x.args(), initial_state=x.s0)
    x.check(o, s, x.s0, 1.0)
