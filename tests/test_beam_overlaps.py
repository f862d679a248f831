"""CPU tests: outputs of the beam-search entry points that lie partly on inputs that other workgroups still read, or on
each other, are refused on the host (A is a stand-in address; nothing is dereferenced)."""

import os

import pytest

from gated_delta_rule_10_amd import beam, kda

A, FAR = 0x100000, 0x100000 + (1 << 20)
INVALID = kda.KDA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        pytest.skip("libkda.so not built")
    return beam.load_library()


# N = 6 requests of W = 8 beams: slots, parents and scores are 192 bytes each
@pytest.mark.parametrize("out", [A, A + 16, A + 176, A - 16, A - 176])
@pytest.mark.parametrize("which", ["slots", "parent"])
def test_reorder(lib, out, which):
    a = dict(slots=FAR, parent=FAR + 4096)
    a[which] = A
    assert lib.kda_state_reorder(2 * FAR, 1 << 20, 1, 64, 4096, a["slots"], a["parent"], out, 6, 8, None) == INVALID


def select(lib, K=8, scores=FAR, done=None, s=2 * FAR, p=3 * FAR, t=4 * FAR):
    return lib.kda_beam_select(5 * FAR, 1000, scores, done, 0, 6, 8, 1000, K, kda.KDA_F32, s, p, t, 6 * FAR, 1 << 40, None)


@pytest.mark.parametrize("by", [-176, -16, 16, 176])
@pytest.mark.parametrize("out", ["s", "p", "t"])
def test_select_over_scores(lib, out, by):
    assert select(lib, scores=A, **{out: A + by}) == INVALID


def test_select_over_the_same_scores(lib):
    assert select(lib, K=4, scores=A, s=A) == INVALID       # in place only where requests keep their width
    assert select(lib, scores=A, p=A) == select(lib, scores=A, t=A) == INVALID


@pytest.mark.parametrize("out", ["s", "p", "t"])
@pytest.mark.parametrize("by", [-176, 0, 32])
def test_select_over_done(lib, out, by):
    assert select(lib, done=A, **{out: A + by}) == INVALID


@pytest.mark.parametrize("a,b", [("s", "p"), ("s", "t"), ("p", "t")])
@pytest.mark.parametrize("by", [0, 16, 176, -176])
def test_select_outputs_over_each_other(lib, a, b, by):
    assert select(lib, **{a: A, b: A + by}) == INVALID
