"""CPU tests: kda_lin_chunk_fwd's final states in the place of the initial ones are the same array or another, not one
that lies partly on it (a sequence's final state would be another's initial one, still to be read); A is a stand-in
address, nothing is dereferenced."""

import os

import pytest

from gated_delta_rule_10_amd import kda, lin

A, FAR, STATE = 1 << 30, 1 << 40, 8 * 64 * 64 * 4  # bytes of a sequence's states


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        pytest.skip("libkda.so not built")
    return lin.load_library()


def call(lib, s0, sT, slots=None, ns=0):
    return lib.kda_lin_chunk_fwd(FAR, FAR, FAR, FAR, FAR, 4, 100, 8, 8, 64, 64, 512, 512, 512, 8, kda.KDA_F32, kda.KDA_F32,
                                 1.0, s0, sT, slots, ns, FAR, FAR, 1 << 30, None)


@pytest.mark.parametrize("by", [16, STATE, 3 * STATE, 4 * STATE - 16])
@pytest.mark.parametrize("sign", [1, -1])
def test_states_partly_in_place(lib, by, sign):
    assert call(lib, A, A + sign * by) == kda.KDA_ERR_INVALID_ARG


def test_slots_partly_in_place(lib):
    assert call(lib, A, A + 8 * STATE, FAR, 9) == kda.KDA_ERR_INVALID_ARG  # caches of nine slots, one of them shared
