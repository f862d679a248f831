"""CPU tests of the linear-attention and beam-search entry points' C ABI and bindings: every symbol of
include/kda_lin.h and include/kda_beam.h is exported, and invalid arguments are refused on the host before any
HIP call."""

import os
import re

import pytest
import torch

from gated_delta_rule_10_amd import beam, kda, lin

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # a 16-byte aligned stand-in address; never dereferenced on the host
B = 0x20000
INVALID, UNSUPPORTED, WORKSPACE = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.LIB_PATH):
        pytest.skip("libkda.so not built")
    lin.load_library()
    return beam.load_library()


@pytest.mark.parametrize("header,wanted", [
    ("kda_lin.h", ["kda_lin_chunk_fwd", "kda_lin_chunk_fwd_workspace_size", "kda_lin_decode_step"]),
    ("kda_beam.h", ["kda_beam_select", "kda_beam_select_workspace_size", "kda_state_reorder"])])
def test_every_declared_function_is_exported_and_bound(lib, header, wanted):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(kda_[a-z_0-9]+)\s*\(", src))) == sorted(wanted)
    import gated_delta_rule_10_amd as g
    for n in wanted:
        assert hasattr(lib, n) and callable(getattr(g, n)) and n in g.__all__


def test_headers_are_c(tmp_path):
    import subprocess
    src = tmp_path / "c.c"
    src.write_text('#include "kda_lin.h"\n#include "kda_beam.h"\nint main(void) { return (int)sizeof(kda_status_t) == 0; }\n')
    try:
        subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__", "-I",
                               os.path.join(ROOT, "include"), "-isystem", "/opt/rocm/include", str(src)])
    except OSError:
        pytest.skip("no C compiler")


def _chunk(lib, **over):
    a = dict(q=A, k=A, v=A, g=A, cu=A, N=2, T=100, H=8, Hk=2, dk=128, dv=128, qs=256, ks=256, vs=1024, gs=8,
             din=kda.KDA_BF16, dout=kda.KDA_BF16, scale=1.0, s0=A, sT=A, slots=None, ns=0, o=A, ws=A, wsb=1 << 40)
    a.update(over)
    return lib.kda_lin_chunk_fwd(a["q"], a["k"], a["v"], a["g"], a["cu"], a["N"], a["T"], a["H"], a["Hk"], a["dk"], a["dv"],
                                 a["qs"], a["ks"], a["vs"], a["gs"], a["din"], a["dout"], a["scale"], a["s0"], a["sT"],
                                 a["slots"], a["ns"], a["o"], a["ws"], a["wsb"], None)


def _step(lib, **over):
    a = dict(q=A, k=A, v=A, g=A, cache=A, idx=None, o=A, B=3, H=8, Hk=2, dk=128, dv=128, qs=256, ks=256, vs=1024, gs=8,
             ns=3, din=kda.KDA_BF16, dout=kda.KDA_BF16, scale=1.0)
    a.update(over)
    return lib.kda_lin_decode_step(a["q"], a["k"], a["v"], a["g"], a["cache"], a["idx"], a["o"], a["B"], a["H"], a["Hk"],
                                   a["dk"], a["dv"], a["qs"], a["ks"], a["vs"], a["gs"], a["ns"], a["din"], a["dout"],
                                   a["scale"], None)


LAYERS = [
    (dict(q=None), INVALID), (dict(k=A + 8), INVALID), (dict(v=None), INVALID), (dict(g=A + 4), INVALID),
    (dict(o=None), INVALID), (dict(H=0), INVALID), (dict(Hk=0), INVALID), (dict(Hk=3), INVALID),
    (dict(qs=248), INVALID), (dict(ks=260), INVALID), (dict(vs=1016), INVALID), (dict(vs=2 ** 24 + 8), INVALID),
    (dict(gs=7), INVALID), (dict(gs=-8), INVALID), (dict(gs=2 ** 24 + 1), INVALID),
    (dict(din=7), INVALID), (dict(dout=7), INVALID), (dict(din=kda.KDA_F32, dout=kda.KDA_BF16), UNSUPPORTED),
    (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
]


@pytest.mark.parametrize("over,status", LAYERS + [
    (dict(N=0), INVALID), (dict(T=-1), INVALID), (dict(T=2 ** 31 - 1024, H=1, Hk=1), INVALID),
    (dict(T=2 ** 28), INVALID),                                                  # T H past int32
    (dict(N=2 ** 19), INVALID),                                                  # launches of 2^32 threads
    (dict(cu=None), INVALID), (dict(cu=A + 4), INVALID), (dict(s0=A + 4), INVALID), (dict(sT=A + 8), INVALID),
    (dict(slots=A), INVALID), (dict(slots=A + 4, ns=2), INVALID), (dict(ws=A + 8), INVALID),
])
def test_lin_chunk_fwd_rejects(lib, over, status):
    assert _chunk(lib, **over) == status


@pytest.mark.parametrize("over,status", LAYERS + [
    (dict(B=0), INVALID), (dict(B=2 ** 19, ns=2 ** 19), INVALID), (dict(cache=None), INVALID), (dict(cache=A + 4), INVALID),
    (dict(idx=A + 4), INVALID), (dict(ns=0), INVALID), (dict(ns=2), INVALID),    # three tokens, two slots, no indices
])
def test_lin_decode_step_rejects(lib, over, status):
    assert _step(lib, **over) == status


def test_workspace_of_long_sequences(lib):
    ws = lin.kda_lin_chunk_fwd_workspace_size
    for dt in (torch.bfloat16, torch.float32):
        assert ws(1, 65, 8, 128, 128, dt) == 0
        assert ws(0, 65, 8, 128, 128, dt) == ws(1, 100000, 8, 96, 128, dt) == ws(1, -1, 8, 128, 128, dt) == 0
        need = ws(1, 100000, 8, 128, 128, dt)
        if need:
            code = kda.KDA_BF16 if dt == torch.bfloat16 else kda.KDA_F32
            over = dict(N=1, T=100000, din=code, dout=code)
            assert _chunk(lib, ws=None, **over) == _chunk(lib, wsb=need - 1, **over) == WORKSPACE


def _select(lib, **over):
    a = dict(x=A, stride=1000, scores=A, done=None, tok=0, N=2, W=4, V=1000, K=8, dt=kda.KDA_F32, os=A, op=A, ot=A, ws=A,
             wsb=1 << 40)
    a.update(over)
    return lib.kda_beam_select(a["x"], a["stride"], a["scores"], a["done"], a["tok"], a["N"], a["W"], a["V"], a["K"], a["dt"],
                               a["os"], a["op"], a["ot"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("over,status", [
    (dict(x=None), INVALID), (dict(x=A + 2), INVALID), (dict(scores=None), INVALID), (dict(os=None), INVALID),
    (dict(op=A + 4), INVALID), (dict(ot=None), INVALID), (dict(done=A + 1), INVALID), (dict(ws=A + 8), INVALID),
    (dict(stride=999), INVALID), (dict(stride=2 ** 31 + 1), INVALID), (dict(dt=7), INVALID),
    (dict(N=0), INVALID), (dict(W=0), INVALID), (dict(W=65), INVALID), (dict(V=0), INVALID), (dict(K=0), INVALID),
    (dict(K=65), INVALID), (dict(N=2 ** 18), INVALID), (dict(V=2 ** 29, stride=2 ** 29), INVALID),
    (dict(done=A, tok=-1), INVALID), (dict(done=A, tok=1000), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE),
])
def test_beam_select_rejects(lib, over, status):
    assert _select(lib, **over) == status


def _reorder(lib, **over):
    a = dict(states=A, stride=1 << 20, layers=2, ns=16, bytes=65536, slots=A, parent=A, out=B, N=2, W=4)
    a.update(over)
    return lib.kda_state_reorder(a["states"], a["stride"], a["layers"], a["ns"], a["bytes"], a["slots"], a["parent"], a["out"],
                                 a["N"], a["W"], None)


@pytest.mark.parametrize("over", [
    dict(states=None), dict(states=A + 8), dict(slots=None), dict(parent=A + 4), dict(out=None), dict(out=A),  # out is slots
    dict(N=0), dict(W=0), dict(W=65), dict(N=2 ** 18), dict(layers=0), dict(ns=0), dict(N=2 ** 17, layers=32),
    dict(bytes=0), dict(bytes=24), dict(bytes=2 ** 37), dict(stride=(1 << 20) - 16), dict(stride=(1 << 20) + 8),
])
def test_state_reorder_rejects(lib, over):
    assert _reorder(lib, **over) == INVALID


def test_select_workspace(lib):
    ws = beam.kda_beam_select_workspace_size
    assert ws(1, 4, 1000, 8) > 0
    assert ws(0, 4, 1000, 8) == ws(1, 65, 1000, 8) == ws(1, 4, 0, 8) == ws(1, 4, 1000, 65) == 0


def test_bindings_refuse_host_tensors_and_wrong_layouts(lib):
    x, cu = torch.zeros((4, 2, 64)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        lin.kda_lin_chunk_fwd(x, x, x, x[:, :, 0], cu)
    with pytest.raises(ValueError, match="GPU"):
        lin.kda_lin_decode_step(x, x, x, x[:, :, 0], x[None])
    with pytest.raises(ValueError, match="GPU"):
        beam.kda_beam_select(x, x[:, :, 0], 2)
    with pytest.raises(ValueError, match="GPU"):
        beam.kda_state_reorder(x, cu[None], cu[None])
    cpu = torch.device("cpu")
    assert lin._decay(torch.zeros(4, 2), 4, 2, cpu) == 2
    assert lin._decay(torch.zeros(4, 6)[:, 2:4], 4, 2, cpu) == 6
    assert lin._decay(torch.zeros(1, 6)[:, 2:4], 1, 2, cpu) == 2
    assert lin._decay(torch.zeros(2), 4, 2, cpu) == 0
    for bad in (torch.zeros(2, 4).t(), torch.zeros(4, 3), torch.zeros(3), torch.zeros(4, 2).double(), torch.zeros(4)[::2]):
        with pytest.raises(ValueError):
            lin._decay(bad, 4, 2, cpu)


def test_outputs_in_the_place_of_inputs_are_refused(lib):
    assert _select(lib, os=A) == INVALID               # K is not W: another request's scores
    assert _reorder(lib, slots=B, parent=A, out=A) == INVALID
