"""The calls of include/elq_ops.h on a machine without a GPU: every declared
symbol is exported and bound, and bad arguments are refused on the host before
any launch (every case here fails validation or has no rows, so nothing is ever
enqueued)."""
import ctypes
import importlib.metadata
import os
import re

import pytest
import torch

from quantized_latent_moe_b200 import build, elq, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20         # stands for a device pointer; never read


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


def test_exports_and_binds_every_declared_symbol(L):
    src = open(os.path.join(ROOT, "include", "elq_ops.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(elq_[a-z0-9_]+)\s*\(", src))
    assert names == set(ops.SIGNATURES)
    for n in names:
        assert hasattr(L, n), n


def _args(defaults, over):
    a = dict(defaults)
    assert set(over) <= set(a)
    a.update(over)
    return list(a.values())


QUANT = dict(x=P, x_type=0, x_rows=4, cols=64, ldx=64, index=None, div=1, rows=4, q=P, ldq=64, scale=P, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), -1), (dict(x_rows=-1), -1), (dict(cols=0), -1), (dict(ldx=63), -1), (dict(div=0), -1),
    (dict(rows=5), -1), (dict(div=2), -1), (dict(x_type=24), -2), (dict(x_type=2), -2), (dict(ldq=48), -1),
    (dict(ldq=72), -3), (dict(q=None), -1), (dict(scale=None), -1), (dict(x=None), -1), (dict(x_rows=0, index=P), -1), (dict(cols=(1 << 30) + 1, ldx=1 << 31, ldq=1 << 31), -2),
    (dict(x=P + 8), -3), (dict(q=P + 8), -3), (dict(scale=P + 2), -3), (dict(index=P + 2), -3),
    (dict(rows=0), 0), (dict(rows=0, x=None, q=None, scale=None, x_rows=0), 0)])
def test_quantize_refusals(L, over, status):
    assert L.elq_quantize_i8(*_args(QUANT, over)) == status


SWIGLU = dict(gu=P, x_type=0, rows=4, I=64, ld=128, q=P, ldq=64, scale=P, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), -1), (dict(I=0), -1), (dict(ld=127), -1), (dict(x_type=24), -2), (dict(ldq=48), -1),
    (dict(ldq=72), -3), (dict(gu=None), -1), (dict(gu=P + 4), -3), (dict(rows=0, gu=None, q=None), 0)])
def test_swiglu_refusals(L, over, status):
    assert L.elq_swiglu_i8(*_args(SWIGLU, over)) == status


COMBINE = dict(o=P, o_type=0, o_rows=8, cols=64, ldo=64, pos=P, weights=P, T=4, k=2, q=P, ldq=64, scale=P, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), -1), (dict(o_rows=-1), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(ldo=60), -1), (dict(o_type=24), -2),
    (dict(pos=None), -1), (dict(weights=None), -1), (dict(o_rows=0), -1), (dict(o=None), -1), (dict(o=P + 4), -3), (dict(pos=P + 1), -3),
    (dict(ldq=65), -3), (dict(T=0, pos=None, weights=None), 0)])
def test_combine_refusals(L, over, status):
    assert L.elq_combine_i8(*_args(COMBINE, over)) == status


MATMUL = dict(x=P, ldx=64, sx=P, T=4, w=P, ldw=64, sw=P, bias=None, N=32, K=64, y=P, y_type=0, ldy=32, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), -1), (dict(T=(1 << 30) + 1), -2), (dict(N=(1 << 30) + 1, ldy=1 << 31), -2), (dict(N=0), -1), (dict(K=0), -1), (dict(ldx=48), -1), (dict(ldw=48), -1),
    (dict(ldy=31), -1), (dict(y_type=24), -2), (dict(K=65537, ldx=65552, ldw=65552), -2), (dict(ldx=72), -3),
    (dict(ldw=72), -3), (dict(x=None), -1), (dict(sx=None), -1), (dict(w=None), -1), (dict(sw=None), -1),
    (dict(y=None), -1), (dict(x=P + 8), -3), (dict(w=P + 8), -3), (dict(y=P + 8), -3), (dict(bias=P + 2), -3),
    (dict(T=0, x=None, sx=None, y=None), 0)])
def test_matmul_refusals(L, over, status):
    assert L.elq_i8_matmul(*_args(MATMUL, over)) == status


TIMEOUT = dict(x=P, ldx=64, sx=P, T=16, w=P, ldw=64, sw=P, N=32, K=64, y=P, ldy=32, stall=1, budget=1 << 24, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(stall=0), -1), (dict(stall=3), -1), (dict(budget=999_999), -1), (dict(budget=2_000_000_001), -1), (dict(T=4), -2),
    (dict(T=0), -2), (dict(x=None), -1), (dict(ldy=31), -1), (dict(ldx=72), -3), (dict(T=-1), -1)])
def test_timeout_refusals(L, over, status):
    assert L.elq_test_i8_matmul_timeout(*_args(TIMEOUT, over)) == status


GROUPED = dict(x=P, x_type=24, ldx=64, sx=P, M=4, w=P, ldw=64, w_stride=64 * 32, sw=P, E=8, N=32, K=64, offsets=P, y=P,
               y_type=0, ldy=32, stream=None)
G16 = dict(x_type=30, sx=None, sw=None)


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), -1), (dict(M=(1 << 30) + 1), -2), (dict(N=(1 << 30) + 1, ldy=1 << 31, w_stride=1 << 40), -2), (dict(E=0), -1), (dict(E=1025), -2), (dict(N=0), -1), (dict(K=0), -1),
    (dict(w_stride=64 * 32 - 16), -1), (dict(w_stride=64 * 32 + 8), -3), (dict(ldx=72), -3), (dict(ldy=31), -1),
    (dict(x_type=0), -2), (dict(y_type=24), -2), (dict(offsets=None), -1), (dict(sx=None), -1), (dict(sw=None), -1),
    (dict(x_type=30), -1), (dict(G16, y_type=1), -2), (dict(G16, ldx=68), -3), (dict(G16, K=65537, ldx=65544, ldw=65544, w_stride=65544 * 32), -2),
    (dict(offsets=P + 2), -3), (dict(y=P + 4), -3), (dict(M=0, x=None, offsets=None), 0)])
def test_grouped_refusals(L, over, status):
    assert L.elq_grouped_matmul(*_args(GROUPED, over)) == status


RMS = dict(x=P, x_type=0, T=4, cols=64, ldx=64, weight=None, eps=1e-6, n=2 * P, n_type=0, ldn=64, scale=None, stream=None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), -1), (dict(cols=0), -1), (dict(cols=(1 << 30) + 1, ldx=1 << 31, ldn=1 << 31), -2), (dict(ldx=60), -1), (dict(ldn=60), -1), (dict(eps=0.0), -1),
    (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(x_type=24), -2), (dict(n_type=9), -2),
    (dict(scale=P), -1), (dict(n_type=24), -1), (dict(n_type=24, scale=P, ldn=72), -3), (dict(x=None), -1),
    (dict(n=None), -1), (dict(n=P, n_type=30), -1), (dict(n=P, ldn=68), -1), (dict(x=P + 4), -3),
    (dict(weight=P + 2), -3), (dict(T=0, x=None, n=None), 0)])
def test_rms_norm_refusals(L, over, status):
    assert L.elq_rms_norm(*_args(RMS, over)) == status


def _residual(**over):
    r = ops.ResidualC(T=4, cols=64, h_type=0, y_type=30, n_type=30, h=P, y=2 * P, h_out=3 * P, n=4 * P, ldh=64, ldy=64,
                      ld_out=64, ldn=64, gate_rows=1, gate_ld=64, gate_cols=64, res_scale=1.0, eps=1e-6)
    for k, v in over.items():
        setattr(r, k, v)
    return ctypes.byref(r)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), -1), (dict(cols=0), -1), (dict(ldh=63), -1), (dict(ldy=63), -1), (dict(ld_out=63), -1),
    (dict(ldn=63), -1), (dict(eps=-1.0), -1), (dict(h_type=24), -2), (dict(y_type=24), -2), (dict(n_type=9), -2),
    (dict(n_type=24), -1), (dict(scale=P), -1), (dict(n=None, scale=P), -1), (dict(n_type=24, scale=P, ldn=72), -3),
    (dict(gate=P, gate_rows=0), -1), (dict(gate=P, gate_cols=2), -1), (dict(gate=P, gate_ld=32), -1),
    (dict(h=None), -1), (dict(y=None), -1), (dict(h_out=None), -1), (dict(h_out=P, ld_out=68), -1),
    (dict(h_out=2 * P), -1), (dict(n=P), -1), (dict(n=2 * P), -1), (dict(n=3 * P), -1), (dict(h=P + 4), -3),
    (dict(gate=P + 2), -3), (dict(T=0, h=None, y=None), 0)])
def test_residual_norm_refusals(L, over, status):
    assert L.elq_residual_norm(_residual(**over), None) == status


def test_residual_norm_null_struct(L):
    assert L.elq_residual_norm(None, None) == -1


def test_binding_refuses_host_tensors_and_shapes(L):
    x = torch.zeros(4, 64)
    rows = ops.I8Rows(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4))
    for call in (lambda: ops.quantize_i8(x), lambda: ops.swiglu_i8(x), lambda: ops.rms_norm(x),
                 lambda: ops.rms_norm_i8(x), lambda: ops.residual_norm(x, x), lambda: ops.i8_matmul(rows, rows),
                 lambda: ops.grouped_matmul(rows, rows, torch.zeros(2, dtype=torch.int32)),
                 lambda: ops.combine_i8(x, torch.zeros(8, dtype=torch.int32), torch.zeros(4, 2)),
                 lambda: ops.quantize_i8(x[0]), lambda: ops.i8_matmul(x, rows), lambda: ops.rms_norm(x.double())):
        with pytest.raises(elq.ElqError):
            call()


def test_binding_is_rebuilt_for_another_torch_or_python(L, monkeypatch, tmp_path):
    """The compiled binding holds for the torch and Python that it was built against, and for no other."""
    ran = []

    def run(cmds):
        ran.extend(cmds)
        open(cmds[0][cmds[0].index("-o") + 1], "w").close()
        return ""

    made = tmp_path / "_ops.so"
    made.write_text("")
    monkeypatch.setattr(build, "BINDING", str(made))
    monkeypatch.setattr(build, "BINDING_FOR", str(tmp_path / "_ops.for"), raising=False)
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "deps", lambda: [build.LIB])     # the library is not this test's to build
    build.build()
    first = len(ran)
    build.build()
    assert len(ran) == first                            # up to date
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.0")
    build.build()
    assert len(ran) == first + 1                        # another torch
    build.build()
    assert len(ran) == first + 1


def test_status_reads_the_streams_device(monkeypatch):
    """The error word is a device's: a stream's own, whatever the current device is."""
    entered = []

    class On:
        def __init__(self, device):
            self.idx = device if device is None or isinstance(device, int) else torch.device(device).index

        def __enter__(self):
            entered.append(self.idx)

        def __exit__(self, *a):
            pass

    class Stream:
        device, cuda_stream = torch.device("cuda", 3), 77

    class Lib:
        @staticmethod
        def elq_ops_status(s):
            return s

    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(ops, "lib", lambda: Lib)
    assert ops.status(stream=Stream()) == 77 and entered == [3]
    assert ops.status(3, stream=Stream()) == 77 and entered == [3, 3]
    with pytest.raises(elq.ElqError):
        ops.status(0, stream=Stream())


def test_dequantize():
    r = ops.I8Rows(torch.tensor([[1, -2], [127, 0]], dtype=torch.int8), torch.tensor([0.5, 2.0]))
    assert torch.equal(r.dequantize(), torch.tensor([[0.5, -1.0], [254.0, 0.0]]))
    assert r.dequantize(torch.bfloat16).dtype == torch.bfloat16 and r.shape == (2, 2)
