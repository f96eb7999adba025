"""Argument checks of the quantized-layer operators and the gated recurrence:
every refusal comes back before any device call (no GPU needed)."""
import ctypes as C
import os
import subprocess

import pytest
import torch

from quantized_state_space_b200 import _native as N
from quantized_state_space_b200 import api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # aligned, never dereferenced
STEP = 0x100000


@pytest.fixture(scope="module")
def L():
    return N.lib()


def _c_name(field):
    for tail in ("_batch_stride", "_row_stride"):
        if field.endswith(tail):
            return field[:-len(tail)] + "." + tail[1:]
    return field


def test_struct_layout_matches_header(tmp_path):
    structs = ((N.NormArgs, "ssmq_norm_args"), (N.LinearArgs, "ssmq_linear_args"),
               (N.GatedArgs, "ssmq_gated_args"),
               (N.GatedGradArgs, "ssmq_gated_grad_args"))
    prog = ["#include <stdio.h>", "#include <stddef.h>", '#include "ssmq.h"', "int main(void){"]
    for cls, cname in structs:
        prog.append('printf("%s %%zu\\n", sizeof(%s));' % (cname, cname))
        for f, _ in cls._fields_:
            prog.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (cname, f, cname, _c_name(f)))
    prog.append("return 0;}")
    src = tmp_path / "layout.c"
    src.write_text("\n".join(prog))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    got = dict(line.split() for line in subprocess.check_output([str(exe)], text=True).splitlines())
    for cls, cname in structs:
        assert int(got[cname]) == C.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(got["%s.%s" % (cname, f)]) == getattr(cls, f).offset, (cname, f)


def test_norm(L):
    base = dict(tokens=8, dim=64, dtype=N.F16, eps=1e-5, x=A, x_stride=64, codes=A + STEP,
                codes_stride=64, scales=A + 2 * STEP)
    S = lambda **kw: L.ssmq_rms_norm_quantize(C.byref(N.NormArgs(**{**base, **kw})), None)
    assert L.ssmq_rms_norm_quantize(None, None) == N.ERR_INVALID_ARG
    assert S(dtype=3) == N.ERR_INVALID_ARG
    assert S(tokens=-1) == N.ERR_INVALID_ARG
    assert S(dim=0) == N.ERR_INVALID_ARG
    assert S(dim=32769, x_stride=40000, codes_stride=40000) == N.ERR_UNSUPPORTED
    assert S(tokens=1 << 31) == N.ERR_UNSUPPORTED
    assert S(eps=-1.0) == N.ERR_INVALID_ARG
    assert S(eps=float("nan")) == N.ERR_INVALID_ARG
    assert S(x=None) == N.ERR_INVALID_ARG
    assert S(codes=None) == N.ERR_INVALID_ARG
    assert S(scales=None) == N.ERR_INVALID_ARG
    assert S(codes=None, scales=None) == N.ERR_INVALID_ARG  # no output at all
    assert S(x_stride=63) == N.ERR_INVALID_ARG
    assert S(codes_stride=10) == N.ERR_INVALID_ARG
    assert S(x=A + 1) == N.ERR_ALIGNMENT
    assert S(scales=A + 2) == N.ERR_ALIGNMENT
    assert S(codes=A) == N.ERR_INVALID_ARG and "codes overlaps x" in N.ssmq_last_error()
    # residual_out: exactly an input, or apart from it
    r = dict(residual=A + 4 * STEP, residual_stride=64, residual_out_stride=64)
    assert S(residual_out=A + 2, **r) == N.ERR_INVALID_ARG
    assert S(residual_out=A, x_stride=128, **r) == N.ERR_INVALID_ARG  # same address, other stride
    assert S(residual_out=A + STEP, **r) == N.ERR_INVALID_ARG         # the codes
    assert S(y=A, y_stride=64) == N.ERR_INVALID_ARG
    assert S(tokens=0, x=None) == N.OK


def test_linear(L, monkeypatch):
    base = dict(tokens=8, out_features=24, in_features=64, dtype=N.F16, x=A, x_stride=64,
                x_scale=A + STEP, w=A + 2 * STEP, w_stride=64, w_scale=A + 3 * STEP,
                y=A + 4 * STEP, y_stride=24)
    args = lambda **kw: C.byref(N.LinearArgs(**{**base, **kw}))
    S = lambda ws=None, nb=0, **kw: L.ssmq_int8_linear(args(**kw), ws, nb, None)
    W = lambda **kw: L.ssmq_int8_linear_workspace_size(args(**kw))
    assert L.ssmq_int8_linear(None, None, 0, None) == N.ERR_INVALID_ARG
    assert S(dtype=9) == N.ERR_INVALID_ARG
    assert S(tokens=-1) == N.ERR_INVALID_ARG
    assert S(in_features=131072, x_stride=1 << 18, w_stride=1 << 18) == N.ERR_UNSUPPORTED
    assert S(tokens=1 << 31) == N.ERR_UNSUPPORTED
    assert S(x=None) == N.ERR_INVALID_ARG
    assert S(w_scale=None) == N.ERR_INVALID_ARG
    assert S(x_scale=A + STEP + 1) == N.ERR_ALIGNMENT
    assert S(x_stride=63) == N.ERR_INVALID_ARG
    assert S(y_stride=23) == N.ERR_INVALID_ARG
    assert S(y=A + 4 * STEP + 1) == N.ERR_ALIGNMENT
    assert S(y=A + 64) == N.ERR_INVALID_ARG and "y overlaps x" in N.ssmq_last_error()
    assert S(w_stride=1 << 41) == N.ERR_UNSUPPORTED
    assert S(tokens=0, x=None) == N.OK and S(out_features=0, w=None) == N.OK
    # the workspace rule: only rows that are off 16-byte boundaries are copied
    assert W() == 0 and W(x=A + 16) == 0 and W(tokens=1, x_stride=3) == 0
    assert W(x=A + 1) == 512 and W(w_stride=65) == 24 * 64
    assert W(x_stride=70, w=A + 2 * STEP + 8) == 512 + 24 * 64
    assert W(in_features=50) == 0 and W(in_features=50, x_stride=50) == 512
    assert L.ssmq_int8_linear_workspace_size(None) == 0
    assert S(x=A + 1) == N.ERR_INVALID_ARG and "workspace" in N.ssmq_last_error()
    assert S(x=A + 1, ws=A + 8 * STEP, nb=511) == N.ERR_INVALID_ARG
    assert S(x=A + 1, ws=A + 8 * STEP + 16, nb=512) == N.ERR_ALIGNMENT
    assert S(x=A + 1, ws=A + 2 * STEP, nb=512) == N.ERR_INVALID_ARG   # on w
    monkeypatch.setenv("SSMQ_FAULT_INJECT", "ssmq_int8_linear")
    assert S() == N.ERR_CUDA
    assert S(x=A + 1, ws=A + 8 * STEP, nb=512) == N.ERR_CUDA


def _gated(**kw):
    f = dict(batch=2, seqlen=100, dim=32, dtype=N.F16, h_final=A + 9 * STEP)
    for i, n in enumerate(("v", "g", "z", "y")):
        f.update({n: A + i * STEP, n + "_batch_stride": 3200, n + "_row_stride": 32})
    f.update(kw)
    return N.GatedArgs(**f)


def test_gated_scan(L):
    S = lambda **kw: L.ssmq_gated_scan(C.byref(_gated(**kw)), None)
    assert L.ssmq_gated_scan(None, None) == N.ERR_INVALID_ARG
    assert S(dtype=7) == N.ERR_INVALID_ARG
    assert S(seqlen=-1) == N.ERR_INVALID_ARG
    assert S(batch=1 << 30, dim=1 << 20) == N.ERR_UNSUPPORTED
    assert S(seqlen=1 << 31) == N.ERR_UNSUPPORTED
    assert S(v=None) == N.ERR_INVALID_ARG
    assert S(y=None) == N.ERR_INVALID_ARG
    assert S(g=A + 1) == N.ERR_ALIGNMENT
    assert S(h0=A + 2) == N.ERR_ALIGNMENT
    assert S(lengths=A + 2) == N.ERR_ALIGNMENT
    assert S(g_row_stride=31) == N.ERR_INVALID_ARG
    assert S(v_batch_stride=-1) == N.ERR_INVALID_ARG
    assert S(v_batch_stride=1 << 62, v_row_stride=1 << 61) == N.ERR_INVALID_ARG
    assert S(y_batch_stride=3199) == N.ERR_INVALID_ARG          # sequences of y overlap
    assert S(y=A) == N.ERR_INVALID_ARG                          # y on v
    assert S(y=A + 2 * STEP + 2) == N.ERR_INVALID_ARG           # shifted against z
    assert S(h_final=A + 3 * STEP) == N.ERR_INVALID_ARG
    assert S(states=A + 9 * STEP) == N.ERR_INVALID_ARG
    assert S(states=A + 8 * STEP, h0=A + 8 * STEP) == N.ERR_INVALID_ARG
    assert S(batch=0, v=None) == N.OK
    assert L.ssmq_gated_scan_state_steps() >= 1


def test_gated_scan_fault_injection(L, monkeypatch):
    """Valid overlaps (y on z, h_final on h0, interleaved columns) reach the launch."""
    monkeypatch.setenv("SSMQ_FAULT_INJECT", "all")
    S = lambda **kw: L.ssmq_gated_scan(C.byref(_gated(**kw)), None)
    assert S() == N.ERR_CUDA
    assert S(y=A + 2 * STEP) == N.ERR_CUDA
    assert S(h0=A + 9 * STEP) == N.ERR_CUDA
    cols = {}
    for i, n in enumerate(("v", "g", "z", "y")):
        cols.update({n: A + 64 * i, n + "_batch_stride": 12800, n + "_row_stride": 128})
    assert S(**cols) == N.ERR_CUDA
    cols["y"] = A + 64 * 3 - 2
    assert S(**cols) == N.ERR_INVALID_ARG
    for i, n in enumerate(("v", "g", "z", "y")):  # the same, rows of both sequences in turn
        cols.update({n: A + 64 * i, n + "_batch_stride": 128, n + "_row_stride": 256})
    assert S(**cols) == N.ERR_CUDA
    cols["y"] = A + 64 * 3 + 2
    assert S(**cols) == N.ERR_INVALID_ARG
    for n in ("v", "g", "z", "y"):  # interleaved unevenly: not told apart
        cols.update({n + "_batch_stride": 128, n + "_row_stride": 300})
    cols["y"] = A + 64 * 3
    assert S(**cols) == N.ERR_INVALID_ARG


def test_gated_backward(L):
    def S(**kw):
        f = dict(batch=2, seqlen=100, dim=32, dtype=N.BF16, states=A + 10 * STEP,
                 dh0=A + 11 * STEP, dh_final=A + 12 * STEP)
        for i, n in enumerate(("v", "g", "z", "dy", "dv", "dg", "dz")):
            f.update({n: A + i * STEP, n + "_batch_stride": 3200, n + "_row_stride": 32})
        f.update(kw)
        return L.ssmq_gated_scan_backward(C.byref(N.GatedGradArgs(**f)), None)
    assert L.ssmq_gated_scan_backward(None, None) == N.ERR_INVALID_ARG
    assert S(dtype=-1) == N.ERR_INVALID_ARG
    assert S(states=None) == N.ERR_INVALID_ARG
    assert S(dv=None) == N.ERR_INVALID_ARG
    assert S(dz=None) == N.ERR_INVALID_ARG and S(z=None) == N.ERR_INVALID_ARG
    assert S(dv=A + 5 * STEP) == N.ERR_INVALID_ARG              # dv is dg
    assert S(dg=A + 64) == N.ERR_INVALID_ARG
    assert S(dh0=A + 10 * STEP) == N.ERR_INVALID_ARG
    assert S(dy_row_stride=16) == N.ERR_INVALID_ARG
    assert S(states=A + 2) == N.ERR_ALIGNMENT
    assert S(dim=0) == N.OK


def test_gated_update(L):
    S = lambda **kw: L.ssmq_gated_update(C.byref(_gated(**{"seqlen": 1, **kw})), None)
    assert S(seqlen=2) == N.ERR_INVALID_ARG
    assert S(h_final=None) == N.ERR_INVALID_ARG
    assert S(states=A) == N.ERR_INVALID_ARG
    assert S(lengths=A) == N.ERR_INVALID_ARG
    assert S(y_batch_stride=31) == N.ERR_INVALID_ARG
    assert S(y=A + STEP) == N.ERR_INVALID_ARG
    assert S(h_final=A) == N.ERR_INVALID_ARG                    # the state on v
    assert S(h_final=A + 3 * STEP) == N.ERR_INVALID_ARG
    assert S(batch=0) == N.OK


def test_python_front_end_refusals():
    """Wrong devices, dtypes, shapes and strides never reach the library."""
    x = torch.zeros(4, 16, dtype=torch.float16)
    with pytest.raises(ValueError):
        api.rms_norm_quantize(x)  # not on a GPU
    with pytest.raises(ValueError):
        api.rms_norm_quantize(x.double())
    q = torch.zeros(4, 16, dtype=torch.int8)
    with pytest.raises(ValueError):
        api.int8_linear(q, torch.ones(4), q, torch.ones(4))
    with pytest.raises(ValueError):
        api.int8_linear(q, torch.ones(4), q, torch.ones(4), dtype=torch.int32)
    with pytest.raises(ValueError):
        api.gated_scan(x, x)
    with pytest.raises(ValueError):
        api.gated_scan(x[None], x[None])
    with pytest.raises(ValueError):
        api.gated_scan(x[None].int(), x[None].int())
    with pytest.raises(ValueError):
        api.gated_scan_backward(x[None], x[None], x[None], x)
    with pytest.raises(ValueError):
        api.gated_update(x, x, x)
