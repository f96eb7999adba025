"""rms_norm_quantize on the GPU against the definition in 64 bits.

Tolerances, from the kernel's arithmetic: a token's sum of squares adds at most
32 products per thread, 5 shuffle and 5 cross-warp partials, so its relative
error is below 43 half-ulps; with the division by dim, the reciprocal square
root (2 ulps), and the products with weight and rstd, v is within 2^-19
relative, and so is the scale.  A code is the nearest integer to v / scale,
|v / scale| <= 127: off by at most 1/2 + 127 * 2 * 2^-19 < 1/2 + 2^-11.
"""
import numpy as np
import pytest
import torch

from gpu_util import H, dev, status_word
from quantized_state_space_b200 import _native as N
from quantized_state_space_b200 import api

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
V_TOL = 2.0 ** -19


def make(seed, shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def reference(x, w, res, eps):
    """(r, v, scale) in 64 bits from CPU tensors; r rounded to the stream's type."""
    r = x if res is None else (x.float() + res.float()).to(x.dtype)
    rd = r.double()
    v = rd / torch.sqrt((rd * rd).mean(-1, keepdim=True) + eps)
    if w is not None:
        v = v * w.double()
    return r, v, v.abs().amax(-1) / 127


def check(x, w, res, eps, codes, scales, r=None, y=None):
    rr, v, s = reference(x, w, res, eps)
    if r is not None:
        assert torch.equal(r.cpu(), rr)
    sc = scales.cpu().double()
    assert ((sc - s).abs() <= V_TOL * s).all()
    off = (codes.cpu().double() * sc[..., None] - v).abs()
    assert (off <= (0.5 + 2.0 ** -11) * sc[..., None]).all()
    assert (codes.cpu().abs() <= 127).all()
    if y is not None:
        tol = (torch.finfo(x.dtype).eps / 2 + V_TOL) * v.abs() + torch.finfo(x.dtype).tiny
        assert ((y.cpu().double() - v).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("d", [1, 7, 8, 31, 32, 40, 64, 100, 128, 250, 256, 264, 512, 513, 520,
                               1536, 2047, 2048, 2056, 2561, 5120, 8200, 16384, 16385, 20000,
                               32768])
def test_widths(dtype, d):
    tokens = 5
    x, res = make(d, (tokens, d), dtype), make(d + 1, (tokens, d), dtype)
    w = make(d + 2, (d,), F32)
    codes, scales, r, y = api.rms_norm_quantize(x.to(dev()), w.to(dev()), residual=res.to(dev()),
                                                want_y=True)
    check(x, w, res, 1e-5, codes, scales, r, y)


@pytest.mark.parametrize("tokens", [0, 1, 2, 3, 33, 1000])
@pytest.mark.parametrize("d", [16, 48, 333])
@pytest.mark.parametrize("residual", [False, True])
def test_token_counts(tokens, d, residual):
    x = make(7, (tokens, d), F16)
    res = make(8, (tokens, d), F16) if residual else None
    out = api.rms_norm_quantize(x.to(dev()), residual=res.to(dev()) if residual else None)
    assert len(out) == (3 if residual else 2)
    if tokens:
        check(x, None, res, 1e-5, out[0], out[1], out[2] if residual else None)
    assert out[0].shape == (tokens, d) and out[1].shape == (tokens,)


def test_codes_are_the_group_quantizers(orc):
    """binary32: the codes are, bit for bit, the group quantizer's codes of the
    returned values with one group per token at the returned scales."""
    for d, seed in ((24, 1), (1537, 2), (4096, 3)):
        x = make(seed, (9, d), F32, 3.0)
        w = make(seed + 9, (d,), F32)
        codes, scales, y = api.rms_norm_quantize(x.to(dev()), w.to(dev()), want_y=True)
        v = H(y)
        for mode in (orc.SCALE_STATIC, orc.SCALE_ABSMAX):
            q, s, _ = orc.quantize_groups(v, 1, 9, d, np.arange(9, dtype=np.int32), 9, mode,
                                          H(scales))
            np.testing.assert_array_equal(H(codes), q.reshape(9, d))
            np.testing.assert_array_equal(H(scales), s)


@pytest.mark.parametrize("d", [64, 63, 1536])
def test_strides_and_rows_behind(d):
    """Column slices as input and output; what lies between the rows stays."""
    T = 6
    wide = make(1, (T, 3 * d + 5), F16).to(dev())
    x, res = wide[:, 1:1 + d], wide[:, d + 2:2 * d + 2]
    out = torch.full((T, 2 * d + 6), 77.0, dtype=F16, device=dev())
    cw = torch.full((T + 1, d + 32), 99, dtype=torch.int8, device=dev())
    sc = torch.full((T + 1,), -1.0, device=dev())
    codes, scales, r, y = api.rms_norm_quantize(
        x, residual=res, residual_out=out[:, :d], y=out[:, d + 3:2 * d + 3],
        codes=cw[:T, :d], scales=sc[:T])
    check(x.cpu(), None, res.cpu(), 1e-5, codes, scales, r, y)
    assert (out[:, d:d + 3] == 77).all() and (out[:, 2 * d + 3:] == 77).all()
    assert (cw[:, d:] == 99).all() and (cw[T] == 99).all() and sc[T] == -1


def test_leading_dimensions_and_padded_codes():
    x = make(3, (2, 5, 333), BF16)
    codes, scales = api.rms_norm_quantize(x.to(dev()))
    assert codes.shape == (2, 5, 333) and scales.shape == (2, 5)
    assert codes.stride(-2) % 16 == 0 and codes.data_ptr() % 16 == 0
    check(x, None, None, 1e-5, codes, scales)


@pytest.mark.parametrize("which", ["x", "residual"])
def test_in_place(which):
    x, res = make(4, (65, 200), BF16), make(5, (65, 200), BF16)
    xg, rg = x.to(dev()), res.to(dev())
    target = xg if which == "x" else rg
    codes, scales, r = api.rms_norm_quantize(xg, residual=rg, residual_out=target)
    assert r.data_ptr() == target.data_ptr()
    check(x, None, res, 1e-5, codes, scales, target)


def test_values_alone():
    x = make(6, (10, 96), F16)
    codes, scales, y = api.rms_norm_quantize(x.to(dev()), want_codes=False, want_y=True)
    assert codes is None and scales is None
    v = reference(x, None, None, 1e-5)[1]
    assert ((y.cpu().double() - v).abs() <= (2.0 ** -11 + V_TOL) * v.abs() + 2.0 ** -25).all()


@pytest.mark.parametrize("d", [24, 29, 300, 1000])
def test_zero_and_non_finite_tokens(d):
    """Zero tokens, infinities, NaN and an overflowing sum: scale 0, codes 0,
    the flag; neighbours are unaffected."""
    x = make(9, (7, d), F32)
    x[1] = 0
    x[2, d // 2] = float("inf")
    x[3, 0] = float("nan")
    x[4] = 3e38
    x[5, d - 1] = -float("inf")
    st = status_word()
    codes, scales = api.rms_norm_quantize(x.to(dev()), status=st)
    assert int(st) == N.DEV_NONFINITE
    for t in (1, 2, 3, 4, 5):
        assert float(scales[t]) == 0.0 and not codes[t].any()
    for t in (0, 6):
        check(x[t:t + 1], None, None, 1e-5, codes[t:t + 1], scales[t:t + 1])
    st.zero_()
    api.rms_norm_quantize(x[:2].to(dev()), status=st)
    assert int(st) == 0


def test_non_finite_weight():
    x = make(10, (3, 64), F16)
    w = torch.ones(64)
    w[5], w[40] = float("inf"), float("nan")
    st = status_word()
    codes, scales = api.rms_norm_quantize(x.to(dev()), w.to(dev()), status=st)
    assert int(st) == N.DEV_NONFINITE
    w[5] = w[40] = 0
    good = torch.tensor([c for c in range(64) if c not in (5, 40)])
    _, v, _ = reference(x, w, None, 1e-5)
    s = v.abs().amax(-1) / 127
    assert ((scales.cpu().double() - s).abs() <= V_TOL * s).all()
    assert not codes[:, 5].any() and not codes[:, 40].any()
    off = (codes.cpu().double() * scales.cpu().double()[:, None] - v)[:, good].abs()
    assert (off <= (0.5 + 2.0 ** -11) * scales.cpu().double()[:, None]).all()


def test_tiny_and_large_values():
    for dtype, scale in ((F16, 1e-4), (F16, 1e4), (BF16, 1e-18), (BF16, 1e15), (F32, 1e-18)):
        x = make(11, (4, 512), dtype, scale)
        codes, scales = api.rms_norm_quantize(x.to(dev()), eps=0.0)
        check(x, None, None, 0.0, codes, scales)


def test_other_stream_and_graph():
    x, res = make(12, (130, 768), F16).to(dev()), make(13, (130, 768), F16).to(dev())
    ref = api.rms_norm_quantize(x, residual=res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = api.rms_norm_quantize(x, residual=res)
    s.synchronize()
    codes, scales, r = (torch.zeros_like(t) for t in ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.rms_norm_quantize(x, residual=res, codes=codes, scales=scales, residual_out=r)
    for _ in range(2):
        codes.zero_()
        g.replay()
    torch.cuda.synchronize()
    for t, u, v in zip(ref, a, (codes, scales, r)):
        assert torch.equal(t, u) and torch.equal(t, v)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("d", list(range(1, 26)) + [63, 65, 127, 129, 255, 257, 511, 515, 1001])
def test_rows_off_16_byte_boundaries(dtype, d):
    """Every distance of a row's start from a 16-byte boundary: rows of d
    elements in a buffer, the first of them shifted as well."""
    T = 9
    for shift in (0, 1, 3):
        buf = make(d, (3, T * d + 16), dtype).to(dev())
        x, res = (buf[k, shift:shift + T * d].view(T, d) for k in (0, 1))
        out = torch.full((2, T * d + 16), 7.0, dtype=dtype, device=dev())
        r, y = (out[k, shift:shift + T * d].view(T, d) for k in (0, 1))
        w = make(d + 1, (d,), F32)
        codes, scales, r, y = api.rms_norm_quantize(x, w.to(dev()), residual=res, residual_out=r, y=y)
        check(x.cpu(), w, res.cpu(), 1e-5, codes, scales, r, y)
        rest = torch.cat((out[:, :shift], out[:, shift + T * d:]), 1)
        assert (rest == 7).all()
