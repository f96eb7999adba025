"""int8_linear on the GPU against the exact integer product.

Tolerance: the integer sum is exact; y = fl(fl(acc) fl(sx sw) + bias) has the
roundings of acc to binary32 and of the scales' product (2 half-ulps), one
fused multiply-add (a half-ulp of the result), then half a step of the type:
3 * 2^-24 |acc sx sw| + (2^-24 + eps / 2) |y|.
"""
import numpy as np
import pytest
import torch

from gpu_util import H, dev, status_word
from quantized_state_space_b200 import api

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def make(seed, m, n, k, bias=False, full=False):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if full else -127
    p = dict(x=torch.randint(lo, 128, (m, k), generator=g, dtype=torch.int8),
             w=torch.randint(lo, 128, (n, k), generator=g, dtype=torch.int8),
             xs=torch.rand(m, generator=g) * 0.02 + 1e-3,
             ws=(torch.rand(n, generator=g) + 0.1) * 1e-3)
    p["bias"] = torch.randn(n, generator=g) if bias else None
    return {a: None if t is None else t.to(dev()) for a, t in p.items()}


def check(y, p):
    acc = p["x"].double() @ p["w"].double().t()  # integers below 2^53: exact
    prod = acc * p["xs"].double()[:, None] * p["ws"].double()[None]
    want = prod if p["bias"] is None else prod + p["bias"].double()
    fi = torch.finfo(y.dtype)
    tol = 3 * 2.0 ** -24 * prod.abs() + (2.0 ** -24 + fi.eps / 2) * want.abs() + fi.tiny * fi.eps
    assert y.shape == want.shape
    bad = (y.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4], want[bad][:4])


def call(p, dtype=F16, **kw):
    return api.int8_linear(p["x"], p["xs"], p["w"], p["ws"], bias=p["bias"], dtype=dtype, **kw)


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 300])
@pytest.mark.parametrize("n,k", [(1, 16), (16, 128), (129, 144), (128, 1024), (333, 2048),
                                 (700, 4112)])
def test_few_tokens(m, n, k):
    p = make(m * 7 + n, m, n, k, bias=n % 2 == 1, full=True)
    check(call(p), p)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("m,n,k", [(2048, 2560, 512), (2500, 2611, 400), (4096, 4100, 128),
                                   (20000, 256, 272), (300, 20000, 640), (5000, 5000, 16)])
def test_many_tokens(m, n, k, dtype):
    """Persistent tiles: several per CTA pair, ragged in every dimension."""
    p = make(m + n + k, m, n, k, bias=True)
    check(call(p, dtype), p)


@pytest.mark.parametrize("k", [1, 2, 15, 17, 31, 100, 127, 129, 1001])
@pytest.mark.parametrize("m", [3, 150])
def test_any_in_features(k, m):
    """Rows that are not on 16-byte boundaries go through the workspace."""
    p = make(k, m, 90, k)
    check(call(p, F32), p)
    y = torch.empty(m, 90, dtype=F32, device=dev())
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    assert torch.equal(api.int8_linear(p["x"], p["xs"], p["w"], p["ws"], out=y, workspace=ws),
                       call(p, F32))


def test_large_and_long():
    p = make(1, 5, 40, 131071, full=True)
    p["x"].fill_(-128)
    p["w"].fill_(-128)  # 131071 * 2^14 = 2^31 - 2^14
    check(call(p, F32), p)
    p = make(2, 400, 300, 20000)
    check(call(p, F32), p)


@pytest.mark.parametrize("m", [7, 200, 3000])
def test_strides(m):
    """Padded rows (bytes behind a row's end do not count), unaligned column
    slices, output as a column slice of a wider tensor."""
    n, k = 500, 200
    p = make(5, m, n, k, bias=True)
    for off, pitch in ((0, 208), (16, 256), (3, 211)):
        q = dict(p)
        for name, rows in (("x", m), ("w", n)):
            wide = torch.full((rows, pitch + off), 111, dtype=torch.int8, device=dev())
            wide[:, off:off + k] = p[name]
            q[name] = wide[:, off:off + k]
        out = torch.full((m, n + 9), 7.0, dtype=BF16, device=dev())
        y = api.int8_linear(q["x"], q["xs"], q["w"], q["ws"], bias=q["bias"], out=out[:, 4:n + 4])
        check(y, p)
        assert (out[:, :4] == 7).all() and (out[:, n + 4:] == 7).all()


def test_leading_dimensions_and_empty():
    p = make(6, 12, 33, 64)
    y = api.int8_linear(p["x"].view(3, 4, 64), p["xs"].view(3, 4), p["w"], p["ws"])
    assert y.shape == (3, 4, 33) and torch.equal(y.view(12, 33), call(p))
    assert api.int8_linear(p["x"][:0], p["xs"][:0], p["w"], p["ws"]).shape == (0, 33)
    assert api.int8_linear(p["x"], p["xs"], p["w"][:0], p["ws"][:0]).shape == (12, 0)
    b = torch.randn(33, device=dev())
    y = api.int8_linear(p["x"][:, :0], p["xs"], p["w"][:, :0], p["ws"], bias=b, dtype=F32)
    assert torch.equal(y, b.expand(12, 33))


def test_rows_are_independent():
    """A token's row has the same bytes whatever the batch around it."""
    p = make(7, 3000, 2700, 512, bias=True)
    y = call(p)
    for rows in (slice(0, 1), slice(40, 90), slice(100, 400)):
        q = dict(p, x=p["x"][rows].contiguous(), xs=p["xs"][rows].contiguous())
        assert torch.equal(call(q), y[rows])


def test_non_finite_scales():
    p = make(8, 20, 40, 64)
    p["xs"][3] = float("inf")
    p["ws"][7] = float("nan")
    y = call(p, F32)
    keep = torch.ones(20, 40, dtype=torch.bool, device=dev())
    keep[3], keep[:, 7] = False, False
    assert torch.isfinite(y[keep]).all() and not torch.isfinite(y[~keep]).any()


def test_status_streams_and_graph():
    for m, n, k in ((4, 1000, 4096), (3000, 3000, 256)):
        p = make(m, m, n, k)
        st = status_word()
        ref = call(p, status=st)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            a = call(p)
        s.synchronize()
        out = torch.zeros_like(ref)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            api.int8_linear(p["x"], p["xs"], p["w"], p["ws"], out=out)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, ref) and torch.equal(out, ref) and int(st) == 0


def test_two_streams_at_once():
    """Both kernels on two streams at the same time."""
    ps = [make(9, 2600, 2600, 1024), make(10, 3, 4000, 4096)]
    refs = [call(p) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(call(ps[i]))
    torch.cuda.synchronize()
    for r, o in zip(refs, outs):
        assert all(torch.equal(r, y) for y in o)
