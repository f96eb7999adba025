"""Bounded device waits of the quantized-layer operators, made to give up on the
first probe (SSMQ_WAIT_LIMIT=0): the call returns, raises SSMQ_DEV_TIMEOUT and
leaves NaN in what it did not finish, nothing outside its output is written,
and the next call is whole again."""
import pytest
import torch

from gpu_util import dev, status_word
from quantized_state_space_b200 import _native as N
from quantized_state_space_b200 import api
from test_gpu_linear import make

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def linear_gives_up(monkeypatch, m, n, k, dtype, off):
    p = make(m + n, m, n, k, bias=True)
    wide = torch.full((m + 1, n + 32), 7.0, dtype=dtype, device=dev())
    out, st = wide[:m, off:off + n], status_word()
    call = lambda: api.int8_linear(p["x"], p["xs"], p["w"], p["ws"], bias=p["bias"], out=out,
                                   status=st)
    monkeypatch.setenv("SSMQ_WAIT_LIMIT", "0")
    call()
    torch.cuda.synchronize()
    assert int(st) == N.DEV_TIMEOUT
    assert torch.isnan(out).all()
    assert (wide[m:] == 7).all() and (wide[:, :off] == 7).all() and (wide[:, off + n:] == 7).all()
    monkeypatch.delenv("SSMQ_WAIT_LIMIT")
    st.zero_()
    call()
    assert int(st) == 0
    assert torch.equal(out, api.int8_linear(p["x"], p["xs"], p["w"], p["ws"], bias=p["bias"],
                                            dtype=dtype))


# outputs through shared memory by TMA (rows on 16 bytes) and straight from
# registers; one K block and many, one tile per pair of CTAs and several (with more
# than five K blocks the MMAs' own wait runs out too, after about a second)
@pytest.mark.parametrize("dtype,off", [(F16, 16), (BF16, 3), (F32, 16)])
@pytest.mark.parametrize("m,n,k", [(4096, 2560, 512), (500, 500, 128), (5000, 5000, 1040)])
def test_product_of_many_tokens(monkeypatch, m, n, k, dtype, off):
    linear_gives_up(monkeypatch, m, n, k, dtype, off)


# token tiles of 16 to 128 columns, K whole or in 2 or 4 parts (the first four copies
# or more need no wait: a short K gives up in the epilogue alone)
@pytest.mark.parametrize("dtype,off", [(F16, 16), (BF16, 3), (F32, 16)])
@pytest.mark.parametrize("m,n,k", [(1, 300, 640), (4, 1000, 4096), (64, 4096, 8192),
                                   (90, 3000, 8192), (777, 1801, 1536), (300, 20000, 640),
                                   (30, 5000, 3008), (20, 300, 16)])
def test_product_of_few_tokens(monkeypatch, m, n, k, dtype, off):
    linear_gives_up(monkeypatch, m, n, k, dtype, off)


def padded(gen, b, L, d, pad, dtype):
    """(b, L, d) in rows of d + pad elements, with one more sequence behind."""
    wide = torch.randn(b + 1, L, d + pad, generator=gen).to(dtype).to(dev())
    return wide[:b, :, :d]


def guarded(b, L, d, pad, dtype):
    """The same layout to write to, and all of it: 7 where nothing was written."""
    wide = torch.full((b + 1, L, d + pad), 7.0, dtype=dtype, device=dev())
    return wide[:b, :, :d], wide


def untouched(wide, b, d):
    return (wide[b:] == 7).all() and (wide[:, :, d:] == 7).all()


def all_nan(*ts):
    return all(bool(torch.isnan(t).all()) for t in ts)


# rows on 16 bytes (copies by TMA), even rows (pairs), odd rows (single channels, and
# words in the gradient); one round and many, whole clusters and a single CTA
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("pad", [0, 2, 3])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("b,L,d", [(2, 300, 64), (1, 9000, 48), (64, 70, 2560), (3, 40, 40)])
def test_gated_recurrence(monkeypatch, b, L, d, z, pad, dtype):
    gen = torch.Generator().manual_seed(L + d)
    v, g, dy = (padded(gen, b, L, d, pad, dtype) for _ in range(3))
    zz = padded(gen, b, L, d, pad, dtype) if z else None
    h0, dh = (torch.randn(b, d, generator=gen).to(dev()) for _ in range(2))
    st = status_word()
    # (a sequence of one tile in a CTA that copies for itself waits for nothing)
    waits = pad == 0 or L > 256 or (L > 64 and b * d < 10000)
    fwd = lambda y: api.gated_scan(v, g, z=zz, h0=h0, y=y, save_states=True, status=st)
    bwd = lambda s, dv, dg, dz: api.gated_scan_backward(dy, v, g, s, z=zz, dh_final=dh, dv=dv,
                                                        dg=dg, dz=dz, status=st)
    outs = [guarded(b, L, d, pad, dtype) for _ in range(4 if z else 3)]
    y, wides = outs[0][0], [o[1] for o in outs]
    grads = [o[0] for o in outs[1:]] + ([] if z else [None])
    _, h, states = fwd(y)
    ref = [t.clone() for t in (y, h, states)]
    ref_g = [t.clone() for t in bwd(states, *grads) if t is not None]
    assert int(st) == 0

    for w in wides:
        w.fill_(7)
    monkeypatch.setenv("SSMQ_WAIT_LIMIT", "0")
    _, h, s = fwd(y)
    torch.cuda.synchronize()
    assert int(st) == (N.DEV_TIMEOUT if waits else 0)
    if waits:
        assert all_nan(y, h, s)
    st.zero_()
    dv, dg, dz, dh0 = bwd(ref[2], *grads)
    torch.cuda.synchronize()
    assert int(st) == (N.DEV_TIMEOUT if waits else 0)
    if waits:
        assert all_nan(dv, dg, dh0)
        if z and pad == 0:  # (else the first round's are whole: they need no exchange)
            assert all_nan(dz)
    assert all(untouched(w, b, d) for w in wides)

    monkeypatch.delenv("SSMQ_WAIT_LIMIT")
    st.zero_()
    again = [t for t in fwd(y)]
    again_g = [t for t in bwd(again[2], *grads) if t is not None]
    assert int(st) == 0
    for r, t in zip(ref + ref_g, again + again_g):
        assert torch.equal(r, t)
