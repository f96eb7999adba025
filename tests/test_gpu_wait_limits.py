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
