"""int8_linear writes every element of its output and nothing beside it.  The tolerance
is that of its own tests (derived there); a NaN counts as a difference."""
import pytest
import torch

from gpu_util import dev
from quantized_state_space_b200 import api
from test_gpu_linear import make

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 37, 64), (5, 501, 1024), (64, 333, 4096), (100, 129, 2048),
                                   (300, 501, 640), (1000, 1001, 256), (3000, 2563, 256),
                                   (5000, 1283, 1040), (2500, 2600, 128)])
def test_product_writes_every_element_and_no_other(m, n, k, dtype):
    """Into a buffer of NaN (unwritten elements show) whose rows are longer than the
    output's, on 16 bytes and off them; widths that end inside 16 bytes."""
    p = make(m + n, m, n, k, bias=True, full=True)
    acc = p["x"].double() @ p["w"].double().t()
    prod = acc * p["xs"].double()[:, None] * p["ws"].double()[None]
    want = prod + p["bias"].double()
    fi = torch.finfo(dtype)
    tol = 3 * 2.0 ** -24 * prod.abs() + (2.0 ** -24 + fi.eps / 2) * want.abs() + fi.tiny * fi.eps
    for off, pitch in ((0, (n + 15) // 16 * 16 + 16), (8, (n + 15) // 16 * 16 + 16), (3, n + 4)):
        wide = torch.full((m + 2, pitch), 7.0, dtype=dtype, device=dev())
        out = wide[1:m + 1, off:off + n]
        out.fill_(float("nan"))
        y = api.int8_linear(p["x"], p["xs"], p["w"], p["ws"], bias=p["bias"], out=out)
        ok = (y.double() - want).abs() <= tol
        assert ok.all(), (int((~ok).sum()), (~ok).nonzero()[:4].tolist())
        keep = torch.ones_like(wide, dtype=torch.bool)
        keep[1:m + 1, off:off + n] = False
        assert (wide[keep] == 7).all()
