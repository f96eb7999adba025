"""rms_norm_quantize where values leave binary32: an element that is not finite for its
weight's sake is coded 0 and left out of the token's maximum, whether the product with
the weight overflows or the product's multiple by rstd."""
import pytest
import torch

from gpu_util import dev, status_word
from quantized_state_space_b200 import _native as N
from quantized_state_space_b200 import api

pytestmark = pytest.mark.gpu

V_TOL = 2.0 ** -19  # as in the norm's own tests


@pytest.mark.parametrize("d", [24, 29, 250, 256, 1000, 2049, 5120])
@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-12])
def test_overflowing_values(d, size):
    """Small tokens (their multiple by rstd overflows, the product with the weight does
    not) and ordinary ones (the product does)."""
    gen = torch.Generator().manual_seed(d)
    x = torch.randn(9, d, generator=gen) * size
    w = torch.ones(d)
    w[::7] = 3e38
    x[4, ::7] = 0  # a token of ordinary values among them
    st = status_word()
    codes, scales, y = api.rms_norm_quantize(x.to(dev()), w.to(dev()), eps=0.0, want_y=True,
                                             status=st)
    r = x.double()
    v = r / torch.sqrt((r * r).mean(-1, keepdim=True)) * w.double()
    top = torch.finfo(torch.float32).max
    # (values within the tolerance of the border may fall on either side: none does)
    assert not ((v.abs() > top * (1 - V_TOL)) & (v.abs() < top * (1 + V_TOL))).any()
    inf = v.abs() > top
    # r w overflows before the multiplication by rstd <= 1 where the token is large
    assert inf.any()
    wide = (r * w.double()).abs() > top
    inf = inf | wide
    finite = torch.where(inf, torch.zeros_like(v), v)
    s = finite.abs().amax(-1) / 127
    sc, q = scales.cpu().double(), codes.cpu().double()
    assert ((sc - s).abs() <= V_TOL * s).all() and (sc > 0).all()
    off = (q * sc[:, None] - finite).abs()
    assert (off <= (0.5 + 2.0 ** -11) * sc[:, None]).all()
    assert not codes.cpu()[inf].any()
    assert int(st) == N.DEV_NONFINITE
    assert torch.isinf(y.cpu())[inf].all() and torch.isfinite(y.cpu())[~inf].all()
