"""Gates at the ends of their range: a NaN logit makes the later states of its
channel NaN (and the gradients that pass through it), in every kernel of the
gated recurrence; g = -inf leaves nothing of the state, however large it is.

The comparison counts a NaN on one side alone as a difference.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev
from quantized_state_space_b200 import api
from test_gpu_gated import Ref, problem

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def agree(ref, name, got):
    """Ref.close with NaN required exactly where the formula has it."""
    want, err = getattr(ref, name), getattr(ref, name + "_err")
    x = got.detach().cpu().double().numpy()
    tol = 2 * err
    if name not in ("h_final", "dh0"):
        fi = torch.finfo(got.dtype)
        tol = tol + fi.eps / 2 * (np.abs(want) + 2 * err) + fi.tiny * fi.eps
    ok = (np.abs(x - want) <= tol) | (np.isnan(x) & np.isnan(want))
    assert ok.all(), (name, np.argwhere(~ok)[:3].tolist(), x[~ok][:3], want[~ok][:3])


def reference(p):
    r = Ref(p["v"], p["g"], p["z"], p["h0"],
            None if p["lengths"] is None else p["lengths"].tolist(), p["dy"], p["dh"])
    r.h_final_err = r.h_err
    return r


def run_and_agree(p):
    y, h, st = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"], lengths=p["lengths"],
                              save_states=True)
    grads = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"], dh_final=p["dh"],
                                    lengths=p["lengths"])
    r = reference(p)
    agree(r, "y", y)
    agree(r, "h_final", h)
    for name, t in zip(("dv", "dg", "dz", "dh0"), grads):
        if t is not None:
            agree(r, name, t)
    return r, y, h


# copies by TMA, by pairs, by single channels (odd widths and strides); wide and
# narrow channel blocks, with and without clusters along time
MODES = [((2, 300, 32), False), ((2, 300, 64), True), ((3, 200, 33), True), ((1, 1000, 48), False),
         ((4, 130, 2560), False), ((64, 70, 66), False)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("size,strided", MODES)
def test_nan_logit(size, strided, z, dtype):
    b, L, d = size
    p = problem(31, b, L, d, dtype, z=z, strided=strided)
    for i, (t, c) in enumerate([(0, 1), (L // 2, d // 2), (L - 1, d - 1)]):
        p["g"][i % b, t, c] = float("nan")
    r, y, h = run_and_agree(p)
    bad = np.isnan(r.y)
    assert bad.any() and not bad.all()
    assert torch.isnan(h).any() and torch.isfinite(h).any()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("d", [1, 8, 33, 64])
def test_nan_logit_of_one_token(d, dtype):
    p = problem(32, 3, 1, d, dtype)
    p["g"][1, 0, d // 2] = float("nan")
    state = p["h0"].clone()
    y = api.gated_update(state, p["v"][:, 0], p["g"][:, 0], z=p["z"][:, 0])
    r = reference(p)
    agree(r, "y", y[:, None])
    agree(r, "h_final", state)
    assert torch.isnan(state).sum() == 1 and torch.isnan(y).sum() == 1


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("size,strided", [((3, 300, 32), False), ((3, 300, 33), True)])
def test_nan_behind_a_sequence_is_not_read(size, strided, dtype):
    b, L, d = size
    lengths = [137, L, 0]
    p = problem(33, b, L, d, dtype, lengths=lengths, strided=strided)
    for i, n in enumerate(lengths):
        p["g"][i, n:] = float("nan")
    r, y, h = run_and_agree(p)
    assert torch.isfinite(y).all() and torch.isfinite(h).all()

@pytest.mark.parametrize("size,strided", MODES)
def test_minus_infinity_leaves_nothing(size, strided):
    """States beyond 2^100: 2^-126 of them would show."""
    b, L, d = size
    p = problem(34, b, L, d, F32, strided=strided)
    p["h0"].fill_(2.0 ** 126)
    p["g"][:, 0] = -float("inf")
    y, h = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"])
    assert torch.equal(*(api.gated_scan(p["v"], p["g"], z=p["z"], h0=h0)[0]
                         for h0 in (p["h0"], None)))
    r = Ref(p["v"], p["g"], p["z"])
    agree(r, "y", y)
    r.h_final_err = r.h_err
    agree(r, "h_final", h)
    _, _, st = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"], save_states=True)
    grads = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"], dh_final=p["dh"])
    assert not grads[3].any() and not grads[1][:, 0].any()  # f = 0: nothing reaches h0 or g


def test_minus_infinity_leaves_nothing_of_one_state():
    for d in (16, 33):
        p = problem(35, 4, 1, d, F32)
        p["g"].fill_(-float("inf"))
        state = torch.full((4, d), 2.0 ** 127, device=dev())
        y = api.gated_update(state, p["v"][:, 0], p["g"][:, 0])
        assert torch.equal(state, p["v"][:, 0]) and torch.equal(y, p["v"][:, 0])
