"""Autograd and the quantized-layer operators: a derivative is computed or refused,
never dropped.  The refusals come before anything else, so most need no GPU."""
import pytest
import torch
from torch.autograd import forward_ad

from quantized_state_space_b200 import api


def f32(*shape, grad=False):
    return torch.ones(*shape, requires_grad=grad)


CALLS = {
    "rms_norm_quantize": (lambda t: api.rms_norm_quantize(
        t["x"], t["weight"], residual=t["residual"], residual_out=t["residual_out"], y=t["y"]),
        dict(x=(4, 16), weight=(16,), residual=(4, 16), residual_out=(4, 16), y=(4, 16))),
    "int8_linear": (lambda t: api.int8_linear(
        torch.zeros(4, 16, dtype=torch.int8), t["x_scale"], torch.zeros(8, 16, dtype=torch.int8),
        t["w_scale"], bias=t["bias"], out=t["out"]),
        dict(x_scale=(4,), w_scale=(8,), bias=(8,), out=(4, 8))),
    "gated_update": (lambda t: api.gated_update(t["state"], t["v"], t["g"], z=t["z"], y=t["y"]),
                     dict(state=(4, 16), v=(4, 16), g=(4, 16), z=(4, 16), y=(4, 16))),
}


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, s) in CALLS.items() for n in s])
def test_gradients_are_refused(call, name):
    fn, shapes = CALLS[call]
    t = {n: f32(*s, grad=n == name) for n, s in shapes.items()}
    with pytest.raises(ValueError, match="%s defines no gradient" % call):
        fn(t)
    # without gradients, and under no_grad, the call goes on (to refuse CPU tensors)
    with pytest.raises(ValueError, match="CUDA|cuda"):
        fn({n: f32(*s) for n, s in shapes.items()})
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA|cuda"):
        fn(t)


@pytest.mark.parametrize("name", ["y", "h_final", "states"])
def test_scan_outputs_that_require_a_gradient(name):
    v = f32(1, 4, 16)
    with pytest.raises(ValueError, match="defines no gradient"):
        api.gated_scan(v, v, **{name: f32(1, 4, 16, grad=True)})


@pytest.mark.parametrize("call,name", [(c, n) for c, (_, s) in CALLS.items() for n in s])
def test_tangents_are_refused(call, name):
    fn, shapes = CALLS[call]
    with forward_ad.dual_level():
        t = {n: f32(*s) for n, s in shapes.items()}
        t[name] = forward_ad.make_dual(t[name], torch.ones_like(t[name]))
        for grad in (True, False):
            with torch.set_grad_enabled(grad), \
                    pytest.raises(ValueError, match="%s defines no forward-mode" % call):
                fn(t)


@pytest.mark.parametrize("name", ["v", "g", "z", "h0"])
def test_scan_tangents_are_refused(name):
    """For inputs that require a gradient as well."""
    for grad in (False, True):
        with forward_ad.dual_level():
            t = {n: f32(1, 4, 16, grad=grad) for n in ("v", "g", "z")}
            t["h0"] = f32(1, 16)
            t[name] = forward_ad.make_dual(t[name], torch.ones_like(t[name]))
            with pytest.raises(ValueError, match="gated_scan defines no forward-mode"):
                api.gated_scan(t["v"], t["g"], z=t["z"], h0=t["h0"])


@pytest.mark.parametrize("name", ["dy", "v", "g", "states", "z", "dh_final"])
def test_scan_backward_tangents_are_refused(name):
    with forward_ad.dual_level():
        t = {n: f32(1, 4, 16) for n in ("dy", "v", "g", "z")}
        t.update(states=f32(1, 1, 16), dh_final=f32(1, 16))
        t[name] = forward_ad.make_dual(t[name], torch.ones_like(t[name]))
        with pytest.raises(ValueError, match="gated_scan_backward defines no forward-mode"):
            api.gated_scan_backward(t["dy"], t["v"], t["g"], t["states"], z=t["z"],
                                    dh_final=t["dh_final"])


def writers():
    """(name, call, the tensors of the caller that it writes)"""
    from gpu_util import dev
    h = lambda *s: torch.ones(*s, device=dev())
    x, g, z, state, q, r = h(4, 16), h(4, 16), h(4, 16), h(4, 16), h(4, 16), h(4, 16)
    codes = torch.zeros(4, 16, dtype=torch.int8, device=dev())
    seq, zs, h0 = h(2, 8, 16), h(2, 8, 16), h(2, 16)
    st = api.gated_scan(seq, seq, save_states=True)[2]
    grads = [h(2, 8, 16) for _ in range(3)] + [h(2, 16)]
    sc, out = h(4), h(4, 4)
    return [
        ("residual in place", lambda: api.rms_norm_quantize(x, residual=r, residual_out=x), [x]),
        ("norm", lambda: api.rms_norm_quantize(r, y=q, codes=codes, scales=sc), [q, codes, sc]),
        ("product", lambda: api.int8_linear(codes, h(4), codes, h(4), out=out), [out]),
        ("scan on z", lambda: api.gated_scan(seq, seq, z=zs, y=zs, h0=h0, h_final=h0, states=st),
         [zs, h0, st]),
        ("gradient", lambda: api.gated_scan_backward(seq, seq, seq, st, z=h(2, 8, 16),
                                                     dv=grads[0], dg=grads[1], dz=grads[2],
                                                     dh0=grads[3]), grads),
        ("update on z", lambda: api.gated_update(state, x, g, z=z, y=z), [state, z]),
    ]


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(6))
def test_written_tensors_count_on(i):
    """A tensor that autograd saved and a call has written since is noticed."""
    from gpu_util import dev
    name, call, written = writers()[i]
    before = [t._version for t in written]
    w = [torch.ones(1, device=dev(), requires_grad=True) for _ in written]
    losses = [(a * t).sum() for a, t in zip(w, written) if t.is_floating_point()]
    call()
    for t, v in zip(written, before):
        assert t._version > v, name
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


@pytest.mark.gpu
def test_written_tensors_of_inference_mode():
    with torch.inference_mode():
        for _, call, _ in writers():
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 16), (2, 1, 16), (1, 2, 16), (32,)])
def test_start_state_of_any_shape(shape):
    """h0 of b d elements in any shape, as the call takes it, gets its gradient in
    that shape."""
    from gpu_util import dev
    gen = torch.Generator().manual_seed(1)
    v, g, h0 = (torch.randn(*s, generator=gen).to(dev()) for s in ((2, 8, 16), (2, 8, 16), (2, 16)))
    leaf = h0.reshape(shape).clone().requires_grad_()
    y, h = api.gated_scan(v, g, h0=leaf)
    y.sum().backward()
    st = api.gated_scan(v, g, h0=h0, save_states=True)[2]
    want = api.gated_scan_backward(torch.ones_like(v), v, g, st)[3]
    assert leaf.grad.shape == leaf.shape and torch.equal(leaf.grad.reshape(2, 16), want)
