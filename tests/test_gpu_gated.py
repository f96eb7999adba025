"""The gated recurrence on the GPU (scan, gradient, one-token update) against
the formula in 64 bits and against differences.

Tolerances come from running error recurrences beside the 64-bit values:
sigmoid's smaller half s has relative error below e(g) = 2^-21 + |g| 2^-23
(argument |g| log2 e: two half-ulps of |g|; ex2 2^-22; 1 + e 2^-24; reciprocal
2^-23; product 2^-24), the larger half the same absolute error plus 2^-25.  A
step of the recurrence then adds at most s e(g) (|h| + |v|) + 3 * 2^-24 (|h_{t-1}| f
+ |n v|) and multiplies the earlier error by f; the composed maps of segments
repeat these roundings once more (factor 2).  An output adds half a step of
its type.
"""
import numpy as np
import pytest
import torch

from gpu_util import dev
from quantized_state_space_b200 import _native as N
from quantized_state_space_b200 import api

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = 2.0 ** -24


def sig(x):
    return 0.5 * (1 + np.tanh(0.5 * x))


def small_err(g):
    """Absolute error of f and n."""
    g = np.clip(g, -80, 80)
    s = 1 / (1 + np.exp(np.abs(g)))
    return s * (2.0 ** -21 + np.abs(g) * 2.0 ** -23) + 2.0 ** -25


def silu_err(z):
    """Relative error of z sigmoid(z)."""
    return 2.0 ** -21 + np.minimum(np.abs(z), 80) * 2.0 ** -23


class Ref:
    """64-bit forward and backward with error bounds of the binary32 path."""

    def __init__(self, v, g, z=None, h0=None, lengths=None, dy=None, dh=None):
        f64 = lambda t: None if t is None else t.detach().cpu().double().numpy()
        self.dtype = v.dtype
        v, g, z, h0, dy, dh = map(f64, (v, g, z, h0, dy, dh))
        b, L, d = v.shape
        ends = [L] * b if lengths is None else [min(max(int(n), 0), L) for n in lengths]
        live = np.arange(L)[None, :, None] < np.array(ends)[:, None, None]
        f = np.where(live, 1 / (1 + np.exp(-np.clip(g, -700, 700))), 1.0)
        n = np.where(live, 1 / (1 + np.exp(np.clip(g, -700, 700))), 0.0)
        df = np.where(live, small_err(g), 0.0)
        v = np.where(live, v, 0.0)
        h = np.zeros((b, L + 1, d))
        e = np.zeros((b, L + 1, d))
        if h0 is not None:
            h[:, 0] = h0
        for t in range(L):
            h[:, t + 1] = f[:, t] * h[:, t] + n[:, t] * v[:, t]
            mag = f[:, t] * np.abs(h[:, t]) + np.abs(n[:, t] * v[:, t])
            e[:, t + 1] = f[:, t] * e[:, t] + 2 * live[:, t] * (
                df[:, t] * (np.abs(h[:, t]) + np.abs(v[:, t])) + 3 * U * mag)
        self.h_final, self.h_err = h[:, L], e[:, L] + 1e-30
        self.h, self.h_all_err = h, e
        y, ye = h[:, 1:], e[:, 1:]
        if z is not None:
            z = np.where(live, z, 0.0)
            sz = z * sig(z)
            ye = ye * np.abs(sz) + np.abs(y * sz) * (silu_err(z) + U)
            y = y * sz
        self.y, self.y_err = y * live, ye
        if dy is None and dh is None:
            return
        dy = np.zeros_like(v) if dy is None else np.where(live, dy, 0.0)
        into, ie = dy, np.zeros_like(dy)
        if z is not None:
            into = dy * sz
            ie = np.abs(into) * (silu_err(z) + U)
        c = np.zeros((b, d)) if dh is None else dh
        ce = np.zeros((b, d))
        self.dv, self.dg = np.zeros_like(v), np.zeros_like(v)
        self.dv_err, self.dg_err = np.zeros_like(v), np.zeros_like(v)
        for t in range(L - 1, -1, -1):
            lam = into[:, t] + c
            # (sums of segments cancel no better than their terms: count magnitudes)
            le = ie[:, t] + ce + 2 * 2 * U * (np.abs(into[:, t]) + np.abs(c))
            al = np.abs(lam) + le
            self.dv[:, t] = n[:, t] * lam
            self.dv_err[:, t] = n[:, t] * le + df[:, t] * al + U * n[:, t] * al
            w = h[:, t] - v[:, t]
            we = e[:, t] + U * np.abs(w)
            fn = f[:, t] * n[:, t]
            # f n: the smaller half's absolute error, the larger is at most 1
            self.dg[:, t] = fn * w * lam
            self.dg_err[:, t] = (fn * (we * al + np.abs(w) * le) +
                                 (2 * df[:, t] * np.maximum(f[:, t], n[:, t]) + 3 * U * fn)
                                 * np.abs(w) * al)
            c = f[:, t] * lam
            ce = f[:, t] * le + df[:, t] * al + 2 * U * np.abs(c)
        self.dv *= live
        self.dg *= live
        self.dh0, self.dh0_err = c, ce + 1e-30
        if z is not None:
            s = sig(z)
            self.dz = dy * h[:, 1:] * (s * (1 + z * (1 - s)))
            self.dz_err = (np.abs(dy) * e[:, 1:] * (1 + np.abs(z)) +
                           np.abs(dy * h[:, 1:]) * (1 + np.abs(z)) ** 2 * 2.0 ** -20)

    def close(self, name, got):
        want, err = getattr(self, name), getattr(self, name + "_err")
        got_np = got.detach().cpu().double().numpy()
        tol = 2 * err
        if got.dtype != F32 or name in ("y", "dv", "dg", "dz"):
            fi = torch.finfo(got.dtype)
            tol = tol + fi.eps / 2 * (np.abs(want) + 2 * err) + fi.tiny * fi.eps
        bad = np.abs(got_np - want) > tol
        assert not bad.any(), (name, np.argwhere(bad)[:3].tolist(), got_np[bad][:3], want[bad][:3],
                               tol[bad][:3])


def problem(seed, b, L, d, dtype, z=True, h0=True, lengths=None, gmean=2.0, strided=True):
    gen = torch.Generator().manual_seed(seed)
    parts = 3 if z else 2
    # (the last 3 columns make row strides odd; strided=False: separate tensors)
    proj = torch.randn(b, L, parts * d + (3 if strided else 0), generator=gen)
    proj[..., d:2 * d] = proj[..., d:2 * d] * 1.5 + gmean
    proj = proj.to(dtype).to(dev())
    v, g = proj[..., :d], proj[..., d:2 * d]
    zz = proj[..., 2 * d:3 * d] if z else None
    if not strided:
        v, g, zz = v.contiguous(), g.contiguous(), zz.contiguous() if z else None
    p = dict(v=v, g=g, z=zz, h0=torch.randn(b, d, generator=gen).to(dev()) if h0 else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32,
                                                               device=dev()))
    p["dy"] = torch.randn(b, L, d, generator=gen).to(dtype).to(dev())
    p["dh"] = torch.randn(b, d, generator=gen).to(dev())
    return p


def check_all(p):
    y, h, states = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"], lengths=p["lengths"],
                                  save_states=True)
    dv, dg, dz, dh0 = api.gated_scan_backward(p["dy"], p["v"], p["g"], states, z=p["z"],
                                              dh_final=p["dh"], lengths=p["lengths"])
    r = Ref(p["v"], p["g"], p["z"], p["h0"],
            None if p["lengths"] is None else p["lengths"].tolist(), p["dy"], p["dh"])
    r.close("y", y)
    got = h.cpu().double().numpy()
    assert (np.abs(got - r.h_final) <= 2 * r.h_err).all()
    st = states.cpu().double().numpy()
    k = N.ssmq_gated_scan_state_steps()
    assert (np.abs(st - r.h[:, :-1][:, ::k]) <= 2 * r.h_all_err[:, :-1][:, ::k] + 1e-30).all()
    r.close("dv", dv)
    r.close("dg", dg)
    if p["z"] is not None:
        r.close("dz", dz)
    else:
        assert dz is None
    r.close("dh0", dh0)
    return y, h


SIZES = [(1, 1, 1), (2, 1, 64), (1, 2, 3), (2, 7, 33), (3, 64, 64), (2, 65, 66), (1, 129, 130),
         (1, 255, 16), (2, 1000, 48), (1, 2600, 16), (1, 2309, 7), (4, 513, 200), (300, 9, 40)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_scan_and_gradient(size, z, dtype):
    b, L, d = size
    check_all(problem(L * 31 + d, b, L, d, dtype, z=z, strided=d % 2 == 1))


@pytest.mark.parametrize("size", [(4, 700, 2560), (1, 300, 9600), (10, 130, 4097)])
def test_wide_layers(size):
    """Wide channel blocks with and without clusters over several rounds."""
    b, L, d = size
    check_all(problem(5, b, L, d, BF16 if d % 2 else F16, z=d % 2 == 0, strided=False))


@pytest.mark.parametrize("size,strided", [((5, 300, 24), False), ((5, 300, 25), True),
                                          ((3, 900, 320), True)])
def test_lengths(size, strided):
    """Padded batches: empty, one-step, full and out-of-range lengths; what is
    behind a sequence's end is not read."""
    b, L, d = size
    lengths = [0, L, 1, 137, -4][:b - 1] + [L + 9]
    p = problem(11, b, L, d, F32, lengths=lengths, strided=strided)
    for i, n in enumerate(lengths):
        n = min(max(n, 0), L)
        for t in (p["v"], p["g"], p["z"], p["dy"]):
            t[i, n:] = float("nan") if i % 2 else float("inf")
    y, h = check_all(p)
    for i, n in enumerate(lengths):
        assert not y[i, min(max(n, 0), L):].any()
    assert torch.equal(h[0], p["h0"][0])


def test_defaults_and_empty():
    p = problem(12, 2, 50, 10, F32, h0=False)
    y, h = api.gated_scan(p["v"], p["g"])
    r = Ref(p["v"], p["g"])
    r.close("y", y)
    assert api.gated_scan(p["v"], p["g"], return_state=False)[1] is None
    h0 = torch.randn(2, 10, device=dev())
    e = p["v"][:, :0]
    y, h, st = api.gated_scan(e, e, h0=h0, save_states=True)
    assert y.shape == (2, 0, 10) and torch.equal(h, h0) and st.shape == (2, 0, 10)
    _, _, _, dh0 = api.gated_scan_backward(e, e, e, st, dh_final=h0)
    assert torch.equal(dh0, h0)
    y, h = api.gated_scan(p["v"][:0], p["g"][:0])
    assert y.shape == (0, 50, 10) and h.shape == (0, 10)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_extreme_gates(dtype):
    """g = -inf forgets (a new sequence), g = +inf keeps; long memories."""
    p = problem(13, 2, 400, 32, dtype, gmean=6.0)
    p["g"][:, 100] = -float("inf")
    p["g"][:, 200:260] = float("inf")
    y, h = check_all(p)
    y2, _ = api.gated_scan(p["v"][:, 100:], p["g"][:, 100:], z=p["z"][:, 100:])
    r = Ref(p["v"][:, 100:], p["g"][:, 100:], p["z"][:, 100:])
    r.close("y", y2)
    r.close("y", y[:, 100:])


def test_split_calls_chain():
    """A sequence cut anywhere: the second call starts from the first's state."""
    p = problem(14, 2, 333, 70, F32)
    y, h = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"])
    r = Ref(p["v"], p["g"], p["z"], p["h0"])
    for cut in (1, 64, 100, 332):
        ya, ha = api.gated_scan(p["v"][:, :cut], p["g"][:, :cut], z=p["z"][:, :cut], h0=p["h0"])
        yb, hb = api.gated_scan(p["v"][:, cut:], p["g"][:, cut:], z=p["z"][:, cut:], h0=ha,
                                h_final=ha)  # (in place on the state)
        assert hb.data_ptr() == ha.data_ptr()
        r.close("y", torch.cat((ya, yb), 1))
        assert (np.abs(hb.cpu().double().numpy() - r.h_final) <= 2 * r.h_err).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("b,d", [(1, 1), (3, 64), (64, 520), (5, 333), (1, 8192)])
@pytest.mark.parametrize("z", [False, True])
def test_update(b, d, z, dtype):
    """Single tokens: equal to the scan of one step within its bounds."""
    p = problem(15, b, 1, d, dtype, z=z, strided=d % 2 == 1)
    state = p["h0"].clone()
    args = [p["v"][:, 0], p["g"][:, 0]]
    y = api.gated_update(state, *args, z=p["z"][:, 0] if z else None)
    r = Ref(p["v"], p["g"], p["z"], p["h0"])
    r.close("y", y[:, None])
    assert (np.abs(state.cpu().double().numpy() - r.h_final) <= 2 * r.h_err).all()
    if z:  # in place on z
        zz = p["z"][:, 0].clone()
        s2 = p["h0"].clone()
        y2 = api.gated_update(s2, *args, z=zz, y=zz)
        assert torch.equal(y2, y) and torch.equal(s2, state)


def test_in_place_outputs():
    p = problem(16, 2, 300, 64, BF16, strided=False)
    y, h, st = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"], save_states=True)
    ref = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"], dh_final=p["dh"])
    zy = p["z"].clone()
    y2, _ = api.gated_scan(p["v"], p["g"], z=zy, h0=p["h0"], y=zy)
    assert torch.equal(y2, y)
    v, g, z, dy, dh = (p[k].clone() for k in ("v", "g", "z", "dy", "dh"))
    got = api.gated_scan_backward(dy, v, g, st, z=z, dh_final=dh, dv=dy, dg=g, dz=z, dh0=dh)
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    # gradients as column slices of the projection's gradient
    wide = torch.full((2, 300, 3 * 64), 5.0, dtype=BF16, device=dev())
    got = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"], dh_final=p["dh"],
                                  dv=wide[..., :64], dg=wide[..., 64:128], dz=wide[..., 128:])
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """Central differences of the 64-bit formula, step 1e-4: their error is
    below 1e-7 (third derivatives of order 1), far below the tolerance."""
    p = problem(17, 2, 9, 3, F32, strided=False)
    _, _, st = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"], save_states=True)
    grads = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"], dh_final=p["dh"])

    def loss(q):
        f = torch.sigmoid(q["g"])
        h, total = q["h0"], 0.0
        for t in range(9):
            h = f[:, t] * h + (1 - f[:, t]) * q["v"][:, t]
            z = q["z"][:, t]
            total = total + (p64["dy"][:, t] * h * z * torch.sigmoid(z)).sum()
        return float(total + (p64["dh"] * h).sum())

    p64 = {k: t.cpu().double() for k, t in p.items() if t is not None}
    for name, grad in zip(("v", "g", "z", "h0"), grads):
        flat = p64[name].reshape(-1)
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + 1e-4
            up = loss(p64)
            flat[i] = keep - 1e-4
            down = loss(p64)
            flat[i] = keep
            assert abs((up - down) / 2e-4 - float(grad.reshape(-1)[i])) < 2e-5, (name, i)


def test_autograd():
    p = problem(18, 2, 100, 20, F32, strided=False)
    leaves = [p[k].clone().requires_grad_() for k in ("v", "g", "z")]
    h0 = p["h0"][:1].clone().requires_grad_()  # one start state for all sequences
    y, h = api.gated_scan(*leaves[:2], z=leaves[2], h0=h0.expand(2, -1).contiguous())
    grads = torch.autograd.grad((y, h), leaves + [h0], (p["dy"], p["dh"]))
    _, _, st = api.gated_scan(p["v"], p["g"], z=p["z"],
                              h0=p["h0"][:1].expand(2, -1).contiguous(), save_states=True)
    ref = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"], dh_final=p["dh"])
    for a, b in zip(grads[:3], ref[:3]):
        assert torch.equal(a, b)
    assert torch.equal(grads[3], ref[3].sum(0, keepdim=True))
    # an expanded gradient, and outputs that are not used
    y, h = api.gated_scan(*leaves[:2], z=leaves[2])
    y.sum().backward()
    ones = torch.ones_like(p["dy"])
    _, _, st = api.gated_scan(p["v"], p["g"], z=p["z"], save_states=True)
    ref = api.gated_scan_backward(ones, p["v"], p["g"], st, z=p["z"])
    assert torch.equal(leaves[0].grad, ref[0]) and torch.equal(leaves[1].grad, ref[1])
    with pytest.raises(ValueError):
        api.gated_scan(*leaves[:2], y=torch.empty_like(p["v"]))


def test_repeatable_streams_and_graph():
    p = problem(19, 3, 1500, 96, F16)
    kw = dict(z=p["z"], h0=p["h0"])

    def both():
        y, h, st = api.gated_scan(p["v"], p["g"], save_states=True, **kw)
        return (y, h) + api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"],
                                                dh_final=p["dh"])

    ref = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = both()
    for t in captured:
        t.zero_()
    g.replay()
    again = both()  # eager beside the graph
    torch.cuda.synchronize()
    for a, b, c, e in zip(ref, other, captured, again):
        assert torch.equal(a, b) and torch.equal(a, c) and torch.equal(a, e)


@pytest.mark.parametrize("d", [64, 50, 33])
def test_layouts(d):
    """Time-major tensors, inputs shared by the batch (batch stride 0) and
    single-row tensors with odd strides give the contiguous call's values."""
    p = problem(22, 3, 200, d, F16, strided=False)
    ref = Ref(p["v"], p["g"], p["z"], p["h0"], None, p["dy"], p["dh"])
    tm = {k: p[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("v", "g", "z", "dy")}
    y = torch.empty_like(tm["v"])
    y, h, st = api.gated_scan(tm["v"], tm["g"], z=tm["z"], h0=p["h0"], y=y, save_states=True)
    ref.close("y", y)
    for name, t in zip(("dv", "dg", "dz", "dh0"), api.gated_scan_backward(
            tm["dy"], tm["v"], tm["g"], st, z=tm["z"], dh_final=p["dh"])):
        ref.close(name, t)
    shared = {k: p[k][:1].expand(3, -1, -1) for k in ("v", "g", "z")}
    ref = Ref(shared["v"], shared["g"], shared["z"], p["h0"], None, p["dy"], p["dh"])
    y, h, st = api.gated_scan(shared["v"], shared["g"], z=shared["z"], h0=p["h0"],
                              save_states=True)
    ref.close("y", y)
    for name, t in zip(("dv", "dg", "dz", "dh0"), api.gated_scan_backward(
            p["dy"], shared["v"], shared["g"], st, z=shared["z"], dh_final=p["dh"])):
        ref.close(name, t)
    one = {k: torch.as_strided(p[k], (1, 1, d), (7, 1, 1)) for k in ("v", "g")}
    y, _ = api.gated_scan(one["v"], one["g"])
    Ref(one["v"], one["g"]).close("y", y)


def test_broadcast_leaves_sum_their_gradients():
    """A leaf shared by the batch gets the sum of the sequences' gradients."""
    p = problem(23, 4, 90, 24, F32, strided=False)
    v, g = p["v"][:1].clone().requires_grad_(), p["g"][:1].clone().requires_grad_()
    z = p["z"].clone().requires_grad_()
    y, h = api.gated_scan(v.expand(4, -1, -1), g.expand(4, -1, -1), z=z)
    got = torch.autograd.grad(y, (v, g, z), p["dy"])
    ev, eg = p["v"][:1].expand(4, -1, -1), p["g"][:1].expand(4, -1, -1)
    _, _, st = api.gated_scan(ev, eg, z=p["z"], save_states=True)
    ref = api.gated_scan_backward(p["dy"], ev, eg, st, z=p["z"])
    assert torch.equal(got[0], ref[0].sum(0, keepdim=True))
    assert torch.equal(got[1], ref[1].sum(0, keepdim=True)) and torch.equal(got[2], ref[2])


def test_status_stays_clear():
    st = torch.zeros(1, dtype=torch.int32, device=dev())
    p = problem(24, 2, 700, 64, F16)
    _, _, states = api.gated_scan(p["v"], p["g"], z=p["z"], save_states=True, status=st)
    api.gated_scan_backward(p["dy"], p["v"], p["g"], states, z=p["z"], status=st)
    assert int(st) == 0


def test_first_call_of_a_thread():
    """A thread that has made no CUDA call yet gets the same bytes: the same
    kernels run (tensor maps need the thread's context)."""
    import threading
    p = problem(21, 2, 700, 64, F16, strided=False)
    q = torch.randint(-127, 128, (300, 256), dtype=torch.int8, device=dev())
    s = torch.rand(300, device=dev())
    calls = [lambda: api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"]),
             lambda: [api.int8_linear(q, s, q, s)],
             lambda: api.rms_norm_quantize(p["v"])]
    for call in calls:
        ref, got = call(), []
        torch.cuda.synchronize()
        t = threading.Thread(target=lambda: got.extend(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert len(got) == len(ref) and all(torch.equal(a, b) for a, b in zip(got, ref))


def test_offsets_past_32_bits():
    """Rows more than 2^32 elements from the base (a long projection buffer)."""
    L, d = 70, 16
    stride = (1 << 26) + 8
    buf = torch.zeros(stride * L + 64, dtype=F16, device=dev())
    p = problem(20, 1, L, d, F16, z=False, strided=False)
    v = torch.as_strided(buf, (1, L, d), (0, stride, 1))
    g = torch.as_strided(buf, (1, L, d), (0, stride, 1), storage_offset=d)
    v.copy_(p["v"])
    g.copy_(p["g"])
    y, h = api.gated_scan(v, g, h0=p["h0"], y=torch.as_strided(buf, (1, L, d), (0, stride, 1),
                                                               storage_offset=2 * d))
    r = Ref(p["v"], p["g"], None, p["h0"])
    r.close("y", y)
