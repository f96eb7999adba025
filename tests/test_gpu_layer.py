"""The quantized-layer operators in a row, as a W8A8 layer uses them: residual
add + norm + codes, int8 projection to (v | g | z), gated recurrence over the
column slices, norm + codes, int8 projection back; in prefill, for one more
token, from a captured graph, and behind the SSD scan."""
import numpy as np
import pytest
import torch

from gpu_util import T, dev
from problems import ssd_problem
from quantized_state_space_b200 import api
from test_gpu_gated import Ref
from test_gpu_linear import check as check_linear
from test_gpu_norm import check as check_norm

pytestmark = pytest.mark.gpu


class Layer:
    """Weights quantized once by the group quantizer, one scale per row."""

    def __init__(self, model, inner, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.dtype, self.inner = dtype, inner
        self.norm1 = (torch.rand(model, generator=g) + 0.5).to(dev())
        self.norm2 = (torch.rand(inner, generator=g) + 0.5).to(dev())
        self.bias = torch.cat((torch.zeros(inner), torch.full((inner,), 2.0),
                               torch.zeros(inner))).to(dev())
        self.w_in, self.s_in = self.quantize(torch.randn(3 * inner, model, generator=g) / model ** 0.5)
        self.w_out, self.s_out = self.quantize(torch.randn(model, inner, generator=g) / inner ** 0.5)

    @staticmethod
    def quantize(w):
        rows, cols = w.shape
        return api.quantize_groups(w.contiguous().to(dev()), 1, rows, cols,
                                   torch.arange(rows, dtype=torch.int32, device=dev()), rows,
                                   absmax=True)

    def _slices(self, proj):
        d = self.inner
        return proj[..., :d], proj[..., d:2 * d], proj[..., 2 * d:]

    def __call__(self, x, residual, h0=None, lengths=None, keep=None):
        """x, residual (b, L, model), or (b, model) for one token on the state h0."""
        codes, scales, res = api.rms_norm_quantize(x, self.norm1, residual=residual)
        proj = api.int8_linear(codes, scales, self.w_in, self.s_in, bias=self.bias,
                               dtype=self.dtype)
        v, g, z = self._slices(proj)
        if x.dim() == 2:
            y, h = api.gated_update(h0, v, g, z=z), h0
        else:
            y, h = api.gated_scan(v, g, z=z, h0=h0, lengths=lengths)
        codes2, scales2 = api.rms_norm_quantize(y, self.norm2)
        out = api.int8_linear(codes2, scales2, self.w_out, self.s_out, dtype=self.dtype)
        if keep is not None:
            keep.update(codes=codes, scales=scales, res=res, proj=proj, y=y, codes2=codes2,
                        scales2=scales2)
        return out, res, h


def inputs(b, L, model, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(b, L, model, generator=g).to(dtype).to(dev()),
            torch.randn(b, L, model, generator=g).to(dtype).to(dev()))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("b,L,model,inner", [(2, 200, 256, 512), (3, 33, 100, 76),
                                             (1, 1500, 1024, 1280)])
def test_prefill(b, L, model, inner, dtype):
    """Every stage against its formula in 64 bits, on the stage before's output."""
    layer = Layer(model, inner, dtype)
    x, res = inputs(b, L, model, dtype)
    k = {}
    out, r, h = layer(x, res, keep=k)
    check_norm(x.cpu(), layer.norm1.cpu(), res.cpu(), 1e-5, k["codes"], k["scales"], r)
    flat = lambda t: t.reshape(-1, t.shape[-1])
    check_linear(flat(k["proj"]), dict(x=flat(k["codes"]), w=layer.w_in, xs=k["scales"].reshape(-1),
                                       ws=layer.s_in, bias=layer.bias))
    v, g, z = layer._slices(k["proj"])
    ref = Ref(v, g, z)
    ref.close("y", k["y"])
    assert (np.abs(h.cpu().double().numpy() - ref.h_final) <= 2 * ref.h_err).all()
    check_norm(k["y"].cpu(), layer.norm2.cpu(), None, 1e-5, k["codes2"], k["scales2"])
    check_linear(flat(out), dict(x=flat(k["codes2"]), w=layer.w_out, xs=k["scales2"].reshape(-1),
                                 ws=layer.s_out, bias=None))


@pytest.mark.parametrize("b,L,model,inner", [(4, 130, 256, 512), (2, 70, 100, 76)])
def test_next_token(b, L, model, inner):
    """One more token on the prefill's state: the row-wise stages give the bytes
    of the longer prefill, the recurrence its values within the bounds."""
    dtype = torch.float16
    layer = Layer(model, inner, dtype)
    x, res = inputs(b, L + 1, model, dtype)
    full = {}
    layer(x, res, keep=full)
    _, _, h = layer(x[:, :L].contiguous(), res[:, :L].contiguous())
    one = {}
    _, r, h = layer(x[:, L], res[:, L], h0=h, keep=one)
    assert torch.equal(one["codes"], full["codes"][:, L])
    assert torch.equal(one["scales"], full["scales"][:, L])
    assert torch.equal(one["proj"], full["proj"][:, L]) and torch.equal(r, full["res"][:, L])
    ref = Ref(*layer._slices(full["proj"]))
    last = ref.y[:, L], ref.y_err[:, L]
    got = one["y"].cpu().double().numpy()
    assert (np.abs(got - last[0]) <= 2 * last[1] + 2.0 ** -11 * np.abs(last[0]) + 2.0 ** -25).all()
    assert (np.abs(h.cpu().double().numpy() - ref.h_final) <= 2 * ref.h_err).all()


def test_padded_batch():
    """A padded batch gives each sequence the bytes it has alone (the recurrence
    within its bounds), and the rows behind the ends do not matter."""
    layer = Layer(128, 96, torch.float16)
    x, res = inputs(3, 90, 128, torch.float16)
    ends = [90, 31, 0]
    lengths = torch.tensor(ends, dtype=torch.int32, device=dev())
    k = {}
    _, _, h = layer(x, res, lengths=lengths, keep=k)
    for i, n in enumerate(ends):
        assert not k["y"][i, n:].any() and not k["codes2"][i, n:].any()
        if n:
            a = {}
            _, _, hi = layer(x[i:i + 1, :n].contiguous(), res[i:i + 1, :n].contiguous(), keep=a)
            assert torch.equal(a["proj"], k["proj"][i:i + 1, :n])
            ref = Ref(*layer._slices(a["proj"]))
            ref.close("y", k["y"][i:i + 1, :n])
            assert (np.abs(h[i:i + 1].cpu().double().numpy() - ref.h_final) <= 2 * ref.h_err).all()
        else:
            assert not h[i].any()


def test_generation_from_a_graph():
    """Tokens through a captured step equal eager ones, byte for byte."""
    b, model, inner = 8, 256, 512
    layer = Layer(model, inner, torch.bfloat16)
    x, res = inputs(b, 5, model, torch.bfloat16)
    h0 = torch.randn(b, inner, device=dev())
    eager, h = [], h0.clone()
    for t in range(5):
        out, r, h = layer(x[:, t], res[:, t], h0=h)
        eager.append((out, r))
    xs, rs, hs = x[:, 0].clone(), res[:, 0].clone(), h0.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(xs, rs, h0=hs.clone())
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, r, _ = layer(xs, rs, h0=hs)
    hs.copy_(h0)
    for t in range(5):
        xs.copy_(x[:, t])
        rs.copy_(res[:, t])
        graph.replay()
        assert torch.equal(out, eager[t][0]) and torch.equal(r, eager[t][1])
    assert torch.equal(hs, h)


def test_behind_the_ssd_scan():
    """The gated SSD output through the block's norm and output projection."""
    b, L, H, P = 2, 130, 4, 64
    p = ssd_problem(970, b, L, H, P, 128, G=1, gs=8, gate=True)
    y, _ = api.ssd_chunk_scan(T(p["x"]), T(p["dt"]), T(p["A"]), T(p["B"]), T(p["C"]),
                              T(p["B_scale"]), T(p["C_scale"]), 8, x_group=T(p["x_group"]),
                              x_scale=T(p["x_scale"]), D=T(p["D"]), z=T(p["z"]))
    y = y.view(b, L, H * P)
    w = torch.rand(H * P, device=dev()) + 0.5
    wq, ws = Layer.quantize(torch.randn(128, H * P) / (H * P) ** 0.5)
    codes, scales = api.rms_norm_quantize(y, w)
    check_norm(y.cpu(), w.cpu(), None, 1e-5, codes, scales)
    out = api.int8_linear(codes, scales, wq, ws)
    check_linear(out.view(-1, 128), dict(x=codes.view(-1, H * P), w=wq, xs=scales.view(-1), ws=ws,
                                         bias=None))


def test_training_step_through_the_projection():
    """Gradients of the recurrence reach the projection's output (one tensor,
    three column slices) and match the explicit call's."""
    b, L, d = 2, 150, 40
    g = torch.Generator().manual_seed(3)
    proj = torch.randn(b, L, 3 * d, generator=g).to(dev()).requires_grad_()
    dy = torch.randn(b, L, d, generator=g).to(dev())
    y, h = api.gated_scan(proj[..., :d], proj[..., d:2 * d], z=proj[..., 2 * d:])
    y.backward(dy)
    p = proj.detach()
    v, gg, z = p[..., :d], p[..., d:2 * d], p[..., 2 * d:]
    _, _, st = api.gated_scan(v, gg, z=z, save_states=True)
    wide = torch.empty_like(p)
    api.gated_scan_backward(dy, v, gg, st, z=z, dv=wide[..., :d], dg=wide[..., d:2 * d],
                            dz=wide[..., 2 * d:])
    ref = Ref(v, gg, z, None, None, dy)
    ref.close("dv", wide[..., :d])
    ref.close("dg", wide[..., d:2 * d])
    ref.close("dz", wide[..., 2 * d:])
    assert torch.equal(proj.grad, wide)


def test_operators_side_by_side():
    """Scans with clusters, gradients, CTA-pair and split products and norms on
    four streams at once give what they give alone."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3000, 1024, generator=g).half().to(dev())
    q = torch.randint(-127, 128, (3000, 1024), generator=g, dtype=torch.int8).to(dev())
    s = torch.rand(3000, generator=g).to(dev())
    p = torch.randn(2, 1500, 3 * 64, generator=g).half().to(dev())
    v, gg, z = p[..., :64], p[..., 64:128], p[..., 128:]
    _, _, st = api.gated_scan(v, gg, z=z, save_states=True)
    jobs = [lambda: api.rms_norm_quantize(x),
            lambda: (api.int8_linear(q, s, q, s), api.int8_linear(q[:5], s[:5], q, s)),
            lambda: api.gated_scan(v, gg, z=z),
            lambda: api.gated_scan_backward(z, v, gg, st, z=z)]
    refs = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[] for _ in jobs]
    for _ in range(8):
        for job, stream, out in zip(jobs, streams, outs):
            with torch.cuda.stream(stream):
                out.append(job())
    torch.cuda.synchronize()
    for ref, out in zip(refs, outs):
        for got in out:
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
