"""The quantized-layer operators and the gated recurrence where a wrong value could
hide: comparisons in which a NaN on one side is a difference, padded batches and
in-place outputs in every type and every way the kernels read their rows.  Tolerances
are those of the operators' own tests (derived there)."""
import pytest
import torch

from gpu_util import dev
from quantized_state_space_b200 import api
from test_gpu_gated import problem
from test_gpu_gated_gates import agree, reference, run_and_agree

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F16, BF16, F32]


def rows_of(t, pad):
    """The tensor in rows of its width + pad elements."""
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    return wide[..., :t.shape[-1]]


# pad 0 and 8: rows on 16 bytes (TMA); 2: even rows (pairs); 1: odd rows (single
# channels, in the gradient of 16-bit types words); odd widths
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 1, 2, 8])
@pytest.mark.parametrize("b,L,d", [(6, 300, 24), (6, 300, 25), (4, 130, 72), (3, 900, 320)])
def test_padded_batches(b, L, d, pad, dtype):
    """Empty, one-step, full and out-of-range lengths.  What lies behind a sequence's
    end is NaN or infinite and reaches nothing; y and the gradients there are 0."""
    lengths = ([0, L, 1, L // 2 + 3, -4, 64] * 2)[:b - 1] + [L + 9]
    p = problem(41, b, L, d, dtype, lengths=lengths, strided=False)
    for k in ("v", "g", "z", "dy"):
        p[k] = rows_of(p[k], pad)
    for i, n in enumerate(lengths):
        n = min(max(n, 0), L)
        for k in ("v", "g", "z", "dy"):
            p[k][i, n:] = float("nan") if i % 2 else float("inf")
    r, y, h = run_and_agree(p)
    st = api.gated_scan(p["v"], p["g"], z=p["z"], h0=p["h0"], lengths=p["lengths"],
                        save_states=True)[2]
    dv, dg, dz, dh0 = api.gated_scan_backward(p["dy"], p["v"], p["g"], st, z=p["z"],
                                              dh_final=p["dh"], lengths=p["lengths"])
    assert torch.isfinite(st).all()
    for i, n in enumerate(lengths):
        n = min(max(n, 0), L)
        for t in (y, dv, dg, dz):
            assert torch.isfinite(t[i]).all() and not t[i, n:].any()
        if n == 0:
            assert torch.equal(h[i], p["h0"][i]) and torch.equal(dh0[i], p["dh"][i])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 1, 2])
@pytest.mark.parametrize("z", [False, True])
@pytest.mark.parametrize("b,L,d", [(2, 300, 64), (3, 200, 33), (1, 2600, 48), (64, 130, 320)])
def test_in_place(b, L, d, z, pad, dtype):
    """y on z and every gradient on every input, against the same call with outputs of
    its own: the same bytes, and nothing between the rows is touched."""
    p = problem(42, b, L, d, dtype, z=z, strided=False)
    names = ["v", "g", "dy"] + (["z"] if z else [])
    kw = dict(h0=p["h0"])

    def fresh():
        out = {}
        for n in names:
            wide = torch.full((b, L, d + pad), 3.0, dtype=dtype, device=dev())
            wide[..., :d] = p[n]
            out[n] = wide
        return out, {n: t[..., :d] for n, t in out.items()}

    _, t = fresh()
    y, h, st = api.gated_scan(t["v"], t["g"], z=t.get("z"), save_states=True, y=fresh()[1]["v"],
                              **kw)
    _, o = fresh()
    ref = api.gated_scan_backward(t["dy"], t["v"], t["g"], st, z=t.get("z"), dh_final=p["dh"],
                                  dv=o["v"], dg=o["g"], dz=o.get("z"))
    r = reference(p)
    agree(r, "y", y)
    for name, got in zip(("dv", "dg", "dz", "dh0"), ref):
        if got is not None:
            agree(r, name, got)
    if z:
        wide, u = fresh()
        y2, _ = api.gated_scan(u["v"], u["g"], z=u["z"], y=u["z"], **kw)
        assert torch.equal(y2, y) and (wide["z"][..., d:] == 3).all()
    for shift in range(len(names)):
        on = names[shift:] + names[:shift]
        wide, u = fresh()
        dh = p["dh"].clone()
        got = api.gated_scan_backward(u["dy"], u["v"], u["g"], st, z=u.get("z"), dh_final=dh,
                                      dv=u[on[0]], dg=u[on[1]], dz=u[on[2]] if z else None, dh0=dh)
        for a, c in zip(ref, got):
            assert a is None or torch.equal(a, c)
        assert all((w[..., d:] == 3).all() for w in wide.values())


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_gates_and_inputs(dtype):
    """-inf and +inf logits, an infinite v that a closed gate ignores nowhere: NaN only
    where the formula has it."""
    p = problem(43, 2, 400, 32, dtype, gmean=6.0)
    p["g"][:, 100] = -float("inf")
    p["g"][:, 200:260] = float("inf")
    run_and_agree(p)


def test_norm_repeats_itself():
    """The same call gives the same bytes, and codes leave the nearest integer of the
    64-bit quotient only within 2^-11 of a tie."""
    gen = torch.Generator().manual_seed(44)
    for t, d, dtype in ((64, 4096, F16), (515, 2561, BF16), (300, 1000, F32)):
        x, res = (torch.randn(t, d, generator=gen).to(dtype).to(dev()) for _ in range(2))
        w = (1 + 0.1 * torch.randn(d, generator=gen)).to(dev())
        ref = api.rms_norm_quantize(x, w, residual=res)
        for _ in range(20):
            for a, c in zip(ref, api.rms_norm_quantize(x, w, residual=res)):
                assert torch.equal(a, c)
        r = ref[2].double()
        v = r / torch.sqrt((r * r).mean(-1, keepdim=True) + 1e-5) * w.double()
        q = v / (v.abs().amax(-1, keepdim=True) / 127)
        off = (ref[0].double() - q).abs()
        assert (off <= 0.5 + 2.0 ** -11).all()
