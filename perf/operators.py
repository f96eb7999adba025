"""Cases that measure the quantized-layer operators and the gated recurrence.

Each case is one call (or, for training, one forward and its gradient) at the
sizes that a W8A8 recurrent layer meets:

  norm    residual add + root-mean-square norm + int8 codes, one scale a token
  linear  int8 matrix product, one scale a token and one a channel
  scan    gated linear recurrence over a sequence
  train   the same recurrence, outputs and gradients
  step    one token of the recurrence on a kept state

``run`` computes a case in its plain form (elementary torch operations in
binary32) or, where ``own`` is true, through the package's public calls.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # one generation step's tokens of a batch of 64 entering a layer of width 4096
        dict(name="norm decode", kind="norm", tokens=64, d=4096, dtype="f16", residual=True),
        # prefill of 4 x 4096 tokens at inner width 80 x 64
        dict(name="norm prefill", kind="norm", tokens=16384, d=5120, dtype="f16", residual=True),
        # a ragged batch of a training-precision stream, width not a multiple of anything
        dict(name="norm ragged", kind="norm", tokens=4099, d=2561, dtype="bf16", residual=True),
        # one token through an input projection
        dict(name="linear token", kind="linear", m=1, n=8192, k=4096, dtype="f16", bias=False),
        # generation for a batch of 64: 128 heads x 64 back to width 4096
        dict(name="linear decode", kind="linear", m=64, n=4096, k=8192, dtype="f16", bias=False),
        # prefill of 4 x 4096 tokens, inner width 80 x 64 to width 2560
        dict(name="linear prefill", kind="linear", m=16384, n=2560, k=5120, dtype="f16", bias=False),
        # a short prompt, output width odd, with a bias
        dict(name="linear ragged", kind="linear", m=777, n=1801, k=1536, dtype="bf16", bias=True),
        # prefill of the 130M-shaped layer: 8 x 2048 tokens, 1536 channels, gated output
        dict(name="scan prefill", kind="scan", b=8, l=2048, d=1536, dtype="f16", z=True,
             lengths=False),
        # one very long sequence of few channels
        dict(name="scan long", kind="scan", b=1, l=65536, d=256, dtype="bf16", z=False,
             lengths=False),
        # training of 4 x 4096 tokens at 80 x 64 channels
        dict(name="train prefill", kind="train", b=4, l=4096, d=5120, dtype="bf16", z=True,
             lengths=False),
        # training on a padded batch of odd sizes in binary32
        dict(name="train ragged", kind="train", b=5, l=1023, d=333, dtype="f32", z=True,
             lengths=True),
        # one generated token for a batch of 64, 128 x 64 channels
        dict(name="step decode", kind="step", b=64, d=8192, dtype="f16", z=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "linear", "scan", "train", "step"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    if kind == "norm":
        d = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            d = max(16, d // 16 * 16)
        tokens = _log(rng, 1, min(65536, 16384 * 5120 // d))
        return dict(kind=kind, tokens=tokens, d=d, dtype=dtype, residual=rng.random() < 0.7)
    if kind == "linear":
        k = _log(rng, 16, 8192)
        if rng.random() < 0.75:
            k = max(16, k // 16 * 16)
        n = _log(rng, 16, 16384)
        if rng.random() < 0.6:
            n = max(16, n // 16 * 16)
        m = _log(rng, 1, min(16384, max(2, 16384 * 2560 * 5120 // (n * k), 2)))
        return dict(kind=kind, m=m, n=n, k=k, dtype=dtype, bias=rng.random() < 0.5)
    if kind == "step":
        return dict(kind=kind, b=_log(rng, 1, 256), d=_log(rng, 16, 16384), dtype=dtype,
                    z=rng.random() < 0.5)
    l = _log(rng, 1, 65536)
    d = _log(rng, 8, min(8192, 4 * 4096 * 5120 // l))
    b = _log(rng, 1, max(1, min(64, 4 * 4096 * 5120 // 2 // (l * d))))
    if kind == "train" and l > 16384:
        kind = "scan"
    return dict(kind=kind, b=b, l=l, d=d, dtype=dtype, z=rng.random() < 0.5,
                lengths=rng.random() < 0.4)


def _codes(gen, rows, cols, dev):
    """int8 codes as a per-row quantizer leaves them: a row's largest is +-127."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    s = x.abs().amax(1, keepdim=True) / 127
    return torch.round(x / s).to(torch.int8), s[:, 0].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(1_000_003 * (seed + 1))
    kind, dt = case["kind"], DTYPES[case["dtype"]]

    def normal(*shape, mean=0.0, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * std + mean

    if kind == "norm":
        x = normal(case["tokens"], case["d"])
        # a few channels carry outliers, as the residual stream of a trained model does
        x *= 1 + 20 * (torch.rand(case["d"], generator=gen, device=dev) < 0.002)
        return dict(case=case, x=x.to(dt), w=normal(case["d"], mean=1.0, std=0.1),
                    residual=normal(case["tokens"], case["d"]).to(dt) if case["residual"] else None)
    if kind == "linear":
        xq, xs = _codes(gen, case["m"], case["k"], dev)
        wq, ws = _codes(gen, case["n"], case["k"], dev)
        return dict(case=case, xq=xq, xs=xs, wq=wq, ws=ws * case["k"] ** -0.5,
                    bias=normal(case["n"], std=0.1) if case["bias"] else None)
    if kind == "step":
        b, d = case["b"], case["d"]
        parts = 3 if case["z"] else 2
        proj = normal(b, parts * d)
        proj[:, d:2 * d] = proj[:, d:2 * d] * 1.5 + 2  # forget logits: memories of 2 to 200 steps
        proj = proj.to(dt)
        return dict(case=case, h=normal(b, d), v=proj[:, :d], g=proj[:, d:2 * d],
                    z=proj[:, 2 * d:] if case["z"] else None)
    b, l, d = case["b"], case["l"], case["d"]
    parts = 3 if case["z"] else 2
    # values, forget logits and gates are column slices of one projection's output
    proj = torch.empty(b, l, parts * d, dtype=dt, device=dev)
    proj[..., :d] = normal(b, l, d)
    proj[..., d:2 * d] = normal(b, l, d, mean=2.0, std=1.5)
    if case["z"]:
        proj[..., 2 * d:] = normal(b, l, d)
    s = dict(case=case, v=proj[..., :d], g=proj[..., d:2 * d],
             z=proj[..., 2 * d:] if case["z"] else None, h0=normal(b, d), lengths=None)
    if case["lengths"]:
        lengths = torch.randint(0, l + 1, (b,), generator=gen, device=dev, dtype=torch.int32)
        lengths[0] = l
        s["lengths"] = lengths
    if kind == "train":
        s["dy"] = normal(b, l, d).to(dt)
        s["dh"] = normal(b, d)
    return s


# ---- the package's calls ------------------------------------------------------

def _own(s):
    from quantized_state_space_b200 import api
    kind = s["case"]["kind"]
    if kind == "norm":
        out = api.rms_norm_quantize(s["x"], s["w"], residual=s["residual"], eps=EPS)
        q, scale = out[0], out[1]
        return (_values(q, scale, s["x"].dtype), scale) + tuple(out[2:])
    if kind == "linear":
        return api.int8_linear(s["xq"], s["xs"], s["wq"], s["ws"], bias=s["bias"],
                               dtype=DTYPES[s["case"]["dtype"]])
    if kind == "step":
        return api.gated_update(s["h"], s["v"], s["g"], z=s["z"]), s["h"]
    if kind == "scan":
        return api.gated_scan(s["v"], s["g"], z=s["z"], h0=s["h0"], lengths=s["lengths"])
    y, h, saved = api.gated_scan(s["v"], s["g"], z=s["z"], h0=s["h0"], lengths=s["lengths"],
                                 save_states=True)
    return (y, h) + tuple(api.gated_scan_backward(
        s["dy"], s["v"], s["g"], saved, z=s["z"], dh_final=s["dh"], lengths=s["lengths"]))


# ---- plain forms --------------------------------------------------------------

def _values(q, scale, dtype):
    """What the codes stand for, rounded to 16 bits."""
    out = torch.empty(q.shape, dtype=torch.float16 if dtype == torch.float16 else torch.bfloat16,
                      device=q.device)
    return torch.mul(q, scale.unsqueeze(-1), out=out)


def _norm(s):
    x, dtype = s["x"].float(), s["x"].dtype
    more = ()
    if s["residual"] is not None:
        r = (x + s["residual"].float()).to(dtype)
        x, more = r.float(), (r,)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w"]
    scale = y.abs().amax(-1) / 127
    q = torch.clamp(torch.round(y / scale.unsqueeze(-1)), -127, 127)
    q = torch.where(scale.unsqueeze(-1) > 0, q, torch.zeros_like(q))
    return (_values(q, scale, dtype), scale) + more


def _linear(s):
    y = torch.matmul(s["xq"].float(), s["wq"].float().t())
    y = y * (s["xs"].unsqueeze(1) * s["ws"].unsqueeze(0))
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(DTYPES[s["case"]["dtype"]])


def _recur(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1 from a zero state, by doubling the span."""
    span = 1
    while span < u.shape[1]:
        u = torch.cat((u[:, :span], u[:, span:] + a[:, span:] * u[:, :-span]), 1)
        a = torch.cat((a[:, :span], a[:, span:] * a[:, :-span]), 1)
        span *= 2
    return u


def _alive(s):
    """1 where a step is inside its sequence, as (b, l, 1); None without lengths."""
    if s["lengths"] is None:
        return None
    t = torch.arange(s["v"].shape[1], device=s["v"].device)
    return (t < s["lengths"].unsqueeze(1)).unsqueeze(-1)


def _gates(s):
    """(f, 1 - f) in binary32; steps behind the end keep the state."""
    g, alive = s["g"].float(), _alive(s)
    f, n = torch.sigmoid(g), torch.sigmoid(-g)
    if alive is not None:
        f, n = torch.where(alive, f, 1.0), torch.where(alive, n, 0.0)
    return f, n, alive


def _states(s, f, n):
    u = n * s["v"].float()
    u[:, 0] += f[:, 0] * s["h0"]
    return _recur(f, u)


def _scan(s, f, n, alive, h):
    y = h
    if s["z"] is not None:
        z = s["z"].float()
        y = h * (z * torch.sigmoid(z))
    if alive is not None:
        y = torch.where(alive, y, 0.0)
    return y.to(s["v"].dtype), h[:, -1].clone()


def _grad(s, f, n, alive, h):
    dt, dy = s["v"].dtype, s["dy"].float()
    if alive is not None:
        dy = torch.where(alive, dy, 0.0)
    dz = None
    dh = dy
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        dz = (dy * h * (sig * (1 + z * (1 - sig)))).to(dt)
        dh = dy * (z * sig)
    dh = dh.clone()
    dh[:, -1] += s["dh"]
    a = torch.cat((f[:, 1:], torch.zeros_like(f[:, :1])), 1)
    lam = _recur(a.flip(1), dh.flip(1)).flip(1)
    before = torch.cat((s["h0"].unsqueeze(1), h[:, :-1]), 1)
    dv = lam * n
    dg = lam * (before - s["v"].float()) * (f * n)
    return dv.to(dt), dg.to(dt), dz, f[:, 0] * lam[:, 0]


def run(s):
    if own:
        return _own(s)
    kind = s["case"]["kind"]
    if kind == "norm":
        return _norm(s)
    if kind == "linear":
        return _linear(s)
    if kind == "step":
        g = s["g"].float()
        h = torch.sigmoid(g) * s["h"] + torch.sigmoid(-g) * s["v"].float()
        s["h"].copy_(h)
        if s["z"] is not None:
            z = s["z"].float()
            h = h * (z * torch.sigmoid(z))
        return h.to(s["v"].dtype), s["h"]
    f, n, alive = _gates(s)
    h = _states(s, f, n)
    out = _scan(s, f, n, alive, h)
    return out + _grad(s, f, n, alive, h) if kind == "train" else out


# ---- floors and 64-bit values --------------------------------------------------

def work(case):
    kind, e = case["kind"], SIZE[case["dtype"]]
    if kind == "norm":
        n = case["tokens"] * case["d"]
        per = (3 * e if case["residual"] else e) + 1
        return dict(bytes=n * per + 4 * (case["tokens"] + case["d"]), flops=8 * n)
    if kind == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return dict(bytes=m * k + n * k + m * n * e + 4 * (m + n), flops=2 * m * n * k)
    b, d = case["b"], case["d"]
    rows = b * case.get("l", 1)
    z = 1 if case["z"] else 0
    if kind == "train":  # v, g, z and dy in; y, dv, dg and dz out; states in and out
        return dict(bytes=rows * d * e * (6 + 2 * z) + 16 * b * d, flops=rows * d * (20 + 12 * z))
    return dict(bytes=rows * d * e * (3 + z) + 8 * b * d, flops=rows * d * (8 + 5 * z))


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        x = s["x"].double()
        more = ()
        if s["residual"] is not None:
            # the sum is held in the stream's type: rounded from binary32, as the operator defines
            r = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
            x, more = r.double(), (r.double(),)
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["d"] + EPS) * s["w"].double()
        scale = y.abs().max(-1).values / 127
        codes = torch.round(y / scale.unsqueeze(-1)).clamp(-127, 127)
        return (codes * scale.unsqueeze(-1), scale) + more
    if kind == "linear":
        y = torch.einsum("mk,nk->mn", s["xq"].double(), s["wq"].double())
        y = y * s["xs"].double()[:, None] * s["ws"].double()[None, :]
        return y if s["bias"] is None else y + s["bias"].double()
    v, g = s["v"].double(), s["g"].double()
    f = 1 / (1 + torch.exp(-g))
    z = s["z"].double() if s["z"] is not None else None
    silu = z / (1 + torch.exp(-z)) if z is not None else None
    if kind == "step":
        h = f * s["h"].double() + (1 - f) * v
        return (h if z is None else h * silu), h
    b, l, d = case["b"], case["l"], case["d"]
    ends = [l] * b if s["lengths"] is None else s["lengths"].tolist()
    live = torch.zeros(b, l, 1, dtype=torch.float64, device=v.device)
    for i, end in enumerate(ends):
        live[i, :end] = 1
    inside = live.bool()
    hs = torch.empty(b, l + 1, d, dtype=torch.float64, device=v.device)
    hs[:, 0] = s["h0"].double()
    keep, put = torch.where(inside, f, 1.0), torch.where(inside, (1 - f) * v, 0.0)
    for t in range(l):
        torch.addcmul(put[:, t], keep[:, t], hs[:, t], out=hs[:, t + 1])
    y = hs[:, 1:] * live
    if z is not None:
        y = y * silu
    if kind == "scan":
        return y, hs[:, l]
    dy = s["dy"].double() * live
    into = dy if z is None else dy * silu
    lam = torch.empty(b, l, d, dtype=torch.float64, device=v.device)
    carry = s["dh"].double()
    for t in range(l - 1, -1, -1):
        torch.add(into[:, t], carry, out=lam[:, t])
        carry = lam[:, t] * keep[:, t]
    dv = lam * (1 - f) * live
    dg = lam * (hs[:, :l] - v) * f * (1 - f) * live
    dz = None
    if z is not None:
        sig = 1 / (1 + torch.exp(-z))
        dz = dy * hs[:, 1:] * sig * (1 + z * (1 - sig))
    return y, hs[:, l], dv, dg, dz, carry
