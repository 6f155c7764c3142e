"""Linear attention with a decay for each head in float64, from the definition
written as one quadratic form per sequence (no chunks, no recurrence):

    o_t = scale (sum_{s <= t} e^{G_t - G_s} (q_t . k_s) v_s + e^{G_t} S_0 q_t)

with G the prefix sums of g.  Gradients come from torch's autograd on that
form.  `bounds` evaluates the same forms on absolute values: the sums of the
absolute values of all terms, against which rounding errors are bounded."""
import torch

F64 = torch.float64


def make(lens, H, Hk, dk, dv, dtype="bf16", decay="token", gate="slow", state=True, seed=0,
         pad=0):
    """Seeded inputs (CPU tensors).  gate: slow | std | steep | unit | reset (some g = -inf).
    pad: rows of NaN behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def normal(*s):
        return torch.randn(*s, generator=gen, dtype=F64)

    d = dict(q=normal(T, Hk, dk), k=normal(T, Hk, dk), v=normal(T, H, dv), do=normal(T, H, dv))
    d = {n: x.to(dt) for n, x in d.items()}
    g = -torch.nn.functional.softplus(normal(T, H) if decay == "token" else normal(H))
    g = {"slow": 0.02 * g, "std": g, "steep": 4 * g, "unit": 0 * g, "reset": 0.1 * g}[gate]
    if gate == "reset":
        g = torch.where(torch.rand(g.shape, generator=gen) < 0.05, float("-inf"), g)
    d["g"] = g.float()
    d["state_in"] = normal(N, H, dv, dk).float() if state else None
    d["dstate_out"] = normal(N, H, dv, dk).float() if state else None
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d["cu"] = torch.tensor(cu, dtype=torch.int32)
    if pad:
        for n in ("q", "k", "v", "do"):
            x = d[n]
            d[n] = torch.cat([x, torch.full((pad, *x.shape[1:]), float("nan")).to(dt)])
        if decay == "token":
            d["g"] = torch.cat([d["g"], torch.full((pad, H), float("nan"))])
    d.update(lens=list(lens), H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, scale=dk ** -0.5)
    return d


def _sequence(q, k, v, g, s0, scale):
    """q, k [H, L, dk], v [H, L, dv], g [H, L], s0 [H, dv, dk] -> o, final state."""
    L = q.shape[1]
    G = g.cumsum(-1)
    low = torch.ones(L, L, dtype=torch.bool, device=q.device).tril()
    gam = torch.where(low, (G[:, :, None] - G[:, None, :]).masked_fill(~low, 0).exp(), 0.0)
    o = ((q @ k.transpose(-1, -2)) * gam) @ v + G.exp()[..., None] * (q @ s0.transpose(-1, -2))
    end = (G[:, -1:] - G).exp() if L else G
    s = (v * end[..., None]).transpose(-1, -2) @ k
    s = s + (G[:, -1].exp()[:, None, None] * s0 if L else s0)
    return scale * o, s


def forward(d, absolute=False, leaves=None):
    """o [T, H, dv] (rows of the sequences) and state_out [N, H, dv, dk], float64."""
    H = d["H"]
    x = leaves or inputs64(d, absolute)
    T = int(d["cu"][-1])
    g = x["g"] if x["g"].dim() == 2 else x["g"].expand(d["q"].shape[0], H)
    g = g.clamp(min=-2000.0)  # e^-2000 is 0 in float64 too, and differences stay finite
    rep = lambda t: t.repeat_interleave(H // t.shape[1], 1)  # noqa: E731
    q, k, v = rep(x["q"]), rep(x["k"]), x["v"]
    os, ss = [], []
    for n, L in enumerate(d["lens"]):
        a = int(d["cu"][n])
        s0 = x["state_in"][n] if x["state_in"] is not None else \
            torch.zeros(H, d["dv"], d["dk"], dtype=F64, device=q.device)
        cut = lambda t: t[a:a + L].transpose(0, 1)  # noqa: E731
        o, s = _sequence(cut(q), cut(k), cut(v), cut(g), s0, abs(d["scale"]) if absolute else d["scale"])
        os.append(o.transpose(0, 1))
        ss.append(s)
    o = torch.cat(os)
    assert o.shape[0] == T
    return o, torch.stack(ss)


def inputs64(d, absolute=False):
    out = {}
    for n in ("q", "k", "v", "do", "g", "state_in", "dstate_out"):
        t = d[n]
        out[n] = None if t is None else t.to(F64)
        if absolute and n != "g" and t is not None:
            out[n] = out[n].abs()
    return out


def backward(d, absolute=False):
    """dq, dk, dv, dg, dstate_in, float64, for the rows of the sequences."""
    x = inputs64(d, absolute)
    T = int(d["cu"][-1])
    x["g"] = x["g"].clamp(min=-2000.0)
    names = [n for n in ("q", "k", "v", "g", "state_in") if x[n] is not None]
    for n in names:
        x[n].requires_grad_(True)
    o, s = forward(d, absolute, leaves=x)
    loss = (o * x["do"][:T]).sum()
    if x["dstate_out"] is not None:
        loss = loss + (s * x["dstate_out"]).sum()
    grads = dict(zip(["d" + n for n in names], torch.autograd.grad(loss, [x[n] for n in names])))
    for n in ("dq", "dk", "dv"):
        grads[n] = grads[n][:T]
    if x["g"].dim() == 2:
        grads["dg"] = grads["dg"][:T]
    grads["_end"] = None
    if x["dstate_out"] is not None:
        grads["_end"] = (s.detach() * x["dstate_out"]).sum((-1, -2))  # [N, H]
    return grads


def bounds(d):
    """Sums of absolute values of the terms of every output and gradient."""
    o, s = forward(d, absolute=True)
    b = {"o": o, "state_out": s}
    g = backward(d, absolute=True)
    x = inputs64(d, absolute=True)
    T, H = int(d["cu"][-1]), d["H"]
    # dg_t is formed as a suffix sum of q.dq - k.dk of its sequence: the error of every term of
    # the sum counts.  Per value head: the absolute sums of one head's dq are at most the group's.
    rep = lambda t: t.repeat_interleave(H // t.shape[1], 1)  # noqa: E731
    per = (rep(x["q"][:T]) * rep(g["dq"])).sum(-1) + (x["v"][:T] * g["dv"]).sum(-1)
    rows = []
    for n, L in enumerate(d["lens"]):
        a = int(d["cu"][n])
        r = per[a:a + L].flip(0).cumsum(0).flip(0)
        rows.append(r if g["_end"] is None else r + g["_end"][n])
    dg = torch.cat(rows)
    b.update({n: g[n] for n in ("dq", "dk", "dv")})
    b["dg"] = dg if d["g"].dim() == 2 else dg.sum(0)
    if "dstate_in" in g:
        b["dstate_in"] = g["dstate_in"]
    return b


def slack(d):
    """Relative error, against the sums of absolute values, that the kernels may make before the
    last rounding.  Each term is a product of inputs, a decay and the scale:
      - intermediates of bf16 inputs are held in two bf16 planes, 2^-18 each (two roundings of
        at most 2^-9), three of them along any path from input to output: 3 * 2^-18; fp32 inputs
        are multiplied in fp32;
      - a decay e^x, x a difference of two prefix sums of at most 64 gates in fp32 (log2 units):
        relative error |G| 2^-23 ln 2 + 2^-22 for the exponential; a path crosses at most three
        (own chunk, a chain of chunk decays counted once a chunk below, the last chunk);
      - fp32 accumulation: at most 64 + 2 * 128 roundings of 2^-24 inside a chunk and 2 for each
        chunk of the chain."""
    g = d["g"].clamp(min=-110.0)
    G = 64 * float(g[: int(d["cu"][-1])].abs().max()) if g.numel() else 0.0
    if g.dim() == 2 and g.shape[0]:
        T = int(d["cu"][-1])
        c = g[:T].double().cumsum(0)
        c = torch.cat([torch.zeros_like(c[:1]), c])
        if T > 64:
            G = float((c[64:] - c[:-64]).abs().max()) + 110
        else:
            G = float(c[-1].abs().max())
    chunks = max(d["lens"]) / 64 + 1
    e = 3 * (1.4427 * G * 2.0 ** -23 + 2.0 ** -22) + (64 + 256 + 4 * chunks) * 2.0 ** -24
    return e + (3 * 2.0 ** -18 if d["dtype"] == "bf16" else 0.0)


def check(name, got, ref, bound, eps, half=0.0):
    """|got - ref| <= eps * bound + half step of the output's rounding, elementwise."""
    got = got.detach().to("cpu", F64)
    ref, bound = ref.detach().cpu(), bound.detach().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - (eps * bound + half * (ref.abs() + eps * bound) + 1e-37)
    at = int(over.argmax())
    assert over.max() <= 0, (name, at, float(got.flatten()[at]), float(ref.flatten()[at]),
                             float(eps * bound.flatten()[at]))
