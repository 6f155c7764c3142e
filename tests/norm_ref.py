"""The norms around a block (gdr_block_norm) in float64 from the definition, gradients by torch's
autograd, and sums of absolute values of the terms, against which rounding errors are bounded."""
import torch

F64 = torch.float64


def make(rows, D, dtype="bf16", after=True, gate="silu", residual=True, before=True, scale=0.7,
         eps=1e-6, seed=0, w_dtype=None):
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wd = dt if w_dtype is None else w_dtype

    def normal(*s):
        return torch.randn(*s, generator=gen, dtype=F64)

    d = dict(x=normal(rows, D).to(dt),
             w_after=(1 + 0.2 * normal(D)).to(wd) if after else None,
             gate=normal(rows, D).to(dt) if gate != "none" else None,
             residual=(2 * normal(rows, D)).to(dt) if residual else None,
             w_before=(1 + 0.2 * normal(D)).to(wd) if before else None,
             dh=normal(rows, D).to(dt), dy=normal(rows, D).to(dt) if before else None)
    d.update(act=gate, scale=scale, eps=eps)
    return d


def forward(d, x=None):
    x = x or {n: d[n].to(F64) for n in ("x", "w_after", "gate", "residual", "w_before")
              if d[n] is not None}
    u = x["x"]
    if "w_after" in x:
        u = u / torch.sqrt(u.pow(2).mean(-1, keepdim=True) + d["eps"]) * x["w_after"]
    if "gate" in x:
        z = x["gate"]
        u = u * torch.sigmoid(z) * (z if d["act"] == "silu" else 1)
    h = d["scale"] * u + (x["residual"] if "residual" in x else 0)
    y = h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + d["eps"]) * x["w_before"] \
        if "w_before" in x else None
    return h, y


def backward(d):
    x = {n: d[n].to(F64).requires_grad_(True)
         for n in ("x", "w_after", "gate", "residual", "w_before") if d[n] is not None}
    h, y = forward(d, x)
    loss = 0
    if d["dh"] is not None:
        loss = loss + (h * d["dh"].to(F64)).sum()
    if y is not None:
        loss = loss + (y * d["dy"].to(F64)).sum()
    return {"d" + n: g for n, g in zip(x, torch.autograd.grad(loss, list(x.values())))}


def bounds(d):
    """Sums of absolute values behind h, y and every gradient."""
    a = {n: None if d[n] is None else d[n].to(F64)
         for n in ("x", "w_after", "gate", "residual", "w_before", "dh", "dy")}
    one = torch.ones((), dtype=F64)
    ix = 1 / torch.sqrt(a["x"].pow(2).mean(-1, keepdim=True) + d["eps"]) \
        if a["w_after"] is not None else one
    n = a["x"].abs() * ix * (a["w_after"].abs() if a["w_after"] is not None else 1)
    act = slope = one
    if a["gate"] is not None:
        z, s = a["gate"], torch.sigmoid(a["gate"])
        act = s * (z.abs() if d["act"] == "silu" else 1)
        slope = s * (1 + z.abs() * (1 - s)) if d["act"] == "silu" else s * (1 - s) + s * s
    sc = abs(d["scale"])
    h = sc * n * act + (a["residual"].abs() if a["residual"] is not None else 0)
    b = {"h": h}
    dh = a["dh"].abs() if a["dh"] is not None else torch.zeros_like(h)
    if a["w_before"] is not None:
        true_h, _ = forward(d)
        ih = 1 / torch.sqrt(true_h.pow(2).mean(-1, keepdim=True) + d["eps"])
        hh = h * ih
        # y = h ih w: the error of h moves ih by at most mean(hh^2) of its own size
        b["y"] = hh * (1 + hh.pow(2).mean(-1, keepdim=True)) * a["w_before"].abs()
        t = a["dy"].abs() * a["w_before"].abs()
        b["dw_before"] = (a["dy"].abs() * hh * (1 + hh.pow(2).mean(-1, keepdim=True))).sum(0)
        dh = dh + ih * (t + hh * (t * hh).mean(-1, keepdim=True)) * \
            (1 + 3 * hh.pow(2).mean(-1, keepdim=True))
    b["dresidual"] = dh
    dn = sc * dh
    b["dgate"] = dn * n * slope
    dn = dn * act
    xh = a["x"].abs() * ix
    b["dw_after"] = (dn * xh).sum(0)
    if a["w_after"] is not None:
        t = dn * a["w_after"].abs()
        dn = ix * (t + xh * (t * xh).mean(-1, keepdim=True))
    b["dx"] = dn
    return b


# Roundings of 2^-24 along one path: sums of squares of at most 16 terms a thread and 10 steps
# across threads, halved by the square root; exp, reciprocals and products with at most 2 steps
# each, four norms and gates deep in the gradient.
FORWARD_EPS = 64 * 2.0 ** -24
BACKWARD_EPS = 256 * 2.0 ** -24


def check(name, got, want, bound, eps, half):
    got = got.detach().to("cpu", F64)
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - want).abs() - (eps * bound + half * (want.abs() + eps * bound) + 1e-37)
    at = int(over.argmax())
    assert over.max() <= 0, (name, at, float(got.flatten()[at]), float(want.flatten()[at]))
