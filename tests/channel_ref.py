"""The recurrence with a decay for each channel (gdr_channel_*) in float64, token by token, its
gradients by torch's autograd, and bounds of the rounding errors of fp32 sums and products.

A term of h_t that entered at s <= t has passed one decay and at most three roundings a token
(the product of decays, the sum, and one more where groups, tiles and blocks of tokens are
joined, fewer than one a token), whatever the grouping.  With e_t the relative error that a token
adds, the error of h is below E_t = a_t E_{t-1} + e_t H_t, H the same recurrence on absolute
values.  e_t = (16 + 12 |g_t|) 2^-24: a decay is off by two units in its last place and by the
rounding of its exponent, |g| 2^-24 of it, or, of a product formed as the exponential of a sum of
up to eight of them, by eight times that."""
import torch

F64 = torch.float64
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(lens, D, gate="log", complement=False, dtype="bf16", gdtype="f32", kind="std", state=True,
         seed=0, pad=0):
    """Seeded inputs (CPU tensors).  kind: std | slow | steep | unit | reset (some decays of 0).
    pad: rows of NaN behind the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def normal(*s):
        return torch.randn(*s, generator=gen, dtype=F64)

    z = normal(T, D) + {"std": 2, "slow": 8, "steep": -3, "unit": 200, "reset": 3}[kind]
    if kind == "reset":
        z = torch.where(torch.rand(z.shape, generator=gen) < 0.05, float("-inf"), z)
    g = z if gate == "logit" else -torch.nn.functional.softplus(-z)
    d = dict(x=normal(T, D).to(DT[dtype]), g=g.to(DT[gdtype]), dh=normal(T, D).to(DT[dtype]),
             state_in=normal(N, D).float() if state else None,
             dstate_out=normal(N, D).float() if state else None)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    d["cu"] = torch.tensor(cu, dtype=torch.int32)
    if pad:
        for n in ("x", "g", "dh"):
            d[n] = torch.cat([d[n], torch.full((pad, D), float("nan")).to(d[n].dtype)])
    d.update(lens=list(lens), D=D, gate=gate, complement=complement)
    return d


def terms(d, leaves=None):
    """a, 1 - a and b of the sequences' rows."""
    T = sum(d["lens"])
    x, g = ((d if leaves is None else leaves)[n][:T].to(F64) for n in ("x", "g"))
    if d["gate"] == "log":
        a, rest = torch.exp(g), -torch.expm1(g)
    else:
        a, rest = torch.sigmoid(g), torch.sigmoid(-g)
    return a, rest, (rest * x if d["complement"] else x)


def scan(d, a, b, s0):
    """h and final states of h_t = a_t h_{t-1} + b_t over the sequences."""
    hs, ends, at = [], [], 0
    for n, L in enumerate(d["lens"]):
        s = s0[n]
        for t in range(at, at + L):
            s = a[t] * s + b[t]
            hs.append(s)
        ends.append(s)
        at += L
    h = torch.stack(hs) if hs else torch.zeros(0, d["D"], dtype=F64)
    return h, torch.stack(ends)


def zero_or(x, d):
    return torch.zeros(len(d["lens"]), d["D"], dtype=F64) if x is None else x.to(F64)


def forward(d, leaves=None):
    a, _, b = terms(d, leaves)
    s0 = zero_or(d["state_in"], d) if leaves is None else leaves["state_in"]
    return scan(d, a, b, s0)


def step_error(d):
    g = d["g"][:sum(d["lens"])].to(F64).abs().clamp(max=110)
    return (16 + 12 * g) * 2.0 ** -24


def forward_bounds(d):
    a, _, b = terms(d)
    H, end = scan(d, a, b.abs(), zero_or(d["state_in"], d).abs())
    E, Eend = scan(d, a, step_error(d) * H, 0 * zero_or(None, d))
    return E, Eend


def flipped(d):
    """The batch with time running backwards (sequences in reverse order too)."""
    return dict(d, lens=d["lens"][::-1])


def adjoint(d, a, u, c0):
    """r_t = u_t + a_{t+1} r_{t+1} within each sequence, c0 for the last token's; r and the
    a_1 r_1 (c0 of an empty one) of every sequence."""
    rs, cs, at = [], [], 0
    for n, L in enumerate(d["lens"]):
        c, out = c0[n], []
        for t in range(at + L - 1, at - 1, -1):
            r = u[t] + c
            out.append(r)
            c = a[t] * r
        rs += out[::-1]
        cs.append(c)
        at += L
    return (torch.stack(rs) if rs else torch.zeros(0, d["D"], dtype=F64)), torch.stack(cs)


def previous(d, h, s0):
    """h_{t-1} of every token."""
    out, at = [], 0
    for n, L in enumerate(d["lens"]):
        if L:
            out += [s0[n:n + 1], h[at:at + L - 1]]
        at += L
    return torch.cat(out) if out else torch.zeros(0, d["D"], dtype=F64)


def backward(d, h):
    """The documented gradient formulas, with h as the forward pass stored it; and bounds."""
    T = sum(d["lens"])
    a, rest, _ = terms(d)
    x, dh = d["x"][:T].to(F64), d["dh"][:T].to(F64)
    ds, s0 = zero_or(d["dstate_out"], d), zero_or(d["state_in"], d)
    r, c = adjoint(d, a, dh, ds)
    R, C = adjoint(d, a, dh.abs(), ds.abs())
    e = step_error(d)
    E, Ec = adjoint(d, a, e * R, 0 * ds)
    Ec = Ec + e.max() * C if T else Ec
    prev = previous(d, h[:T].to(F64), s0)
    if d["complement"]:
        prev = prev - x
    slope = a * rest if d["gate"] == "logit" else a
    gain = rest if d["complement"] else torch.ones_like(rest)
    want = dict(dx=gain * r, dg=slope * r * prev, dstate_in=c)
    bounds = dict(dx=gain * (E + e * R), dg=slope * prev.abs() * (E + 2 * e * R), dstate_in=Ec)
    return want, bounds


def autograd(d):
    """dx, dg and dstate_in by torch's autograd on the forward recurrence."""
    T = sum(d["lens"])
    leaves = {n: d[n].to(F64).requires_grad_(True) for n in ("x", "g")}
    leaves["state_in"] = zero_or(d["state_in"], d).requires_grad_(True)
    h, end = forward(d, leaves)
    loss = (h * d["dh"][:T].to(F64)).sum() + (end * zero_or(d["dstate_out"], d)).sum()
    return dict(zip(("dx", "dg", "dstate_in"), torch.autograd.grad(loss, list(leaves.values()))))


def check(name, got, want, bound):
    got = got.detach().to("cpu")
    half, got = HALF[got.dtype], got.to(F64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    if not got.numel():
        return
    over = (got - want).abs() - (bound + half * (want.abs() + bound) + 1e-36)
    at = int(over.argmax())
    assert over.max() <= 0, (name, at, float(got.flatten()[at]), float(want.flatten()[at]),
                             float(bound.flatten()[at]))
