"""A block in 8 bits as a model's layer runs it: norm of the residual stream in 8 bits, projection
to inputs and gates, the recurrence with a decay for each channel, norm and gate in 8 bits and the
projection back; norm= with both on every recurrence; and the gradients through recurrence, norm
and gate.  Every stage is checked against float64 on the inputs that it was given."""
import pytest
import torch

import channel_ref
import linear_ref
import norm_ref
import product_ref
from gpu_util import say
from test_gpu_block import norm_case
from test_gpu_norm8 import check as check_norm8

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16


def normal(gen, *shape, size=1.0):
    return size * torch.randn(*shape, generator=gen)


def weight8(gen, F, K):
    """A weight matrix in 8 bits with a scale for each 128 x 128, on the GPU."""
    w = normal(gen, F, K, size=K ** -0.5)
    kb, fb = -(-K // 128), -(-F // 128)
    p = torch.nn.functional.pad(w, (0, kb * 128 - K, 0, fb * 128 - F)).reshape(fb, 128, kb, 128)
    s = p.abs().amax((1, 3)) / 448
    q = (p / s[:, None, :, None]).clamp(-448, 448).reshape(fb * 128, kb * 128)[:F, :K].to(E4M3)
    return q.contiguous().cuda(), s.cuda()


def empty8(*shape):
    return (torch.full(shape, 1.0, device="cuda").to(E4M3),
            torch.full((*shape[:-1], -(-shape[-1] // 128)), float("nan"), device="cuda"))


def nans(*shape, dtype=BF16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("D, F", [(256, 384), (112, 256)])
def test_recurrent_block_prompt_then_tokens(D, F):
    """D values a token in the residual stream, F channels in the recurrence."""
    import gated_delta_rule_100_amd as gdr
    gen = torch.Generator().manual_seed(D)
    lens = [70, 0, 1, 200]
    T, N = sum(lens), len(lens)
    win, sin = weight8(gen, 3 * F, D)       # inputs, decays and output gates
    wout, sout = weight8(gen, D, F)
    wn, wg = (1 + normal(gen, n, size=0.1) for n in (D, F))
    wn, wg = wn.cuda().to(BF16), wg.cuda().to(BF16)
    cu = torch.tensor([0, 70, 70, 71, 271], dtype=torch.int32, device="cuda")
    state = normal(gen, N, F).cuda()

    def block(x, residual, step):
        """One pass over rows x [tokens, D]; step(x, z, h, norm) runs the recurrence."""
        rows = x.shape[0]
        h = nans(rows, D)
        y8, ys = empty8(rows, D)
        gdr.gdr_block_norm8(x, y8, ys, h, residual=residual, scale=0.5, w_before=wn)
        torch.cuda.synchronize()
        check_norm8(norm_case(x, residual=residual, scale=0.5, w_before=wn), y8, ys, h)
        proj = nans(rows, 3 * F)
        gdr.gdr_product8(y8, ys, win, sin, proj)
        torch.cuda.synchronize()
        product_ref.check("in", proj, dict(a=y8, sa=ys, w=win, sw=sin))
        u, z, gate = proj[:, :F], proj[:, F:2 * F], proj[:, 2 * F:].contiguous()
        o, (o8, os), out = nans(rows, F), empty8(rows, F), nans(rows, D)
        step(u, z, o, dict(y8=o8, y_scale=os, w_after=wg, gate=gate,
                           project=dict(w=wout, w_scale=sout, out=out)))
        torch.cuda.synchronize()
        check_norm8(norm_case(o, w_after=wg, gate=gate), o8, os)
        product_ref.check("out", out, dict(a=o8, sa=os, w=wout, sw=sout))
        return u, z, o, out

    def reference(u, z, s0, seqs):
        return dict(x=u.cpu(), g=z.cpu(), state_in=s0.cpu(), lens=seqs, D=F, gate="logit",
                    complement=True)

    say(f"block prompt D {D} F {F}")
    x, r = (normal(gen, T, D).cuda().to(BF16) for _ in range(2))
    end = torch.full_like(state, float("nan"))
    u, z, o, out = block(x, r, lambda u, z, o, norm: gdr.gdr_channel_prefill(
        u, z, cu, state, end, o, gate="logit", complement=True, norm=norm))
    d = reference(u, z, state, lens)
    (want_h, want_s), (eh, es) = channel_ref.forward(d), channel_ref.forward_bounds(d)
    channel_ref.check("h", o, want_h, eh)
    channel_ref.check("state", end, want_s, es)
    for t in range(3):
        say(f"block token {t}")
        x, r, before = out[:N], normal(gen, N, D).cuda().to(BF16), end.clone()
        u, z, o, out = block(x, r, lambda u, z, o, norm: gdr.gdr_channel_decode(
            u, z, end, o, gate="logit", complement=True, norm=norm))
        d = reference(u, z, before, [1] * N)
        (want_h, want_s), (eh, es) = channel_ref.forward(d), channel_ref.forward_bounds(d)
        channel_ref.check("h", o, want_h, eh)
        channel_ref.check("state", end, want_s, es)


@pytest.mark.parametrize("heads", [True, False])
def test_norm8_and_product_behind_every_recurrence(heads):
    """The same bits as the calls one after the other; rows of w over all heads, or over one."""
    import gated_delta_rule_100_amd as gdr
    H, d, lens = 3, 128, [40, 0, 30]
    T, N = sum(lens), len(lens)
    x = linear_ref.make(lens, H, H, d, d, "bf16", "token", "std", True, seed=5)
    x = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in x.items()}
    q, k, v, g = x["q"], torch.nn.functional.normalize(x["k"].float(), dim=-1).to(BF16), x["v"], x["g"]
    beta = torch.sigmoid(g)
    gen = torch.Generator().manual_seed(6)
    w, sw = weight8(gen, 96, H * d if heads else d)
    wa = (1 + normal(gen, d, size=0.1)).cuda()
    gates = normal(gen, T, H, d).cuda().to(BF16)
    states = normal(gen, T, H, d, d, size=0.1).cuda()
    s1, cu = torch.empty_like(x["state_in"]), x["cu"]
    four = lambda t: t[:, None].contiguous()  # noqa: E731
    calls = {
        "gdr_decode_step": lambda o, n: gdr.gdr_decode_step(q, k, v, g, beta, states.clone(), o, norm=n),
        "gdr_decode_mtp": lambda o, n: gdr.gdr_decode_mtp(four(q), four(k), four(v), four(g), four(beta),
                                                          states, None, o, norm=n),
        "gdr_chunk_prefill": lambda o, n: gdr.gdr_chunk_prefill(q, k, v, g, beta, cu, x["state_in"], s1,
                                                                o, norm=n),
        "gdr_chunk_prefill_noalloc": lambda o, n: gdr.gdr_chunk_prefill_noalloc(
            q, k, v, g, beta, cu, x["state_in"], s1, o, norm=n),
        "gdr_linear_decode": lambda o, n: gdr.gdr_linear_decode(q, k, v, g, states.clone(), o, norm=n),
        "gdr_linear_prefill": lambda o, n: gdr.gdr_linear_prefill(q, k, v, g, cu, x["state_in"], s1, o,
                                                                  norm=n),
    }
    for name, call in calls.items():
        say(f"norm8 and product behind {name}")
        shape = (T, 1, H, d) if name == "gdr_decode_mtp" else (T, H, d)
        o, (o8, os) = nans(*shape), empty8(*shape)
        out = nans(*(shape[:-2] if heads else shape[:-1]), 96)
        gate = gates.view(shape)
        call(o, dict(y8=o8, y_scale=os, w_after=wa, gate=gate, project=dict(w=w, w_scale=sw, out=out)))
        alone, (a8, as_) = nans(*shape), empty8(*shape)
        call(alone, None)
        gdr.gdr_block_norm8(alone, a8, as_, w_after=wa, gate=gate)
        want = nans(out.numel() // 96, 96)
        gdr.gdr_product8(a8.view(want.shape[0], -1), as_.view(want.shape[0], -1), w, sw, want)
        torch.cuda.synchronize()
        assert torch.equal(o, alone) and torch.equal(os, as_), name
        assert torch.equal(o8.float(), a8.float()) and torch.equal(out.view(-1, 96), want), name
        assert torch.isfinite(out).all()
    # without the product
    o, (o8, os) = nans(T, H, d), empty8(T, H, d)
    calls["gdr_linear_prefill"](o, dict(y8=o8, y_scale=os, w_after=wa, gate=gates))
    torch.cuda.synchronize()
    assert torch.equal(o8.float(), a8.float()) and torch.equal(os, as_)


def test_heads_of_half_a_block_are_refused():
    """Heads of 64 values have scales of their own, which no block of 128 of a product has."""
    import gated_delta_rule_100_amd as gdr
    d, H, T = 64, 4, 10
    q = torch.randn(T, H, d, device="cuda").to(BF16)
    o, (o8, os) = nans(T, H, d), empty8(T, H, d)
    w, sw = weight8(torch.Generator().manual_seed(7), 96, H * d)
    before = o.clone()
    with pytest.raises(gdr.GdrError, match="whole blocks of 128"):
        gdr.gdr_linear_decode(q, q, q, torch.zeros(T, H, device="cuda"),
                              torch.zeros(T, H, d, d, device="cuda"), o,
                              norm=dict(y8=o8, y_scale=os, project=dict(w=w, w_scale=sw,
                                                                        out=nans(T, 96))))
    torch.cuda.synchronize()
    assert torch.isnan(o).all() and torch.isnan(before).all()


def test_gradients_through_recurrence_norm_and_gate():
    """fp32, end to end against float64 autograd: roundings of 2^-24 along sums of at most 2^8
    terms, in two operators, are below 1e-5 of a result's size."""
    import gated_delta_rule_100_amd as gdr
    lens, D = [150, 3, 64], 136
    d = channel_ref.make(lens, D, "logit", True, "f32", "f32", seed=8)
    gen = torch.Generator().manual_seed(9)
    T = sum(lens)
    w, gate, dy = 1 + normal(gen, D, size=0.1), normal(gen, T, D), normal(gen, T, D)
    x = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in d.items()}
    form = dict(gate="logit", complement=True)
    h, y, s = (nans(*n, dtype=torch.float32) for n in ((T, D), (T, D), (len(lens), D)))
    gdr.gdr_channel_prefill(x["x"], x["g"], x["cu"], x["state_in"], s, h, **form,
                            norm=dict(h=y, w_after=w.cuda(), gate=gate.cuda()))
    dh, dgate, dw = torch.empty_like(h), torch.empty_like(h), torch.empty(D, device="cuda")
    gdr.gdr_block_norm_backward(h, dy.cuda(), None, dh, w_after=w.cuda(), gate=gate.cuda(),
                                dgate=dgate, dw_after=dw)
    got = dict(dx=torch.empty_like(h), dg=torch.empty_like(h), dstate_in=torch.empty_like(s))
    gdr.gdr_channel_backward(x["x"], x["g"], h, x["cu"], x["state_in"], dh, x["dstate_out"],
                             got["dx"], got["dg"], dstate_in=got["dstate_in"], **form)
    torch.cuda.synchronize()

    F64 = torch.float64
    leaves = {n: d[n].to(F64).requires_grad_(True) for n in ("x", "g", "state_in")}
    wl, gl = w.to(F64).requires_grad_(True), gate.to(F64).requires_grad_(True)
    rh, rs = channel_ref.forward(d, leaves)
    ry, _ = norm_ref.forward(dict(act="silu", scale=1.0, eps=1e-6), dict(x=rh, w_after=wl, gate=gl))
    loss = (ry * dy.to(F64)).sum() + (rs * d["dstate_out"].to(F64)).sum()
    want = torch.autograd.grad(loss, [*leaves.values(), wl, gl])
    got = [got["dx"], got["dg"], got["dstate_in"], dw, dgate]
    for n, a, b in zip(("x", "g", "state_in", "w", "gate"), got, want):
        err = float((a.cpu().to(F64) - b).norm() / b.norm())
        assert err < 1e-5, (n, err)
    assert float((y.cpu().to(F64) - ry.detach()).norm() / ry.detach().norm()) < 1e-5
