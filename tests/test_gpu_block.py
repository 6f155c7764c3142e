"""The recurrences with the norms around them, run as a model's layer runs them: prompts and
single tokens through the output norm and gate to the next layer's input, and the gradients of
both.  Every stage is checked against float64 on the inputs that it was given, so that the bounds
of the single operators apply to the run."""
import pytest
import torch

import linear_ref
import norm_ref
from gpu_util import say
from test_gpu_linear import HALF, check_backward, check_prefill, dev

pytestmark = pytest.mark.gpu


def normal(gen, *shape, dtype=torch.float32, mean=0.0, size=1.0):
    return (mean + size * torch.randn(*shape, generator=gen, dtype=torch.float64)).to(dtype)


def layer(T, H, dv, dtype, seed):
    """Gate, weights and residual stream of a layer whose heads give [T, H, dv]."""
    gen = torch.Generator().manual_seed(seed)
    return dict(gate=normal(gen, T, H, dv, dtype=dtype), w_after=normal(gen, dv, mean=1.0, size=0.2),
                residual=normal(gen, T, H * dv, dtype=dtype, size=2.0),
                w_before=normal(gen, H * dv, mean=1.0, size=0.2))


def norm_case(x, **over):
    """The dict that norm_ref works on, for rows x."""
    d = dict(x=x, w_after=None, gate=None, act="silu", residual=None, scale=1.0, w_before=None,
             eps=1e-6, dh=None, dy=None)
    d.update(over)
    if d["w_before"] is not None:
        d["dy"] = torch.zeros_like(x)
    D = x.shape[-1]
    return {n: t.cpu().reshape(-1, D) if isinstance(t, torch.Tensor) and t.dim() > 1 else
            (t.cpu() if isinstance(t, torch.Tensor) else t) for n, t in d.items()}


def check_norm(d, h=None, y=None):
    want_h, want_y = norm_ref.forward(d)
    b = norm_ref.bounds(d)
    for n, got, want in (("h", h, want_h), ("y", y, want_y)):
        if got is not None:
            norm_ref.check(n, got.reshape(want.shape), want, b[n], norm_ref.FORWARD_EPS,
                           HALF[got.dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens_with_norms(dtype):
    import gated_delta_rule_100_amd as gdr
    H, Hk, dk, dv, lens = 4, 2, 128, 64, [70, 1, 129]
    N, T = len(lens), sum(lens)
    d = linear_ref.make(lens, H, Hk, dk, dv, dtype, "token", "slow", True, seed=61)
    x = dev(d)
    p = dev(layer(T, H, dv, x["q"].dtype, 62))
    o, h = (torch.empty(T, H, dv, device="cuda", dtype=x["q"].dtype) for _ in range(2))
    s = torch.empty_like(x["state_in"])
    say(f"prompt {dtype}")
    gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], s, o,
                           scale=d["scale"], norm=dict(h=h, w_after=p["w_after"], gate=p["gate"]))
    stream, y = torch.empty_like(p["residual"]), torch.empty_like(p["residual"])
    gdr.gdr_block_norm(h.view(T, H * dv), stream, y, residual=p["residual"], scale=0.5,
                       w_before=p["w_before"])
    torch.cuda.synchronize()
    check_prefill(d, o, s)
    check_norm(norm_case(o, w_after=p["w_after"], gate=p["gate"]), h)
    check_norm(norm_case(h.view(T, H * dv), residual=p["residual"], scale=0.5,
                         w_before=p["w_before"]), stream, y)
    for j in range(3):
        say(f"token {j} {dtype}")
        t = linear_ref.make([1] * N, H, Hk, dk, dv, dtype, "token", "slow", False, seed=70 + j)
        t["state_in"] = s.cpu()
        xt, pt = dev(t), dev(layer(N, H, dv, x["q"].dtype, 80 + j))
        o1 = torch.empty(N, H, dv, device="cuda", dtype=x["q"].dtype)
        h1 = torch.empty_like(o1)
        gdr.gdr_linear_decode(xt["q"], xt["k"], xt["v"], xt["g"], s, o1, scale=t["scale"],
                              norm=dict(h=h1, w_after=pt["w_after"], gate=pt["gate"], act="sigmoid"))
        torch.cuda.synchronize()
        want_o, want_s = linear_ref.forward(t)
        b, eps = linear_ref.bounds(t), (dk + 8) * 2.0 ** -24
        linear_ref.check("o", o1, want_o, b["o"], eps, HALF[o1.dtype])
        linear_ref.check("state", s, want_s, b["state_out"], eps)
        check_norm(norm_case(o1, w_after=pt["w_after"], gate=pt["gate"], act="sigmoid"), h1)


@pytest.mark.parametrize("in_graph", [False, True])
def test_gradients_through_the_norm(in_graph):
    """d of the gated output -> d of the heads' outputs -> gradients of the recurrence."""
    import gated_delta_rule_100_amd as gdr
    H, Hk, dk, dv, lens = 4, 2, 64, 128, [100, 0, 65]
    T = sum(lens)
    d = linear_ref.make(lens, H, Hk, dk, dv, "bf16", "token", "slow", True, seed=63)
    x, p = dev(d), dev(layer(T, H, dv, torch.bfloat16, 64))
    dh = normal(torch.Generator().manual_seed(65), T, H, dv, dtype=torch.bfloat16).cuda()
    o, h, d_o, dz = (torch.empty(T, H, dv, device="cuda", dtype=torch.bfloat16) for _ in range(4))
    dw = torch.empty(dv, device="cuda")
    out = {n: torch.empty_like(x[n[1:]]) for n in ("dq", "dk", "dv", "dg", "dstate_in")}
    ws_f = torch.empty(max(1, gdr.gdr_linear_prefill_workspace_bytes(T, 3, H, dk, dv)),
                       dtype=torch.uint8, device="cuda")
    ws_b = torch.empty(gdr.gdr_linear_backward_workspace_bytes(T, 3, H, Hk, dk, dv),
                       dtype=torch.uint8, device="cuda")
    ws_n = torch.empty(gdr.gdr_block_norm_backward_workspace_bytes(T * H, dv), dtype=torch.uint8,
                       device="cuda")

    def step(stream=None):
        gdr.gdr_linear_prefill(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], None, o,
                               scale=d["scale"], workspace=ws_f, stream=stream,
                               norm=dict(h=h, w_after=p["w_after"], gate=p["gate"]))
        gdr.gdr_block_norm_backward(o, dh, None, d_o, w_after=p["w_after"], gate=p["gate"],
                                    dgate=dz, dw_after=dw, workspace=ws_n, stream=stream)
        gdr.gdr_linear_backward(x["q"], x["k"], x["v"], x["g"], x["cu"], x["state_in"], d_o,
                                x["dstate_out"], out["dq"], out["dk"], out["dv"], dg=out["dg"],
                                dstate_in=out["dstate_in"], scale=d["scale"], workspace=ws_b,
                                stream=stream)

    say(f"gradients through the norm, graph {in_graph}")
    step()
    torch.cuda.synchronize()
    results = [o, h, d_o, dz, dw, *out.values()]
    if in_graph:
        want = [t.clone() for t in results]
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            step(stream)
        for r in range(4):
            for t in results:
                t.fill_(float("nan"))
            junk = torch.full((1 << 20,), float(r), device="cuda") * 2.0
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            del junk
            assert all(torch.equal(t, w) for t, w in zip(results, want)), r
        return
    check_prefill(d, o, None)
    n = norm_case(o, w_after=p["w_after"], gate=p["gate"], dh=dh)
    check_norm(n, h)
    want, b = norm_ref.backward(n), norm_ref.bounds(n)
    for name, got in (("dx", d_o), ("dgate", dz), ("dw_after", dw)):
        eps = norm_ref.BACKWARD_EPS + (T * H * 2.0 ** -24 if name == "dw_after" else 0)
        norm_ref.check(name, got.reshape(want[name].shape), want[name], b[name], eps, HALF[got.dtype])
    d["do"] = d_o.cpu()
    check_backward(d, out)


def gated_delta_inputs(shape, H, d, seed):
    """Inputs of the gated delta rule on the GPU: q, k, v bf16 [*shape, H, d], g, beta fp32."""
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (normal(gen, *shape, H, d) for _ in range(3))
    q, k = (torch.nn.functional.normalize(t, dim=-1) for t in (q, k))
    g = -0.1 * torch.rand(*shape, H, generator=gen)
    beta = torch.rand(*shape, H, generator=gen)
    return [t.to(torch.bfloat16).cuda() for t in (q, k, v)] + [g.cuda(), beta.cuda()]


@pytest.mark.parametrize("d", [64, 128])
def test_gated_delta_rule_with_the_norm(d):
    """The norm that a recurrence's call asks for is the norm of its output, bit for bit, and the
    recurrence's own results stay as they are."""
    import gated_delta_rule_100_amd as gdr
    H, N, T = 3, 2, 90
    gen = torch.Generator().manual_seed(d)
    w = normal(gen, d, mean=1.0, size=0.2).cuda()
    cu = torch.tensor([0, 33, T], dtype=torch.int32, device="cuda")
    s0 = normal(gen, N, H, d, d, size=0.1).cuda()

    def check(shape, call, seed):
        args = gated_delta_inputs(shape, H, d, seed)
        z = normal(torch.Generator().manual_seed(seed), *shape, H, d).cuda()
        plain, o, h, want = (torch.full((*shape, H, d), float("nan"), device="cuda") for _ in range(4))
        s_plain, s = s0.clone(), s0.clone()
        call(args, s_plain, plain, None)
        gdr.gdr_block_norm(plain, want, w_after=w, gate=z, act="sigmoid")
        call(args, s, o, dict(h=h, w_after=w, gate=z, act="sigmoid"))
        torch.cuda.synchronize()
        assert torch.equal(o, plain) and torch.equal(s, s_plain) and torch.equal(h, want)
        check_norm(norm_case(o, w_after=w, gate=z, act="sigmoid"), h)
        # in place: o becomes the normed output
        s = s0.clone()
        call(args, s, o, dict(h=o, w_after=w, gate=z, act="sigmoid"))
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(s, s_plain)

    say(f"gated delta rule with the norm d {d}")
    check((N,), lambda a, s, o, n: gdr.gdr_decode_step(*a, s, o, norm=n), 1)
    check((N, 3), lambda a, s, o, n: gdr.gdr_decode_mtp(*a, s, s, o, norm=n), 2)
    check((T,), lambda a, s, o, n: gdr.gdr_chunk_prefill(*a, cu, s, s, o, norm=n), 3)
    check((T,), lambda a, s, o, n: gdr.gdr_chunk_prefill_noalloc(*a, cu, s, s, o, norm=n), 4)


def test_a_refused_norm_leaves_everything_as_it_was():
    import gated_delta_rule_100_amd as gdr
    args = gated_delta_inputs((2,), 3, 64, 5)
    s = torch.zeros(2, 3, 64, 64, device="cuda")
    o = torch.full((2, 3, 64), float("nan"), device="cuda")
    h, w = torch.empty_like(o), torch.ones(64, device="cuda")
    for norm, word in ((dict(), "required"), (dict(h=h, y=o), "exactly"),
                       (dict(h=h, w_before=w), "exactly"), (dict(h=h, w_after=w[:32]), "weights"),
                       (dict(h=h, w_after=w, eps=-1.0), "eps"),
                       (dict(h=h, y=h, w_before=w), "one buffer"),
                       (dict(h=h, w_after=w, gate=h, act="gelu"), "act"),
                       (dict(h=h, residual=h.bfloat16()), "row operands")):
        with pytest.raises(gdr.GdrError, match=word):
            gdr.gdr_decode_step(*args, s, o, norm=norm)
    torch.cuda.synchronize()
    assert torch.isnan(o).all() and not s.any()
