"""Norms around a block on the GPU against float64, elementwise within norm_ref's bounds."""
import pytest
import torch

import norm_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
PARTS = [dict(), dict(after=False, gate="none"), dict(gate="sigmoid", residual=False),
         dict(residual=False, before=False), dict(after=False, gate="none", residual=False),
         dict(gate="none", before=False), dict(after=False, before=False, gate="sigmoid")]


def dev(d):
    return {n: (x.cuda() if isinstance(x, torch.Tensor) else x) for n, x in d.items()}


OPERANDS = ("w_after", "gate", "act", "residual", "scale", "w_before", "eps")


def forward(d, out_dtype=None, x=None, want_h=True):
    import gated_delta_rule_100_amd as gdr
    x = x or dev(d)
    like = lambda: torch.full(x["x"].shape, float("nan"), device="cuda",  # noqa: E731
                              dtype=out_dtype or x["x"].dtype)
    h = like() if want_h or x["w_before"] is None else None
    y = like() if x["w_before"] is not None else None
    gdr.gdr_block_norm(x["x"], h, y, **{n: x[n] for n in OPERANDS})
    torch.cuda.synchronize()
    return h, y


def check_forward(d, h, y):
    want_h, want_y = ref.forward(d)
    b = ref.bounds(d)
    if h is not None:
        ref.check("h", h, want_h, b["h"], ref.FORWARD_EPS, HALF[h.dtype])
    if y is not None:
        ref.check("y", y, want_y, b["y"], ref.FORWARD_EPS, HALF[y.dtype])


def backward(d, out_dtype=None, x=None, workspace=None):
    import gated_delta_rule_100_amd as gdr
    x = x or dev(d)
    out = {}
    for n in ("x", "gate", "residual"):
        if x[n] is not None:
            out["d" + n] = torch.full(x["x"].shape, float("nan"), device="cuda",
                                      dtype=out_dtype or x["x"].dtype)
    for n in ("w_after", "w_before"):
        if x[n] is not None:
            out["d" + n] = torch.full(x[n].shape, float("nan"), device="cuda")
    kw = {n: out.get(n) for n in ("dgate", "dresidual", "dw_after", "dw_before")}
    gdr.gdr_block_norm_backward(x["x"], x["dh"], x["dy"], out["dx"], workspace=workspace,
                                **{n: x[n] for n in OPERANDS}, **kw)
    torch.cuda.synchronize()
    return out


def check_backward(d, out):
    want, b = ref.backward(d), ref.bounds(d)
    for n, got in out.items():
        # weight gradients: fp32 sums over the rows
        eps = ref.BACKWARD_EPS + (d["x"].shape[0] * 2.0 ** -24 if n.startswith("dw") else 0)
        ref.check(n, got, want[n], b[n], eps, HALF[got.dtype])


# widths of every kernel shape, their edges, odd ones and the largest
WIDTHS = [1, 7, 8, 63, 64, 65, 128, 200, 256, 300, 512, 777, 1024, 1100, 2048, 2056, 4096, 5000,
          8192, 16383, 16384]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widths(D, dtype):
    for rows in (1, 5, 67):
        say(f"norm rows {rows} D {D} {dtype}")
        d = ref.make(rows, D, dtype, seed=D + rows)
        check_forward(d, *forward(d))
        check_backward(d, backward(d))


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("dtype, D, rows", [("bf16", 128, 1000), ("f32", 64, 333),
                                            ("bf16", 2048, 40), ("f32", 1001, 9)])
def test_parts(parts, dtype, D, rows):
    say(f"norm {parts} {dtype} rows {rows} D {D}")
    d = ref.make(rows, D, dtype, seed=7, **parts)
    check_forward(d, *forward(d))
    check_backward(d, backward(d))
    check_forward(d, *forward(d, torch.float32, want_h=False))
    check_backward(d, backward(d, torch.float32))


def test_fp32_weights_with_bf16_rows():
    d = ref.make(50, 256, "bf16", seed=8, w_dtype=torch.float32)
    check_forward(d, *forward(d))
    check_backward(d, backward(d))


def test_gradient_of_y_alone():
    d = ref.make(50, 128, "bf16", seed=9)
    d["dh"] = None
    check_backward(d, backward(d))


def test_rows_of_zeros():
    d = ref.make(20, 128, "f32", residual=False, seed=10)
    d["x"][3] = 0
    d["gate"][5] = 0
    h, y = forward(d)
    assert not h[3].any() and not y[3].any() and not y[5].any()
    check_forward(d, h, y)
    check_backward(d, backward(d))


def test_large_gates():
    # sigmoid saturates at both ends without overflow
    d = ref.make(4, 64, "f32", residual=False, before=False, seed=11)
    d["gate"][0], d["gate"][1], d["gate"][2] = 200.0, -200.0, 80.0
    check_forward(d, *forward(d))
    check_backward(d, backward(d))


def test_no_rows():
    import gated_delta_rule_100_amd as gdr
    x = torch.empty(0, 64, device="cuda")
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), float("nan"), device="cuda")
    gdr.gdr_block_norm(x, x.clone(), w_after=w)
    gdr.gdr_block_norm_backward(x, x.clone(), None, x.clone(), w_after=w, dw_after=dw)
    torch.cuda.synchronize()
    assert not dw.any()


@pytest.mark.parametrize("into", ["x", "gate", "residual"])
@pytest.mark.parametrize("D", [128, 999, 3000])
def test_in_place(into, D):
    d = ref.make(70, D, "bf16", seed=12)
    want_h, want_y = forward(d)
    import gated_delta_rule_100_amd as gdr
    for which in ("h", "y"):
        x = dev(d)
        other = torch.empty_like(x["x"])
        h, y = (x[into], other) if which == "h" else (other, x[into])
        gdr.gdr_block_norm(x["x"], h, y, **{n: x[n] for n in OPERANDS})
        torch.cuda.synchronize()
        assert torch.equal(h, want_h) and torch.equal(y, want_y), which


def test_many_rows_and_more_than_2_31_elements():
    import gated_delta_rule_100_amd as gdr
    rows, D = (1 << 31) // 4096 + 3, 4096
    say(f"norm rows {rows} D {D}")
    d = ref.make(3, D, "bf16", residual=False, before=False, seed=13)
    x, z = (torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    for at, i in ((0, 0), (rows // 2, 1), (rows - 1, 2)):
        x[at].copy_(d["x"][i])
        z[at].copy_(d["gate"][i])
    h = torch.empty_like(x)
    w = d["w_after"].cuda()
    gdr.gdr_block_norm(x, h, w_after=w, gate=z, scale=d["scale"], eps=d["eps"])
    torch.cuda.synchronize()
    at = [0, rows // 2, rows - 1]
    check_forward(d, h[at], None)
    dh = torch.zeros_like(x)
    for a, i in zip(at, range(3)):
        dh[a].copy_(d["dh"][i])
    dz, dw = torch.empty_like(x), torch.empty(D, device="cuda")
    gdr.gdr_block_norm_backward(x, dh, None, h, w_after=w, gate=z, scale=d["scale"], eps=d["eps"],
                                dgate=dz, dw_after=dw)
    torch.cuda.synchronize()
    check_backward(d, dict(dx=h[at], dgate=dz[at], dw_after=dw))


def test_repeated_streams_and_graph():
    import gated_delta_rule_100_amd as gdr
    d = ref.make(3000, 128, "bf16", seed=14)
    x = dev(d)
    h, y = forward(d, x=x)
    b = backward(d, x=x)
    ws = torch.empty(gdr.gdr_block_norm_backward_workspace_bytes(3000, 128), dtype=torch.uint8,
                     device="cuda")
    h2, y2 = torch.empty_like(h), torch.empty_like(y)
    b2 = {n: torch.empty_like(t) for n, t in b.items()}

    def step(s1=None, s2=None):
        gdr.gdr_block_norm(x["x"], h2, y2, stream=s1, **{n: x[n] for n in OPERANDS})
        gdr.gdr_block_norm_backward(x["x"], x["dh"], x["dy"], b2["dx"], workspace=ws, stream=s2,
                                    **{n: x[n] for n in OPERANDS},
                                    **{n: b2[n] for n in b2 if n != "dx"})

    def same():
        torch.cuda.synchronize()
        return torch.equal(h, h2) and torch.equal(y, y2) and all(torch.equal(b[n], b2[n]) for n in b)

    torch.cuda.synchronize()
    step(torch.cuda.Stream(), torch.cuda.Stream())
    assert same()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(stream, stream)
    for r in range(4):
        for t in (h2, y2, *b2.values()):
            t.fill_(float(r))
        torch.cuda.synchronize()
        graph.replay()
        assert same(), r
