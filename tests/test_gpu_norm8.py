"""The norms around a block with an output in 8 bits on the GPU against float64."""
import pytest
import torch

import norm_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
PARTS = [dict(), dict(after=False, gate="none"), dict(gate="sigmoid", residual=False),
         dict(residual=False, before=False), dict(after=False, gate="none", residual=False),
         dict(gate="none", before=False), dict(after=False, before=False, gate="sigmoid")]
OPERANDS = ("w_after", "gate", "act", "residual", "scale", "w_before", "eps")


def dev(d):
    return {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in d.items()}


def run(d, x=None, h=None, want_h=False, **kw):
    import gated_delta_rule_100_amd as gdr
    x = x or dev(d)
    shape = x["x"].shape
    y8 = torch.full(shape, 1.0, device="cuda").to(E4M3)
    s = torch.full((*shape[:-1], -(-shape[-1] // 128)), float("nan"), device="cuda")
    if want_h and h is None:
        h = torch.full(shape, float("nan"), device="cuda", dtype=x["x"].dtype)
    gdr.gdr_block_norm8(x["x"], y8, s, h, **{n: x[n] for n in OPERANDS}, **kw)
    torch.cuda.synchronize()
    return y8, s, h


def blocks_of(t):
    """[..., D] -> [..., ceil(D / 128), 128], filled up with zeros."""
    D = t.shape[-1]
    kb = -(-D // 128)
    return torch.nn.functional.pad(t, (0, kb * 128 - D)).reshape(*t.shape[:-1], kb, 128)


def check(d, y8, s, h=None):
    want_h, want_y = ref.forward(d)
    b = ref.bounds(d)
    if h is not None:
        ref.check("h", h, want_h, b["h"], ref.FORWARD_EPS,
                  2.0 ** -8 if h.dtype == torch.bfloat16 else 2.0 ** -24)
    want, err = (want_y, b["y"]) if want_y is not None else (want_h, b["h"])
    err = blocks_of(ref.FORWARD_EPS * err)
    y, got, s = blocks_of(want), blocks_of(y8.cpu().double()), s.cpu().double()
    # the scale: the error of the largest value and a division
    top = y.abs().amax(-1)
    assert ((s * 448 - top).abs() <= err.amax(-1) + 2.0 ** -23 * top).all()
    # a value: its own error, three roundings of the quotient, and half a step of e4m3, 2^-4 of
    # it and 2^-10 (of the scale) at least
    off = (got * s[..., None] - y).abs()
    most = err + 2.0 ** -22 * y.abs()
    half = torch.maximum(2.0 ** -4 * (y.abs() + most), 2.0 ** -10 * s[..., None])
    assert (off <= most + half).all(), float((off - most - half).max())
    # the largest of a block uses the whole range
    assert (got.abs().amax(-1)[s > 0] == 448).all()


@pytest.mark.parametrize("D", [16, 48, 64, 80, 112, 128, 144, 256, 304, 512, 528, 1024, 1040, 2048,
                               2064, 4096, 5008, 8192, 8208, 16384])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widths(D, dtype):
    for rows in (1, 5, 67):
        say(f"norm8 rows {rows} D {D} {dtype}")
        d = ref.make(rows, D, dtype, seed=D + rows)
        y8, s, h = run(d, want_h=True)
        check(d, y8, s, h)


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("dtype, D, rows", [("bf16", 128, 1000), ("f32", 64, 333),
                                            ("bf16", 2048, 40), ("f32", 1008, 9)])
def test_parts(parts, dtype, D, rows):
    say(f"norm8 {parts} {dtype} rows {rows} D {D}")
    d = ref.make(rows, D, dtype, seed=7, **parts)
    for want_h in (False, True):
        check(d, *run(d, want_h=want_h))


def test_the_same_values_as_the_norm():
    """8 bits of the fp32 result that gdr_block_norm writes, and the same h."""
    import gated_delta_rule_100_amd as gdr
    d = ref.make(300, 384, "bf16", seed=8, w_dtype=torch.float32)
    x = dev(d)
    y8, s, h = run(d, want_h=True)
    h32, y32 = (torch.empty(300, 384, device="cuda") for _ in range(2))
    gdr.gdr_block_norm(x["x"], h32, y32, **{n: x[n] for n in OPERANDS})
    torch.cuda.synchronize()
    assert torch.equal(h, h32.bfloat16())
    # on the host, by tensors: torch divides by a number as a product with its reciprocal
    y = blocks_of(y32.cpu())
    top = y.abs().amax(-1)
    full = torch.full_like(top, 448)
    assert torch.equal(s.cpu(), top / full)
    q = (y * (full / top)[..., None]).to(E4M3)
    assert torch.equal(blocks_of(y8.float().cpu()), q.float())


def test_shapes_with_heads():
    d = ref.make(24, 128, "bf16", residual=False, before=False, seed=9)
    x = dev(d)
    y8, s, _ = run(d)
    y3, s3, _ = run(d, x={n: (t.view(6, 4, 128) if isinstance(t, torch.Tensor) and t.dim() == 2
                              else t) for n, t in x.items()})
    assert torch.equal(y8.view(6, 4, 128).float(), y3.float()) and torch.equal(s.view(6, 4, 1), s3)


def test_rows_of_zeros_and_tiny_values():
    d = ref.make(8, 256, "f32", after=False, gate="none", residual=False, before=False, scale=1.0)
    x = d["x"]
    x[0] = 0
    x[1, :128] = 0
    x[2, :128] *= 2.0 ** -120          # below what a scale holds: zeros
    x[3] *= 2.0 ** -90
    x[4] *= 2.0 ** 100
    y8, s, _ = run(d)
    assert not y8[0].float().any() and not s[0].any()
    assert not y8[1, :128].float().any() and s[1, 0] == 0 and s[1, 1] > 0
    assert not y8[2, :128].float().any() and s[2, 0] == 0 and s[2, 1] > 0
    keep = [3, 4, 5, 6, 7]
    d["x"], d["dh"] = x[keep], None
    check(d, y8[keep], s[keep])


def test_infinities_and_nan():
    d = ref.make(6, 384, "f32", after=False, gate="none", residual=False, before=False, scale=1.0)
    clean = run(d)
    d["x"][1, 5] = float("nan")
    d["x"][2, 200] = float("inf")
    d["x"][3, 383] = float("-inf")
    y8, s, _ = run(d)
    nan = torch.isnan(y8.float())
    assert nan[1, 5] and nan[1].sum() == 1
    assert torch.isinf(s[2, 1]) and nan[2, 200] and torch.isinf(s[3, 2]) and nan[3, 383]
    read = y8.float().cpu() * s.cpu().repeat_interleave(128, -1)
    assert not torch.isfinite(read[2, 128:256]).any() and not torch.isfinite(read[3, 256:]).any()
    same = torch.ones(6, 3, dtype=torch.bool)
    same[1, 0] = same[2, 1] = same[3, 2] = False
    assert torch.equal(blocks_of(y8.float().cpu())[same], blocks_of(clean[0].float().cpu())[same])
    assert torch.equal(s.cpu()[same], clean[1].cpu()[same])


@pytest.mark.parametrize("into", ["x", "gate", "residual"])
def test_h_in_place(into):
    d = ref.make(70, 512, "bf16", seed=12)
    y8, s, h = run(d, want_h=True)
    x = dev(d)
    y2, s2, _ = run(d, x=x, h=x[into])
    assert torch.equal(x[into], h) and torch.equal(y8.float(), y2.float()) and torch.equal(s, s2)


def test_no_rows():
    import gated_delta_rule_100_amd as gdr
    x = torch.empty(0, 64, device="cuda")
    gdr.gdr_block_norm8(x, x.to(E4M3), torch.empty(0, 1, device="cuda"))
    torch.cuda.synchronize()


def test_more_than_2_31_elements():
    import gated_delta_rule_100_amd as gdr
    rows, D = (1 << 31) // 4096 + 3, 4096
    say(f"norm8 rows {rows} D {D}")
    d = ref.make(3, D, "bf16", residual=False, before=False, gate="none", seed=13)
    x = torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16)
    at = [0, rows // 2, rows - 1]
    x[at] = d["x"].cuda()
    y8 = torch.empty(rows, D, device="cuda", dtype=E4M3)
    s = torch.empty(rows, D // 128, device="cuda")
    gdr.gdr_block_norm8(x, y8, s, w_after=d["w_after"].cuda(), scale=d["scale"], eps=d["eps"])
    torch.cuda.synchronize()
    check(d, torch.stack([y8[a].float() for a in at]).to(E4M3), s[at])


def test_streams_and_graph():
    import gated_delta_rule_100_amd as gdr
    d = ref.make(500, 256, "bf16", seed=14)
    x = dev(d)
    y8, s, h = run(d, want_h=True)
    y2, s2, h2 = torch.zeros_like(y8), torch.zeros_like(s), torch.zeros_like(h)

    def step(stream):
        gdr.gdr_block_norm8(x["x"], y2, s2, h2, stream=stream, **{n: x[n] for n in OPERANDS})

    def same():
        torch.cuda.synchronize()
        return torch.equal(y8.float(), y2.float()) and torch.equal(s, s2) and torch.equal(h, h2)

    torch.cuda.synchronize()
    step(torch.cuda.Stream())
    assert same()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(stream)
    for r in range(3):
        s2.fill_(float(r))
        h2.fill_(float(r))
        torch.cuda.synchronize()
        graph.replay()
        assert same(), r
