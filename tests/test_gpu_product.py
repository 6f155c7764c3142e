"""The product in 8 bits on the GPU against float64, elementwise within product_ref's bounds."""
import pytest
import torch

import product_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


def cuda(d):
    return {n: t.cuda() for n, t in d.items()}


def run(d, dtype=torch.float32, **kw):
    import gated_delta_rule_100_amd as gdr
    x = cuda(d)
    out = torch.full((d["a"].shape[0], d["w"].shape[0]), float("nan"), dtype=dtype, device="cuda")
    gdr.gdr_product8(x["a"], x["sa"], x["w"], x["sw"], out, **kw)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257, 600])
@pytest.mark.parametrize("N, K", [(1, 16), (100, 128), (128, 144), (257, 1040), (1000, 2064),
                                  (512, 4096)])
def test_sizes(M, N, K):
    say(f"product M {M} N {N} K {K}")
    d = ref.make(M, N, K, seed=M + N + K)
    for dtype in (torch.float32, torch.bfloat16):
        ref.check(f"{M} {N} {K}", run(d, dtype), d)


@pytest.mark.parametrize("K", [16, 32, 48, 112, 128, 144, 240, 256, 272, 384, 400, 512, 528])
@pytest.mark.parametrize("M", [3, 48, 130, 300])
def test_depths(M, K):
    say(f"product M {M} K {K}")
    d = ref.make(M, 200, K, seed=K)
    ref.check(f"{M} {K}", run(d), d)


# a size for each shape of workgroup: rows of 16 x 16 and 16 x 32, tiles of 32, 64, 64 x 128,
# 128 and (bf16 results) 256
SHAPES = [(40, 100), (100, 1000), (128, 2000), (300, 1000), (1000, 2000), (2000, 4000), (4100, 4100)]


@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 272, 400, 512, 528, 1024, 1152, 2064])
@pytest.mark.parametrize("M, N", SHAPES)
def test_depths_of_every_shape(M, N, K):
    """One block, blocks that do not go round the groups of waves, last blocks that are not
    whole, one group of eight scales and more."""
    say(f"product M {M} N {N} K {K}")
    d = ref.make(M, N, K, seed=K + M)
    x = cuda(d)
    want = ref.product(x, "cuda")
    for dtype in (torch.float32, torch.bfloat16):
        ref.check(f"{M} {N} {K}", run(d, dtype), d, want)


@pytest.mark.parametrize("M, N, K", [(4096, 2048, 2048), (2048, 4100, 1024), (3000, 1024, 8192),
                                     (1024, 128, 640), (8, 16384, 512), (40, 200, 16384)])
def test_large(M, N, K):
    say(f"product M {M} N {N} K {K}")
    d = ref.make(M, N, K, seed=1)
    x = cuda(d)
    want = ref.product(x, "cuda")
    ref.check("f32", run(d), d, want)
    ref.check("bf16", run(d, torch.bfloat16), d, want)


@pytest.mark.parametrize("M, N", [(5, 270), (70, 270), (700, 270)] + SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_and_columns_by_themselves(M, N, dtype):
    """NaN and infinite scales, NaN values and zero scales touch their own row or column only."""
    if N < 270:
        N = 270
    d = ref.make(M, N, 400, seed=2)
    clean = run(d, dtype)
    d["sa"][1, 2], d["sa"][M - 1, 0] = float("nan"), float("inf")
    d["a"].view(torch.uint8)[3, 17] = 0x7F
    d["w"].view(torch.uint8)[200, 399] = 0xFF
    got = run(d, dtype)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1] = bad[3] = bad[M - 1] = True
    bad[:, 200] = True
    assert torch.equal(got[~bad], clean[~bad]) and not torch.isfinite(got[bad]).any()
    d = ref.make(M, N, 400, seed=3)
    d["sa"][2] = 0
    d["sw"][1] = 0
    got = run(d, dtype)
    assert not got[2].any() and not got[:, 128:256].any()
    ref.check("zero scales", got, d, ref.product(cuda(d), "cuda"))


def test_whole_range_of_scales():
    """Scales far apart: no product of two of them is lost before it meets the sum."""
    d = ref.make(40, 40, 256, seed=4)
    d["sa"] = torch.full_like(d["sa"], 2.0 ** 60)
    d["sw"] = torch.full_like(d["sw"], 2.0 ** -90)
    ref.check("far apart", run(d), d)


@pytest.mark.parametrize("M, N, K", [(64, 1000, 2064), (700, 500, 1040), (5, 128, 4096)] +
                         [(*s, 1040) for s in SHAPES])
def test_repeated_streams_and_graph(M, N, K):
    import gated_delta_rule_100_amd as gdr
    d = ref.make(M, N, K, seed=5)
    x = cuda(d)
    out = run(d, torch.bfloat16)
    got = torch.empty_like(out)

    def step(stream=None):
        gdr.gdr_product8(x["a"], x["sa"], x["w"], x["sw"], got, stream=stream)

    def same():
        torch.cuda.synchronize()
        return torch.equal(out, got)

    torch.cuda.synchronize()
    step(torch.cuda.Stream())
    assert same()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=stream):
        step(stream)
    for r in range(4):
        got.fill_(float(r))
        torch.cuda.synchronize()
        graph.replay()
        assert same(), r


def test_no_rows():
    d = ref.make(3, 10, 32, seed=6)
    d["a"], d["sa"] = d["a"][:0], d["sa"][:0]
    assert run(d).shape == (0, 10)


@pytest.mark.parametrize("which", ["a", "w", "out"])
def test_more_than_2_31_elements(which):
    import gated_delta_rule_100_amd as gdr
    M, N, K = dict(a=(1 << 20, 24, 2064), w=(40, 1 << 20, 2064), out=(1 << 16, (1 << 15) + 8, 144))[which]
    say(f"product M {M} N {N} K {K}")
    gen = torch.Generator(device="cuda").manual_seed(7)

    def bits(*s):
        x = torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=gen)
        x[(x & 127) == 127] = 0
        return x.view(ref.E4M3)

    kb = -(-K // 128)
    a, w = bits(M, K), bits(N, K)
    sa = torch.rand(M, kb, device="cuda", generator=gen)
    sw = torch.rand(-(-N // 128), kb, device="cuda", generator=gen)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    gdr.gdr_product8(a, sa, w, sw, out)
    torch.cuda.synchronize()
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    at = torch.cat([torch.arange(128), N // 256 * 128 + torch.arange(128), torch.arange(N - 1 - (N - 1) % 128, N)]) \
        if N > 1000 else torch.arange(N)
    at = at.cuda()

    def take(t, i):  # (rows of 8 bits, picked as bytes)
        return t.view(torch.uint8)[i].view(ref.E4M3)

    d = dict(a=take(a, rows), sa=sa[rows], w=take(w, at),
             sw=sw[at[::128] // 128] if N > 1000 else sw)
    ref.check(which, out[rows][:, at], d)


@pytest.mark.parametrize("N, K, times, dtype", [(65544, 144, 71, torch.bfloat16),
                                                (65544, 144, 71, torch.float32),
                                                (136, 8192, 600, torch.bfloat16)])
def test_more_than_2_32(N, K, times, dtype):
    """More than 2^32 results, and more than 2^32 bytes of rows: the same 1000 rows again and again."""
    import gated_delta_rule_100_amd as gdr
    say(f"product {times * 1000} {N} {K} {dtype}")
    d = ref.make(1000, N, K, seed=K)
    x = cuda(d)
    a = x["a"].view(torch.uint8).repeat(times, 1).view(ref.E4M3)
    out = torch.full((times * 1000, N), float("nan"), dtype=dtype, device="cuda")
    gdr.gdr_product8(a, x["sa"].repeat(times, 1), x["w"], x["sw"], out)
    torch.cuda.synchronize()
    ref.check("first", out[:1000], d, ref.product(x, "cuda"))
    for i in range(1, times):
        assert torch.equal(out[i * 1000:(i + 1) * 1000], out[:1000]), i
