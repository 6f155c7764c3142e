"""The product in 8 bits (gdr_product8) in float64, and bounds of its rounding errors."""
import torch

F64 = torch.float64
E4M3 = torch.float8_e4m3fn
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(M, N, K, seed=0):
    """Seeded operands (CPU tensors): every e4m3 number but NaN may occur."""
    gen = torch.Generator().manual_seed(seed)
    kb = -(-K // 128)

    def values(*s):
        x = torch.randn(*s, generator=gen) * 2.0 ** torch.randint(-6, 7, s, generator=gen)
        return x.clamp(-448, 448).to(E4M3)

    def scales(*s):
        return torch.rand(*s, generator=gen) * 2.0 ** torch.randint(-12, 3, s, generator=gen)

    return dict(a=values(M, K), sa=scales(M, kb), w=values(N, K), sw=scales(-(-N // 128), kb))


def wide(d, device="cpu"):
    """Both matrices as the float64 numbers that they stand for."""
    (M, K), N = d["a"].shape, d["w"].shape[0]
    a = d["a"].to(device).to(F64) * d["sa"].to(device).to(F64).repeat_interleave(128, 1)[:, :K]
    w = d["w"].to(device).to(F64) * \
        d["sw"].to(device).to(F64).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return a, w


def product(d, device="cpu"):
    a, w = wide(d, device)
    return a @ w.T, a.abs() @ w.abs().T


def check(name, got, d, want=None):
    """Products of e4m3 numbers are exact in fp32; a block's sum has at most 128 roundings, one
    more for each block, and three for its scales.  bf16 results come from sums that keep the
    products of 8 consecutive k as multiples of 2^-13 of the largest one's power of two: each of
    the other 7 loses less than that, so together less than 7 2^-13 of the largest, and of the
    sum of absolute values all the more."""
    half = HALF[got.dtype]
    rough = 7 * 2.0 ** -13 if got.dtype == torch.bfloat16 else 0.0
    want, terms = want or product(d, got.device)
    got = got.to(F64)
    kb = d["sa"].shape[1]
    bound = ((min(128, d["a"].shape[1]) + kb + 3) * 2.0 ** -24 + rough) * terms
    assert got.shape == want.shape, name
    assert torch.isfinite(got).all(), f"{name}: not finite"
    if not got.numel():
        return
    over = (got - want).abs() - (bound + half * (want.abs() + bound) + 1e-36)
    at = int(over.argmax())
    assert over.max() <= 0, (name, at, float(got.flatten()[at]), float(want.flatten()[at]),
                             float(bound.flatten()[at]))
