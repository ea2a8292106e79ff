"""The 8-bit output head where it can go wrong: values halfway between two codes, products of several
tiles a CTA."""
import numpy as np
import pytest
import torch

from canvas_sampler_gb300 import head
from oracle import head as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------------------------- codes
def quotients(y, fmt, block_rows):
    """y / scale in 64 bits as y F / max, which is exact where it lies halfway between two codes."""
    R, C = y.shape
    m = np.empty_like(y)
    for i in range(0, R, block_rows):
        for j in range(0, C, 128):
            at = np.s_[i:i + block_rows, j:j + 128]
            m[at] = max(np.abs(y[at]).max(), O.TINY)
    return y * O.FORMATS[fmt][2] / m


def ties(v, fmt):
    """How many of v lie exactly halfway between two codes."""
    x = np.abs(v) / O.fp8_step(v, fmt)
    return int(np.sum(x - np.floor(x) == 0.5))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_codes_of_a_matrix_are_those_of_the_quotient(dt, block_rows, fmt):
    """The quotient is known to 2^-44, so its fp32 rounding, and with it the code, is the definition's
    unless the quotient lies within 2^-44 of the middle between two fp32 numbers: none of these do."""
    g = gen(31)
    for R, C, shift in ((512, 2816, 0), (200, 1111, 1)):
        buf = (torch.randn(R * C + shift, device="cuda", generator=g) / 16).to(DT[dt])
        x = buf[shift:].view(R, C)
        x[3] = x[3] * 2.0 ** 20
        x[5] = 0
        x[128:256, 128:256] *= 2.0 ** -80
        q, s = head.quantize_fp8(x, block_rows=block_rows, fp8=fmt)
        v = quotients(f64(x), fmt, block_rows)
        assert dt == "fp32" or C != 2816 or ties(v, fmt) > 20  # what this is about
        assert np.array_equal(f64(q), O.fp8_round(v.astype(np.float32), fmt))
        half = 2.0 ** -24  # the scale is one division
        want = O.block_scales(f64(x), fmt, block_rows)
        assert np.all(np.abs(f64(s) - want) <= half * want)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("R,d", [(256, 2816), (40, 5000), (33, 515), (7, 8200)])
def test_codes_of_a_norm_see_one_rounding(dt, fmt, R, d):
    """1 / sqrt(mean + eps) divides out of y / scale. What is left is h (offset + w), rounded to fp32
    once (2^-24 of it, in the element and in the block's maximum), and the quotient's own rounding
    (2^-24): codes are those of the quotient moved by no more than 3 2^-24, and of the quotient itself
    where the product is exact (two bf16 factors)."""
    g = gen(R + d)
    x = torch.randn(R, d, device="cuda", generator=g).to(DT[dt])
    res = (4 * torch.randn(R, d, device="cuda", generator=g)).to(DT[dt])
    for off, scale in ((0.0, 1.0), (1.0, 0.2)):
        w = (scale * torch.randn(d, device="cuda", generator=g)).to(DT[dt])
        q, s, h = head.rmsnorm_fp8(x, w, res, weight_offset=off, fp8=fmt)
        got, v = f64(q), quotients(f64(h) * (off + f64(w)), fmt, 1)
        if dt == "bf16" and off == 0.0:
            assert np.array_equal(got, O.fp8_round(v.astype(np.float32), fmt))
        slack = 1 + 3 * 2.0 ** -24
        a, b = O.fp8_round(v / slack, fmt), O.fp8_round(v * slack, fmt)
        assert np.all((got == a) | (got == b))
        assert np.mean(a != b) < 1e-2  # nearly every code is pinned to one value (ties to two)


# ------------------------------------------------------------------------------------- product
def operands(m, n, k, seed):
    """Codes and scales of an A [m, k] and a B [n, k]."""
    g = gen(seed)
    cols = -(-k // 16) * 16
    code = lambda r: (torch.randn(r, cols, device="cuda", generator=g) * 100).clamp(-400, 400).to(  # noqa: E731
        torch.float8_e4m3fn)[:, :k]
    scale = lambda r: torch.exp(torch.randn(r, -(-k // 128), device="cuda", generator=g)) / 100  # noqa: E731
    return code(m), scale(m), code(n), scale(-(-n // 128))


# with 152 SMs: the first five have two and more 64-column tiles a CTA, the next three 128-column
# ones, the last 256-column ones of CTA pairs
@pytest.mark.parametrize("m,n,k", [(300, 6464, 128), (1409, 1600, 128), (20000, 64, 128), (25000, 120, 160),
                                   (640, 7688, 256), (40000, 128, 128), (300, 14000, 128), (1409, 3200, 128),
                                   (1409, 12000, 128)])
def test_products_of_several_tiles_a_cta(m, n, k):
    """The same sums leave in both types: the bf16 product is the fp32 one rounded."""
    for seed in range(3):
        ops = operands(m, n, k, seed)
        full = head.matmul_fp8(*ops, out_dtype="fp32")
        for _ in range(3):
            out = torch.full((m, n), 7.0, dtype=torch.bfloat16, device="cuda")
            assert torch.equal(head.matmul_fp8(*ops, out=out), full.bfloat16())
    # and the fp32 ones are the definition's: sums of 128 products cut to no worse than 2^-23 of their
    # absolute terms each, one addition a block, half a step of the output
    rows = torch.arange(0, m, max(1, m // 50), device="cuda")
    want, mag = O.matmul(f64(ops[0][rows]), f64(ops[1][rows]), f64(ops[2]), f64(ops[3]))
    bound = (128 + ops[1].shape[1]) * 2.0 ** -23 * mag
    assert np.all(np.abs(f64(full[rows]) - want) <= bound + 2.0 ** -24 * (np.abs(want) + bound))
    assert head.head_status() == 0


# ------------------------------------------------------------------------------------- sampling
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("R", [2, 400])
def test_sampling_with_thousands_of_ties_at_the_kth_logit(dt, R):
    """The list overflows, and top-p is a share of the first k tokens, the lowest indices of the tie."""
    V, k = 20011, 50
    g = gen(R)
    logits = torch.randn(R, V, device="cuda", generator=g).clamp(max=0.25)
    logits[:, 7000] = 1.5
    logits = logits.to(DT[dt])
    u = torch.rand(R, device="cuda", generator=g)
    full = lambda v, t=torch.float32: torch.full((R,), v, dtype=t, device="cuda")  # noqa: E731
    for p in (0.77, 0.3):
        token, prob = head.sample_logits(logits, u, top_k=full(k, torch.int32), top_p=full(p))
        for r in range(0, R, max(1, R // 20)):
            want, pw, margin = O.sample_row(f64(logits[r]), float(u[r]), top_k=k,
                                            top_p=float(np.float32(p)))
            assert margin > 2.0 ** -24 and int(token[r]) == want
            assert abs(float(prob[r]) - pw) <= 2.0 ** -20 * pw
