"""dz = dy act'(z) of linear_backward reaches the products to more than its 16
bits: gradients against plain 64-bit formulas, with no room for a rounding of dz.

Tolerances: dz in two parts of type t is off by half(t)^2 of a value (fp16: and
half of its smallest number); the slope is good to 2^-20 of values up to 1.2.
The tensor cores add 16 products at a time, each time dropping less than a step
of the largest partial sum; the result is rounded once."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):  # half the spacing of t's smallest numbers
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def slope64(z, name):
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    u, du = z, torch.ones_like(z)
    if name == "gelu_tanh":
        a = 2 * math.sqrt(2 / math.pi)
        u, du = a * (z + 0.044715 * z ** 3), a * (1 + 0.134145 * z * z)
    s = torch.sigmoid(u)
    return s + z * s * (1 - s) * du


def near(got, a, b, t, what):
    """got: a b, with a in two parts"""
    want, m = a @ b, a.abs() @ b.abs()
    tol = half(t) * want.abs() + (half(t) ** 2 + 2.0 ** -19 + (2 * a.shape[1] / 16 + 4) * 2 * U) * m + tiny(t)
    if t is HF:
        tol = tol + 2 * tiny(t) * b.abs().sum(0)
    d = (got.double() - want).abs()
    assert (d <= tol).all(), f"{what}: {int((d > tol).sum())} of {d.numel()} off, worst {float((d / tol).max()):.3g} tolerances"


# tiles by clusters (up to 32 rows and more) and by CTA pairs, unaligned rows
@pytest.mark.parametrize("rows,n,k", [(1, 40, 24), (3, 520, 300), (20, 4104, 256), (100, 1000, 136), (700, 392, 520), (701, 391, 521), (2500, 2600, 1304)])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_gradients_hold_dz_beyond_16_bits(mpq, rows, n, k, act, dtype):
    g = gen(rows + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w = rnd(rows, k).to(dtype), (rnd(n, k) / 8).to(dtype)
    dy, z = rnd(rows, n).to(dtype), (1.5 * rnd(rows, n)).to(dtype)
    dz = dy.double() * slope64(z.double(), act)
    got = mpq.linear_backward(dy, x, w, z, act, bias_dtype=F32)
    near(got["dx"], dz, w.double(), dtype, "dx")
    near(got["dweight"], dz.T, x.double(), dtype, "dweight")
    frozen = mpq.linear_backward(dy, None, w, z, act, dweight=False)
    assert torch.equal(frozen["dx"], got["dx"])
    # rounded where the caller asks for it: the product of the rounded dz, within the slope's own 2^-20, which may
    # turn a rounding
    low = mpq.linear_backward(dy, x, w, z, act, bias_dtype=F32, round_dz=True)
    m = dz.abs() @ w.double().abs()
    off = (low["dx"].double() - dz @ w.double()).abs()
    assert (off <= half(dtype) * (dz @ w.double()).abs() + (half(dtype) + 2.0 ** -19 + (n / 16 + 4) * 2 * U) * m + tiny(dtype)
            + 2 * tiny(dtype) * w.double().abs().sum(0)).all()
    assert torch.equal(low["dbias"], got["dbias"])


def test_gradients_past_the_range_of_fp16(mpq):
    """dy is at fp16's largest value, dz = dy * 1.128 passes it, dx and dweight do not."""
    for rows in (4, 300):
        n, k = 8, 72
        dy = torch.zeros(rows, n, dtype=HF, device="cuda")
        dy[:, 1], dy[:, 2] = 65504, -65504
        z = torch.full((rows, n), 1.4, dtype=HF, device="cuda")
        w = torch.zeros(n, k, dtype=HF, device="cuda")
        w[1, :3], w[2, 3:5] = 0.5, 0.25
        x = torch.full((rows, k), 2.0 ** -9, dtype=HF, device="cuda")
        dz = dy.double() * slope64(z.double(), "gelu")
        assert float(dz.abs().max()) > 65520
        got = mpq.linear_backward(dy, x, w, z, "gelu")
        near(got["dx"], dz, w.double(), HF, "dx")
        near(got["dweight"], dz.T, x.double(), HF, "dweight")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_infinite_and_nan_dz_keep_to_their_rows(mpq, dtype):
    g = gen(3)
    for rows in (6, 300):
        dy = torch.randn(rows, 64, generator=g, device="cuda").to(dtype)
        dy[0, 3], dy[1, 5] = math.inf, math.nan
        w = (torch.rand(64, 80, generator=g, device="cuda") + 0.5).to(dtype)
        z = torch.ones_like(dy)
        dx = mpq.linear_backward(dy, None, w, z, "silu", dweight=False)["dx"]
        assert (dx[0] == math.inf).all() and torch.isnan(dx[1]).all() and torch.isfinite(dx[2:]).all()
