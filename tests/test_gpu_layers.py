"""linear and layer_norm with their backward passes against plain 64-bit
formulas.

Tolerances count roundings.  `half(t)` is half a step of type t relative to
the value (torch.finfo(t).eps / 2); an fp32 sum in s sequential steps is off
by at most s 2^-24 times the sum of magnitudes.  Where inputs are small whole
numbers every product and sum is exact in fp32, so that the result has to be
the correctly rounded one, bit for bit."""
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


def whole(g, *shape, lim=2):
    return torch.randint(-lim, lim + 1, shape, generator=g, device="cuda").double()


def within(got, ref, tol, what=""):
    d = (got.double() - ref).abs()
    bad = d > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d - tol).max()):.3g} over " \
                          f"tolerance at {torch.nonzero(bad)[0].tolist()}"


def act64(z, name):
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


# rows, n, k: one token to several tiles; sizes that no tile, vector or
# swizzled box divides; contractions of one element and of many steps
SHAPES = [(1, 1, 1), (1, 4096, 512), (2, 129, 65), (2, 2056, 4104), (2, 2050, 4101), (5, 8, 4104),
          (16, 256, 64), (17, 130, 1000), (63, 1000, 333), (64, 136, 2048), (128, 512, 200), (129, 257, 72),
          (300, 384, 520), (777, 130, 1001), (1100, 1032, 264), (2048, 2000, 129), (3000, 2500, 64), (4097, 1304, 96)]


@pytest.mark.parametrize("rows,n,k", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (HF, F32)])
def test_linear_of_whole_numbers_is_exact(mpq, rows, n, k, dtype, out):
    g = gen(rows + n + k)
    x, w, b, r = whole(g, rows, k), whole(g, n, k), whole(g, n), whole(g, rows, n, lim=9)
    y, z = mpq.linear(x.to(dtype), w.to(dtype), b.to(F32 if out is BF else dtype), r.to(out), "relu", out, preact=True)
    want = x @ w.T + b
    assert torch.equal(z, want.to(dtype))
    assert torch.equal(y, (torch.relu(want) + r).to(out))


@pytest.mark.parametrize("rows,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_backward_of_whole_numbers_is_exact(mpq, rows, n, k, dtype):
    g = gen(rows * 3 + n + k)
    x, w, dy, z = whole(g, rows, k), whole(g, n, k), whole(g, rows, n), whole(g, rows, n)
    out = mpq.linear_backward(dy.to(dtype), x.to(dtype), w.to(dtype), z.to(dtype), "relu", bias_dtype=F32)
    dz = dy * (z > 0)
    assert torch.equal(out["dx"], (dz @ w).to(dtype))
    assert torch.equal(out["dweight"], (dz.T @ x).to(dtype))
    assert torch.equal(out["dbias"], dz.sum(0).to(F32))
    plain = mpq.linear_backward(dy.to(dtype), None, w.to(dtype), dweight=False)  # frozen, no activation
    assert set(plain) == {"dx", "dbias"}
    assert torch.equal(plain["dx"], (dy @ w).to(dtype)) and torch.equal(plain["dbias"], dy.sum(0).to(dtype))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows,n,k,dtype,out", [(3, 520, 300, BF, BF), (700, 392, 520, HF, F32), (700, 390, 521, BF, F32)])
def test_linear_activations_and_gradients(mpq, act, rows, n, k, dtype, out):
    g = gen(len(act) + rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, w = rnd(rows, k).to(dtype), (rnd(n, k) * (2.0 / k ** 0.5)).to(dtype)
    b, r, dy = rnd(n).to(dtype), rnd(rows, n).to(out), rnd(rows, n).to(dtype)
    y, z = mpq.linear(x, w, b, r, act, out, preact=True)
    z64 = (x.double() @ w.double().T + b.double()).requires_grad_()
    y64 = act64(z64, act)
    mag = x.double().abs() @ w.double().abs().T + b.double().abs()
    # the tensor core adds 16 products to the accumulator at a time, each time
    # dropping less than a step of the largest partial sum
    acc = (k / 16 + 4) * 2 * U * mag
    within(z, z64.detach(), half(dtype) * z64.detach().abs() + acc + tiny(dtype), "z")
    want = (y64 + r.double()).detach()
    # slopes are below 1.13; the activation itself is good to 2^-20
    within(y, want, half(out) * want.abs() + 1.13 * acc + 2.0 ** -20 * (y64.detach().abs() + r.double().abs()), "y")
    # gradients at the z that was kept
    zk = z.double().requires_grad_()
    yk = act64(zk, act)
    yk.backward(dy.double())
    dz = zk.grad
    h = 2.0 ** -12  # the formula against differences, away from relu's corner
    diff = (act64(zk.detach() + h, act) - act64(zk.detach() - h, act)) / (2 * h) * dy.double()
    smooth = zk.detach().abs() > 2 * h
    within(dz[smooth], diff[smooth], 4 * h * h * dy.double().abs()[smooth] + 1e-9, "formula")
    got = mpq.linear_backward(dy, x, w, z, act)
    # dz is rounded to the operands' type: independent errors of at most
    # half(t) |dz|, standard deviation half(t) |dz| / sqrt(3); six deviations.
    # The slope itself is good to 2^-20 of values up to 1.2.
    def product(a, c, name, exact_dz):
        want = a @ c
        spread = torch.sqrt(a.square() @ c.square())
        m = a.abs() @ c.abs()
        tol = half(dtype) * want.abs() + (a.shape[1] / 16 + 4) * 2 * U * m + tiny(dtype)
        if not exact_dz:
            tol = tol + 6 / math.sqrt(3) * half(dtype) * spread + 2.0 ** -19 * m + tiny(dtype) * c.abs().sum(0)
        within(got[name], want, tol, name)
    product(dz, w.double(), "dx", act in ("none", "relu"))
    product(dz.T, x.double(), "dweight", act in ("none", "relu"))
    s = dz.sum(0)
    within(got["dbias"], s, half(dtype) * s.abs() + (rows / 64 + 24) * U * dz.abs().sum(0) + 2.0 ** -19 * dy.double().abs().sum(0)
           + tiny(dtype), "dbias")


@pytest.mark.parametrize("rows,n,k", [(300, 1031, 1999), (777, 1032, 8192), (40, 300, 14336), (1, 200, 14336), (130, 128, 8192)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_of_long_contractions_keeps_fp32(mpq, rows, n, k, dtype):
    """fp32 results of long contractions: chains of 512 products lose at most a last bit of the accumulator at each
    of 32 steps (2^-23 of a partial sum, half of that on average), and are then added with rounding, k / 512 times.
    Over many results the error in the 2-norm stays near 16 half bits, 16 * 2^-24, of the partial sums' size, which
    for independent terms is the result's; twice that is allowed."""
    g = gen(k)
    x = torch.randn(rows, k, generator=g, device="cuda").to(dtype)
    w = (torch.randn(n, k, generator=g, device="cuda") / k ** 0.5).to(dtype)
    y = mpq.linear(x, w, out_dtype=F32).double()
    want = x.double() @ w.double().T
    assert (y - want).norm() <= 32 * U * want.norm()


def test_linear_takes_slices_batches_and_shared_rows(mpq):
    g = gen(7)
    x3, wide = whole(g, 3, 5, 80).to(BF), whole(g, 70, 99).to(BF)
    w, odd = wide[:, :80], wide[:, 3:83]          # aligned start and not, stride of 99 elements
    for wt in (w, odd):
        y = mpq.linear(x3, wt)
        assert y.shape == (3, 5, 70) and torch.equal(y, (x3.double() @ wt.double().T).to(BF))
    one = whole(g, 1, 80).to(BF).expand(300, 80)  # one row for all
    assert torch.equal(mpq.linear(one, w), (one.double() @ w.double().T).to(BF))
    r = whole(g, 300, 200).to(BF)[:, 7:77]
    b = whole(g, 90).to(BF)[3:73]
    assert torch.equal(mpq.linear(one, w, b, r), (one.double() @ w.double().T + b.double() + r.double()).to(BF))
    dy = whole(g, 300, 101).to(BF)[:, 1:71]
    zz = whole(g, 300, 73).to(BF)[:, 2:72]
    xs = whole(g, 300, 83).to(BF)[:, :80]
    out = mpq.linear_backward(dy, xs, odd, zz, "relu")
    dz = dy.double() * (zz > 0)
    assert torch.equal(out["dx"], (dz @ odd.double()).to(BF)) and torch.equal(out["dbias"], dz.sum(0).to(BF))
    assert torch.equal(out["dweight"], (dz.T @ xs.double()).to(BF))


def test_linear_without_rows(mpq):
    w = torch.ones(6, 8, dtype=BF, device="cuda")
    x = torch.ones(0, 8, dtype=BF, device="cuda")
    assert mpq.linear(x, w).shape == (0, 6)
    out = mpq.linear_backward(torch.ones(0, 6, dtype=BF, device="cuda"), x, w)
    assert out["dx"].shape == (0, 8) and not out["dweight"].any() and not out["dbias"].any()


def test_linear_keeps_infinities_and_nans_to_their_rows(mpq):
    g = gen(9)
    for rows in (3, 400):
        x, w = whole(g, rows, 96).to(BF), whole(g, 300, 96).abs().add(1).to(BF)
        x[0, 5], x[2, 95] = math.nan, math.inf
        y = mpq.linear(x, w)
        assert torch.isnan(y[0]).all() and torch.isinf(y[2]).all() and torch.isfinite(y[1]).all()
        assert torch.equal(y[1:2], (x[1:2].double() @ w.double().T).to(BF)) and torch.isfinite(y[3:]).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("rows", [1, 40, 300])  # a kernel each
def test_linear_activations_at_infinity(mpq, act, rows):
    """z = +inf, -inf, NaN: the limits inf, 0 and NaN, and slopes 1, 0 and NaN."""
    x = torch.ones(rows, 64, device="cuda", dtype=BF)
    w = torch.zeros(16, 64, device="cuda", dtype=BF)
    w[0, 3], w[1, 3], w[2, 3], w[3, 3], w[4, 3] = math.inf, -math.inf, math.nan, 1e30, -1e30
    want = torch.tensor([math.inf, 0, math.nan, w[3, 3].item()] + [0] * 12, device="cuda", dtype=BF).expand(rows, 16)
    y, z = mpq.linear(x, w, activation=act, preact=True)
    assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(want, nan=7.0))
    d = mpq.linear_backward(torch.ones_like(y), None, None, z, activation=act, dx=False, dweight=False,
                            bias_dtype=torch.float32)["dbias"]
    # slopes are taken at |z| <= 30: 29 e^-30 = 2.8e-12 is left of silu's there; a rounding or two of 1 + e^-30
    assert torch.isnan(d[2])
    torch.testing.assert_close(d[[0, 1, 3, 4]], torch.tensor([rows, 0, rows, 0], device="cuda", dtype=F32),
                               rtol=2**-21, atol=3e-12 * rows)


# ------------------------------------------------------------- layer norm --
LN = [(1, 1), (1, 16), (3, 5), (33, 64), (700, 17), (9, 256), (130, 257), (5, 1000), (300, 1024), (64, 4096), (1, 8192),
      (7, 8200), (3, 16384), (2, 16400), (5, 32768), (3, 40001)]


def ln64(x, w, b, eps):
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + eps)
    return (x - mean) * rstd * w + b, mean, rstd


@pytest.mark.parametrize("rows,n", LN)
@pytest.mark.parametrize("dtype,param", [(BF, F32), (HF, HF), (F32, F32)])
def test_layer_norm_and_gradients(mpq, rows, n, dtype, param):
    g = gen(rows * 7 + n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = (rnd(rows, n) * 2 + 3 * rnd(rows, 1)).to(dtype)
    w, b, dy = (1 + 0.3 * rnd(n)).to(param), rnd(n).to(param), rnd(rows, n).to(dtype)
    eps = 1e-3
    y, mean, rstd = mpq.layer_norm(x, w, b, eps, stats=True)
    x64, w64, b64 = x.double(), w.double(), b.double()
    want, m64, r64 = ln64(x64, w64, b64, eps)
    ax = x64.abs().mean(-1, keepdim=True)
    steps = 64 + n / 1024  # sequential adds per thread and levels of the tree, twice over
    within(mean, m64[:, 0], steps * U * ax[:, 0] + tiny(F32), "mean")
    within(rstd, r64[:, 0], 2 * steps * U * r64[:, 0], "rstd")
    xh = (x64 - m64) * r64
    tol = half(dtype) * want.abs() + U * (steps * ax * r64 + (2 * steps + 8) * xh.abs()) * w64.abs() + 4 * U * b64.abs()
    within(y, want, tol + tiny(dtype), "y")

    got = mpq.layer_norm_backward(dy, x, mean, rstd, w)
    xh = (x64 - mean.double()[:, None]) * rstd.double()[:, None]  # from the statistics that were kept
    gr = dy.double() * w64
    dx = rstd.double()[:, None] * (gr - gr.mean(-1, keepdim=True) - xh * (gr * xh).mean(-1, keepdim=True))
    size = rstd.double()[:, None] * (gr.abs() + gr.abs().mean(-1, keepdim=True)
                                     + xh.abs() * (gr * xh).abs().mean(-1, keepdim=True))
    # (x - mean) is off by a rounding of x's own size where x nearly cancels
    off = U * (x64.abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
    within(got["dx"], dx, half(dtype) * dx.abs() + 2 * steps * U * size + tiny(dtype), "dx")
    dw, db = (dy.double() * xh).sum(0), dy.double().sum(0)
    adds = rows / 64 + 64
    within(got["dweight"], dw, half(param) * dw.abs() + ((adds + 4) * U * (dy.double() * xh).abs()
                                                        + off * dy.double().abs()).sum(0) + tiny(param), "dweight")
    within(got["dbias"], db, half(param) * db.abs() + adds * U * dy.double().abs().sum(0) + tiny(param), "dbias")
    if n > 1:  # the formula against autograd of the definition
        leaf, wl = x64.clone().requires_grad_(), w64.clone().requires_grad_()
        ln64(leaf, wl, b64, eps)[0].backward(dy.double())
        within(dx, leaf.grad, 1e-4 * size + 1e-9, "formula")
        within(dw, wl.grad, 1e-4 * (dy.double() * xh).abs().sum(0) + 1e-6 * dy.double().abs().sum(0), "formula of dweight")


def test_layer_norm_gradient_against_differences(mpq):
    g = gen(3)
    x = torch.randn(6, 40, generator=g, device="cuda")
    w, b, dy, d = (torch.randn(*s, generator=g, device="cuda") for s in ((40,), (40,), (6, 40), (6, 40)))
    y, mean, rstd = mpq.layer_norm(x, w, b, stats=True)
    got = mpq.layer_norm_backward(dy, x, mean, rstd, w)
    h = 2.0 ** -10
    f = lambda t: (ln64(t, w.double(), b.double(), 1e-5)[0] * dy.double()).sum()
    slope = float((f(x.double() + h * d.double()) - f(x.double() - h * d.double())) / (2 * h))
    have = float((got["dx"].double() * d.double()).sum())
    # third derivatives of x/|x| are a few times |dy w| rstd^3 |d|^3: h^2 of that, and fp32's roundings
    size = float((dy * w).double().abs().sum() * rstd.double().max() ** 3 * d.double().abs().max() ** 3)
    assert abs(slope - have) <= h * h * 4 * size + 1e-4 * size * 2.0 ** -8, (slope, have)


@pytest.mark.parametrize("n", [48, 1001, 4096, 12000, 20000])
def test_layer_norm_slices_missing_parameters_and_edges(mpq, n):
    g = gen(n)
    wide = torch.randn(4, 3, n + 5, generator=g, device="cuda").to(BF)
    x = wide[..., 1:n + 1]
    y = mpq.layer_norm(x)
    # other layouts may take other orders of the same fp32 sums: both results are within 128 roundings of the
    # magnitudes that go into them, so within twice that and one step of bf16 of each other
    x64 = x.double()
    y2, m2, r2 = mpq.layer_norm(x.contiguous(), stats=True)
    scale = x64.abs().mean(-1, keepdim=True) * r2[..., None] + y2.double().abs()
    within(y, y2.double(), 2 * half(BF) * y2.double().abs() + 256 * U * scale, "y")
    assert y.shape == (4, 3, n) and m2.shape == (4, 3)
    one, zero = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    assert torch.equal(y, mpq.layer_norm(x, one, zero))
    y, mean, rstd = mpq.layer_norm(x, stats=True)
    dy = torch.randn(4, 3, n + 3, generator=g, device="cuda").to(BF)[..., 2:n + 2]
    a = mpq.layer_norm_backward(dy, x, mean, rstd, param_dtype=F32)
    c = mpq.layer_norm_backward(dy.contiguous(), x.contiguous(), mean, rstd, one)
    # other layouts may take other orders of the same fp32 sums: each is within 128 roundings of its magnitudes
    # (12 rows, 64 levels and chains), so the two are within twice that, and one step of bf16 apart at most
    xh, m = (x.double() - mean.double()[..., None]).abs() * rstd.double()[..., None], dy.double().abs()
    size = rstd.double()[..., None] * (m + m.mean(-1, keepdim=True) + xh * (m * xh).mean(-1, keepdim=True))
    within(a["dx"], c["dx"].double(), 2 * half(BF) * c["dx"].double().abs() + 256 * U * size, "dx")
    within(a["dweight"], c["dweight"].double(), 256 * U * (m * xh).sum((0, 1)), "dweight")
    within(a["dbias"], c["dbias"].double(), 256 * U * m.sum((0, 1)), "dbias")
    only = mpq.layer_norm_backward(dy, x, mean, rstd, dweight=False, dbias=False)
    assert set(only) == {"dx"}
    within(only["dx"], c["dx"].double(), 2 * half(BF) * c["dx"].double().abs() + 256 * U * size, "dx alone")
    # a constant row has variance 0: y is the bias; a NaN stays in its row
    z = torch.full((3, n), 2.5, device="cuda", dtype=F32)
    z[1, n // 2] = math.nan
    y = mpq.layer_norm(z, one, zero + 4.0)
    assert (y[0] == 4).all() and (y[2] == 4).all() and torch.isnan(y[1]).all()
    empty = mpq.layer_norm_backward(dy[:0], x[:0], mean[:0], rstd[:0], one)
    assert empty["dx"].shape == (0, 3, n) and not empty["dweight"].any() and not empty["dbias"].any()


def test_layer_norm_of_a_far_mean(mpq):
    # the variance is taken around the mean: a mean of 1000 deviations costs
    # the roundings of x - mean only
    g = gen(5)
    x = 1000 + torch.randn(16, 5000, generator=g, device="cuda")
    y = mpq.layer_norm(x)
    want = ln64(x.double(), 1.0, 0.0, 1e-5)[0]
    within(y, want, 80 * U * 1000 + 2.0 ** -20 * want.abs(), "y")


# --------------------------------------------------------- how calls behave --
def test_refusals(mpq):
    c = lambda *s, t=BF: torch.ones(*s, dtype=t, device="cuda")
    bad = [lambda: mpq.linear(c(2, 8, t=F32), c(4, 8, t=F32)), lambda: mpq.linear(c(2, 8), c(4, 9)),
           lambda: mpq.linear(c(2, 8), c(4, 8, t=HF)), lambda: mpq.linear(c(2, 8), c(4, 8), c(5)),
           lambda: mpq.linear(c(2, 8), c(4, 8), c(4, t=HF)), lambda: mpq.linear(c(2, 8), c(4, 8), residual=c(2, 5)),
           lambda: mpq.linear(c(2, 8), c(4, 8), residual=c(2, 4, t=F32)), lambda: mpq.linear(c(2, 8), c(4, 8), activation="tanh"),
           lambda: mpq.linear(c(2, 8), c(4, 8), out_dtype=HF), lambda: mpq.linear(c(8, 2).T, c(4, 8)),
           lambda: mpq.linear(c(2, 8).cpu(), c(4, 8)), lambda: mpq.linear(c(2, 8), c(4, 8).cpu()),
           lambda: mpq.linear(c(2, 3, 4, 8).transpose(0, 2), c(4, 8)), lambda: mpq.linear(c(2, 0), c(4, 0)),
           lambda: mpq.linear_backward(c(2, 4), None, c(4, 8)), lambda: mpq.linear_backward(c(2, 4), c(2, 8), c(4, 8), activation="silu"),
           lambda: mpq.linear_backward(c(2, 4), c(3, 8), c(4, 8)), lambda: mpq.linear_backward(c(2, 4), c(2, 9), c(4, 8)),
           lambda: mpq.layer_norm(c(2, 8), c(7)), lambda: mpq.layer_norm(c(2, 8), c(8), c(8, t=F32)),
           lambda: mpq.layer_norm(c(2, 8), c(8, t=HF)), lambda: mpq.layer_norm(c(2, 8), eps=0.0),
           lambda: mpq.layer_norm(c(2, 8, t=torch.float64)), lambda: mpq.layer_norm(c(2, 0)),
           lambda: mpq.layer_norm_backward(c(2, 8), c(2, 8), c(2, t=F32), c(3, t=F32)),
           lambda: mpq.layer_norm_backward(c(2, 8), c(2, 8), c(2), c(2)),
           lambda: mpq.layer_norm_backward(c(2, 8), c(2, 8), c(2, t=F32), c(2, t=F32), c(8), param_dtype=F32)]
    before = mpq.kernel_launch_count()
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was accepted")
    assert mpq.kernel_launch_count() == before


def test_repeatable_on_other_streams_and_in_graphs(mpq):
    g = gen(11)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    x, w, dy = mk(500, 512), mk(640, 512), mk(500, 640)
    odd = mk(640, 511)
    gw = 1 + mk(512)

    def step():
        h, mean, rstd = mpq.layer_norm(x, gw, stats=True)
        y, z = mpq.linear(h, w, activation="gelu", preact=True)
        d = mpq.linear_backward(dy, h, w, z, "gelu")
        e = mpq.layer_norm_backward(d["dx"], x, mean, rstd, gw)
        return [y, z, d["dx"], d["dweight"], d["dbias"], e["dx"], e["dweight"], e["dbias"],
                mpq.linear(x[:, 1:], odd), mpq.linear(x[:3], w, residual=y[:3])]

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    again = step()  # both streams at work
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, again):
        assert torch.equal(a, b) and torch.equal(a, c)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step()
        graphs.append((gr, out))
    for t in (x, w, dy, gw):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(BF))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for (gr, _), s in zip(graphs, streams):  # two graphs share no scratch
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    want = step()
    for a, b, c in zip(want, graphs[0][1], graphs[1][1]):
        assert torch.equal(a, b) and torch.equal(a, c)
    mpq.ops_status()


def test_rows_past_32_bit_offsets(mpq):
    # 2^32 + elements: the last rows are far beyond 32-bit offsets
    rows, n = 70001, 65536 // 2
    x = torch.zeros(rows * 2, n, dtype=BF, device="cuda")  # 4.6e9 elements
    g = gen(1)
    tail = whole(g, 3, n).to(BF)
    x[-3:] = tail
    y = mpq.layer_norm(x)
    assert torch.equal(y[-3:], mpq.layer_norm(tail)) and not y[:5].any()
    del y
    w = whole(g, 16, n).to(BF)
    y = mpq.linear(x, w, out_dtype=F32)
    assert torch.equal(y[-3:], (tail.double() @ w.double().T).float()) and not y[:-3].any()
