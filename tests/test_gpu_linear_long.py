"""linear and its gradients over long contractions and over more tiles than
there are workers, against plain 64-bit formulas.

The tensor cores add 16 products to an accumulator at a time and drop what
falls below its last bit: less than 2^-23 of the partial sum each time, always
towards zero.  A chain of 4096 products so loses at most 256 * 2^-23 of its own
sum of magnitudes, whatever the whole contraction's length; the chains are then
added with rounding, k / 4096 times, each 2^-24 of what is summed so far."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(g, *shape, lim=2):
    return torch.randint(-lim, lim + 1, shape, generator=g, device="cuda").double()


def long_sum_is_near(got, want, length, t):
    """`want`: sums of `length` terms of one sign (so the magnitudes' sum is the result's).  The fp32 sum lies within
    `lost` of them, and rounding keeps order: each result lies between the roundings of the two ends.  (Nothing is
    left for half a step: the results lie close together, where a loss shows as a rounding to the other side.)"""
    lost = (256 * 2 + length / 4096) * U
    lo, hi = (want * (1 - lost)).to(t), (want * (1 + lost)).to(t)
    bad = (got < lo) | (got > hi)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"


# by CTA pairs; by clusters that share the contraction, tiles of up to 32 rows and of more
@pytest.mark.parametrize("rows,n,k", [(300, 520, 1 << 18), (16, 128, 1 << 20), (128, 96, 1 << 20)])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_linear_of_one_sign_over_a_long_contraction(mpq, rows, n, k, dtype):
    g = gen(k + rows)
    x = torch.rand(rows, k, generator=g, device="cuda").to(dtype)
    w = (torch.rand(n, k, generator=g, device="cuda") / 256).to(dtype)
    long_sum_is_near(mpq.linear(x, w), x.double() @ w.double().T, k, dtype)


@pytest.mark.parametrize("rows,n,k", [(1 << 20, 64, 72), (1 << 18, 300, 520)])
def test_weight_gradient_of_one_sign_over_many_rows(mpq, rows, n, k):
    g = gen(n)
    dy = (torch.rand(rows, n, generator=g, device="cuda") / 256).to(HF)
    x = torch.rand(rows, k, generator=g, device="cuda").to(HF)
    got = mpq.linear_backward(dy, x, None, dx=False, dbias=False)["dweight"]
    long_sum_is_near(got, dy.double().T @ x.double(), rows, HF)


def test_input_gradient_of_one_sign_over_many_outputs(mpq):
    g = gen(5)
    for rows, n, k in ((300, 1 << 18, 392), (20, 1 << 20, 64)):
        dy = (torch.rand(rows, n, generator=g, device="cuda") / 256).to(HF)
        w = torch.rand(n, k, generator=g, device="cuda").to(HF)
        got = mpq.linear_backward(dy, None, w, dweight=False, dbias=False)["dx"]
        long_sum_is_near(got, dy.double() @ w.double(), n, HF)


# More tiles than workers and more steps than the ring has stages, so that ring
# and accumulators go on from tile to tile in the middle of a turn; small whole
# numbers, so that the results are exact before their one rounding.  Whole waves
# of wide tiles with and without a last one of halves; one step more than a
# chain; steps that no chain or ring divides.
LONG = [(2600, 2500, 1000, BF), (2600, 2500, 4136, HF), (4400, 2300, 472, BF), (2304, 2304, 2056, BF), (2500, 5000, 4200, BF)]


@pytest.mark.parametrize("rows,n,k,dtype", LONG)
@pytest.mark.parametrize("out", [None, F32])
def test_linear_over_many_tiles_is_exact(mpq, rows, n, k, dtype, out):
    g = gen(rows + k)
    x, w, r = whole(g, rows, k), whole(g, n, k), whole(g, rows, n, lim=9)
    y, z = mpq.linear(x.to(dtype), w.to(dtype), residual=r.to(out or dtype), activation="relu", out_dtype=out, preact=True)
    want = x @ w.T
    assert torch.equal(z, want.to(dtype))
    assert torch.equal(y, (torch.relu(want) + r).to(out or dtype))
    assert torch.equal(mpq.linear(x.to(dtype), w.to(dtype), out_dtype=out), want.to(out or dtype))


@pytest.mark.parametrize("rows,n,k,dtype", LONG)
def test_linear_backward_over_many_tiles_is_exact(mpq, rows, n, k, dtype):
    g = gen(rows * 5 + k)
    # dx sums over n and has rows x k results, dweight sums over rows and has n x k
    x, w, dy, z = whole(g, rows, n), whole(g, k, n), whole(g, rows, k), whole(g, rows, k)
    out = mpq.linear_backward(dy.to(dtype), x.to(dtype), w.to(dtype), z.to(dtype), "relu")
    dz = dy * (z > 0)
    assert torch.equal(out["dx"], (dz @ w).to(dtype))
    assert torch.equal(out["dweight"], (dz.T @ x).to(dtype))
    assert torch.equal(out["dbias"], dz.sum(0).to(dtype))
