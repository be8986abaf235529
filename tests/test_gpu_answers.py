"""token_logprobs and topk_distill against plain 64-bit formulas, and the run
of all layer operators around a solve.

Tolerances: a softmax sum over v logits is added by 256 threads or more, in two
chains each: v / 512 sequential fp32 adds and a tree, exponentials good to 2^-22 and scaled
logits rounded by 2^-24 of their size; `rel(v)` is the sum of these."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24
LOWEST = {t: torch.finfo(t).min for t in (BF, HF, F32)}


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).tiny * torch.finfo(t).eps / 2


def rel(v):
    return (v / 512 + 40) * U + 2.0 ** -21


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logp64(l):
    d = l - l.max(-1, keepdim=True).values  # first: next to -3e38 even 64 bits lose a log-sum
    return d - d.exp().sum(-1, keepdim=True).log()


def top64(l, k):
    val, idx = torch.sort(l, dim=-1, descending=True, stable=True)
    return val[..., :k], idx[..., :k]


def close(got, want, tol, what):
    same = (got.double() == want) | (torch.isnan(got) & torch.isnan(want))
    d = torch.where(same, torch.zeros_like(want), (got.double() - want).abs())
    d = torch.where(torch.isnan(d), torch.full_like(d, math.inf), d)
    assert (d <= tol).all(), f"{what}: worst {float((d - tol).max()):.3g} over tolerance at {torch.nonzero(d > tol)[0].tolist()}"


def check_logprobs(mpq, logits, tokens, top):
    v = logits.shape[-1]
    out = mpq.token_logprobs(logits, tokens, top=top)
    l = logits.double()
    lp = logp64(l)
    safe = tokens.clamp(0, v - 1)
    want = torch.where(tokens == -100, 0.0, lp.gather(-1, safe[..., None])[..., 0])
    # scaled logits are rounded by 2^-24 of their distance from the maximum
    close(out["logprob"], want, rel(v) + 4 * U * torch.nan_to_num(want, neginf=0.0).abs(), "logprob")
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    close(out["entropy"], ent, rel(v) * (4 + 2 * math.log(v)), "entropy")
    if top:
        _, idx = top64(l, top)
        assert torch.equal(out["top_id"], idx)
        tl = lp.gather(-1, idx)
        close(out["top_logprob"], tl, rel(v) + 4 * U * torch.nan_to_num(tl, neginf=0.0).abs(), "top_logprob")
    else:
        assert "top_id" not in out
    return out


# rows, v, top: one column; fewer columns than threads; clusters of 2 to 8
# CTAs; one CTA a row; the longest lists
CASES = [(1, 1, 1), (3, 7, 7), (2, 130, 5), (5, 1000, 64), (1, 2000, 100), (4, 4095, 128), (3, 4096, 1), (2, 8192, 20),
         (1, 50001, 5), (20, 33000, 128), (70, 20001, 0), (150, 8200, 16), (400, 1003, 3), (300, 32768, 20), (2, 200003, 33)]


@pytest.mark.parametrize("rows,v,top", CASES)
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_logprobs(mpq, rows, v, top, dtype):
    g = gen(rows + v)
    l = (torch.randn(rows, v, generator=g, device="cuda") * 3).to(dtype)
    l[:, torch.randint(0, v, (1,), generator=g, device="cuda")] += 9
    tok = torch.randint(0, v, (rows,), generator=g, device="cuda")
    tok[rows // 2] = -100
    check_logprobs(mpq, l, tok, top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logprobs_of_slices_and_masks(mpq, dtype):
    g = gen(2)
    wide = (torch.randn(6, 5, 9100, generator=g, device="cuda") * 2).to(dtype)
    l = wide[..., 3:9004]
    tok = torch.randint(0, 9001, (6, 5), generator=g, device="cuda")
    check_logprobs(mpq, l, tok, 40)
    l[0, 0, 100:] = -math.inf                 # few logits left: the list ends in -inf, lowest ids first
    l[0, 1] = -math.inf
    l[0, 1, 77] = 1.0                         # one left
    l[0, 2, ::2] = LOWEST[dtype]              # masks of the lowest value
    l[0, 3] = LOWEST[dtype]                   # all of it: uniform
    l[0, 4, :4000] = LOWEST[dtype]
    l[0, 4, 4000:] = -math.inf                # uniform over the lowest values
    l[1, 0] = 2.0                             # all equal
    l[1, 1, :] = torch.arange(9001, device="cuda").to(dtype)   # ascending
    l[1, 2, :] = -torch.arange(9001, device="cuda").to(dtype)  # descending
    l[1, 3] = 0.0
    l[1, 3, 5::7] = -0.0                      # equal to 0
    l[1, 4, 512 * 8:512 * 8 + 300] = 50.0     # many ties in few columns
    tok[0, 0], tok[0, 1], tok[0, 2], tok[0, 3], tok[0, 4], tok[1, 0] = 50, 77, 1, 9, 5, 9000
    out = check_logprobs(mpq, l, tok, 128)
    assert (out["entropy"] >= 0).all() and out["entropy"][0, 1] <= 8 * U and out["logprob"][0, 1].abs() <= 8 * U


def test_logprobs_with_most_of_the_large_logits_in_few_threads(mpq):
    # columns 8 g + 0..7 with g = 3 mod 256 belong to one thread: its columns
    # alone hold more large logits than the candidate buffer
    v = 512 * 8 * 40
    for rows in (1, 300):
        l = torch.randn(rows, v, generator=gen(rows), device="cuda")
        cols = torch.arange(v, device="cuda")
        for j in range(40):
            l[:, ((cols // 8) % 512) == 3 + j] += 100
        check_logprobs(mpq, l, torch.zeros(rows, dtype=torch.int64, device="cuda"), 64)


def test_logprobs_rows_without_a_distribution(mpq):
    for v in (50, 20000):
        for dtype in (BF, F32):
            l = torch.randn(6, v, generator=gen(v), device="cuda").to(dtype)
            l[0] = -math.inf
            l[1, v // 2] = math.nan
            l[2, 3] = math.inf
            l[3] = math.nan
            tok = torch.tensor([4, 5, 6, 7, v, -1], device="cuda")
            out = mpq.token_logprobs(l, tok, top=9)
            lp, en, tl, ti = (out[k].cpu() for k in ("logprob", "entropy", "top_logprob", "top_id"))
            assert lp[0] == -math.inf and en[0] == 0 and (tl[0] == -math.inf).all() and ti[0].tolist() == list(range(9))
            for r in (1, 2, 3):
                assert math.isnan(lp[r]) and math.isnan(en[r]) and torch.isnan(tl[r]).all()
            assert ti[2, 0] == 3 and (ti[3] == -1).all()
            rest = l[1].float().clone()
            rest[v // 2] = -math.inf
            assert torch.equal(ti[1], top64(rest.double(), 9)[1].cpu())
            assert torch.isnan(lp[4:]).all() and torch.isfinite(en[4:]).all()  # tokens outside the vocabulary
            assert torch.equal(ti[4:], top64(l[4:].double(), 9)[1].cpu())
    assert mpq.token_logprobs(l[:0], tok[:0], top=2)["top_id"].shape == (0, 2)


# ---------------------------------------------------------------- distill --
def distill64(l, tl, ids, w, temp):
    """The definition: padding and -inf entries drop out, equal ids add up."""
    use = ids >= 0
    t = torch.where(use, tl.double(), -math.inf) / temp
    live = t.max(-1, keepdim=True).values > -math.inf
    logq = torch.where(live, t - torch.logsumexp(t, -1, keepdim=True), -math.inf)
    q = logq.exp()
    logp = logp64(l.double() / temp)
    at = logp.gather(-1, ids.clamp_min(0))
    loss = torch.where(q > 0, q * (logq - at), 0.0).sum(-1)
    p = torch.where(live, logp.exp(), 0.0)
    grad = p.scatter_add(-1, ids.clamp_min(0), -q) * (w / temp)[..., None]
    grad = torch.where((w == 0)[..., None], 0.0, grad)
    return loss, grad, q, logq, at, p


def check_distill(mpq, l, tl, ids, w, temp):
    v = l.shape[-1]
    out = mpq.topk_distill(l, tl, ids, weight=w, temperature=temp)
    loss, grad, q, logq, at, p = distill64(l, tl, ids, w.double(), temp)
    fin = lambda x: torch.nan_to_num(x, neginf=0.0, posinf=0.0)
    size = torch.where(q > 0, q * (1 + fin(logq).abs() + fin(at).abs()), 0.0).sum(-1)
    close(out["loss"], loss, 2 * rel(v) * size + 64 * U * size, "loss")
    assert out["dlogits"].dtype == l.dtype and out["dlogits"].shape == l.shape
    tol = half(l.dtype) * grad.abs() + tiny(l.dtype)
    # p = 2^y / S with y rounded by 2^-24 of its size (p large: y small)
    big = p * (rel(v) + 2 * U * fin(p.log()).abs())
    big = big.scatter_add(-1, ids.clamp_min(0), q * 256 * U)
    close(out["dlogits"], grad, tol + big * (w.double().abs() / temp)[..., None], "dlogits")
    assert torch.equal(mpq.topk_distill(l, tl, ids, weight=w, temperature=temp, grad=False)["loss"], out["loss"])
    return out


@pytest.mark.parametrize("rows,v,top", [(1, 1, 1), (3, 9, 4), (2, 300, 128), (5, 4097, 7), (1, 33001, 8), (40, 20000, 20),
                                        (200, 5000, 64), (310, 2003, 32), (2, 150000, 50)])
@pytest.mark.parametrize("dtype,temp", [(BF, 2.0), (HF, 0.7), (F32, 1.0)])
def test_distill(mpq, rows, v, top, dtype, temp):
    g = gen(v + top)
    l = (torch.randn(rows, v, generator=g, device="cuda") * 3).to(dtype)
    teacher = l.float() + torch.randn(rows, v, generator=g, device="cuda")
    k = min(top, v)
    tl, ids = (t.contiguous() for t in teacher.topk(k, dim=-1))
    w = torch.rand(rows, generator=g, device="cuda") + 0.1
    check_distill(mpq, l, tl, ids, w, temp)


@pytest.mark.parametrize("dtype,cut", [(BF, 0), (F32, 0), (BF, 3), (HF, 5), (F32, 1)])
def test_distill_edges(mpq, dtype, cut):
    g = gen(cut + 1)
    v, top = 12001, 6
    l = (torch.randn(4, 3, v + 9, generator=g, device="cuda") * 2).to(dtype)[..., cut:cut + v]
    ids = torch.stack([torch.randperm(v, generator=g, device="cuda")[:top] for _ in range(12)]).view(4, 3, top)
    tl = torch.randn(4, 3, top, generator=g, device="cuda")
    w = torch.rand(4, 3, generator=g, device="cuda") + 0.5
    ids[0, 0, 2:] = -1                        # padding
    ids[0, 1] = -1                            # nothing left
    tl[0, 2] = -math.inf                      # nothing left either
    tl[1, 0, 1:] = -math.inf                  # one entry left
    ids[1, 1, 3] = ids[1, 1, 0]               # an id twice
    ids[1, 2] = v - 1                         # one id in all entries, the last column
    w[2, 0] = 0.0
    l[2, 1, ::3] = -math.inf
    ids[2, 1, 0] = 1
    ids[2, 1, 1:] = torch.tensor([2, 4, 5, 7, 8], device="cuda")
    l[2, 2] = LOWEST[dtype]                   # uniform
    l[3, 0, :-1] = -math.inf                  # one logit left
    ids[3, 0, 1:] = -1
    ids[3, 0, 0] = v - 1
    out = check_distill(mpq, l, tl, ids, w, 1.0)
    for r in ((0, 1), (0, 2), (2, 0)):
        assert not out["dlogits"][r].any()
    assert out["loss"][0, 1] == 0 and out["loss"][0, 2] == 0
    # one logit and one entry: log q = 0 and log p = ln2 y - ln S with y = l k - M the rounding of M, at most
    # |M| 2^-24, S = 2^y: what is left are the roundings of 2^y and ln S (2 ulp and 1 ulp of numbers near 1 and y)
    assert out["loss"][3, 0].abs() <= 8 * U
    # a teacher's logit where the student has none: infinite loss, finite gradient
    ids[2, 1, 0] = 3
    bad = mpq.topk_distill(l, tl, ids, weight=w)
    assert bad["loss"][2, 1] == math.inf and torch.isfinite(bad["dlogits"][2, 1]).all()
    # garbage in rows of weight 0 stays out of the gradient; an id outside v makes NaN
    l[2, 0] = math.nan
    ids[3, 1, 2] = v
    bad = mpq.topk_distill(l, tl, ids, weight=w)
    assert not bad["dlogits"][2, 0].any() and torch.isnan(bad["loss"][3, 1]) and torch.isnan(bad["dlogits"][3, 1]).all()
    assert torch.equal(bad["dlogits"][3, 2], out["dlogits"][3, 2])
    assert mpq.topk_distill(l[:0], tl[:0], ids[:0])["loss"].shape == (0, 3)


def test_distill_gradient_against_differences(mpq):
    g = gen(4)
    v, top, temp = 700, 9, 1.5
    l = torch.randn(5, v, generator=g, device="cuda") * 2
    tl, ids = (t.contiguous() for t in (l + torch.randn(5, v, generator=g, device="cuda")).topk(top, dim=-1))
    w = torch.rand(5, generator=g, device="cuda")
    d = torch.randn(5, v, generator=g, device="cuda").double()
    got = mpq.topk_distill(l, tl, ids, weight=w, temperature=temp)
    h = 2.0 ** -9
    f = lambda t: (distill64(t, tl, ids, w.double(), temp)[0] * w.double()).sum()
    slope = float((f(l.double() + h * d) - f(l.double() - h * d)) / (2 * h))
    have = float((got["dlogits"].double() * d).sum())
    # third derivative of a log-sum: at most (2 max |d| / temp)^3 a row
    third = float(w.double().sum()) * (2 * float(d.abs().max()) / temp) ** 3
    tol = h * h / 6 * third + 2 * rel(v) * float((w.double()[:, None] * d.abs()).amax(1).sum()) / temp * 2
    assert abs(slope - have) <= tol, (slope, have, tol)


def test_answers_refusals(mpq):
    c = lambda *s, t=F32: torch.ones(*s, dtype=t, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int64, device="cuda")
    bad = [lambda: mpq.token_logprobs(c(2, 8, t=torch.float64)), lambda: mpq.token_logprobs(c(2, 8), i(3)),
           lambda: mpq.token_logprobs(c(2, 8), i(2).int()), lambda: mpq.token_logprobs(c(2, 8), i(2).cpu()),
           lambda: mpq.token_logprobs(c(2, 8), top=9), lambda: mpq.token_logprobs(c(2, 800), top=129),
           lambda: mpq.token_logprobs(c(2, 8), top=-1), lambda: mpq.token_logprobs(c(8, 2).T),
           lambda: mpq.token_logprobs(c(2, 0)), lambda: mpq.topk_distill(c(2, 8), c(2, 3), i(2, 4)),
           lambda: mpq.topk_distill(c(2, 8), c(2, 3, t=BF), i(2, 3)), lambda: mpq.topk_distill(c(2, 8), c(2, 3), i(2, 3).int()),
           lambda: mpq.topk_distill(c(2, 8), c(2, 0), i(2, 0)), lambda: mpq.topk_distill(c(2, 800), c(2, 129), i(2, 129)),
           lambda: mpq.topk_distill(c(2, 8), c(2, 3), i(2, 3), weight=c(3)),
           lambda: mpq.topk_distill(c(2, 8), c(2, 3), i(2, 3), temperature=0.0),
           lambda: mpq.topk_distill(c(2, 8), c(2, 3), i(2, 6)[:, ::2])]
    before = mpq.kernel_launch_count()
    for n, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {n} was accepted")
    assert mpq.kernel_launch_count() == before


def test_answers_repeatable_on_streams_and_in_graphs(mpq):
    g = gen(12)
    l = torch.randn(9, 40000, generator=g, device="cuda").to(BF)
    tok = torch.randint(0, 40000, (9,), generator=g, device="cuda")

    def step():
        a = mpq.token_logprobs(l, tok, top=20)
        b = mpq.topk_distill(l, a["top_logprob"], a["top_id"].flip(0), temperature=1.3)
        return [*a.values(), *b.values()]

    first = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    again = step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step()
    l.copy_(torch.randn(9, 40000, generator=g, device="cuda").to(BF))
    gr.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, again):
        assert torch.equal(a, b) and torch.equal(a, c)
    for a, b in zip(step(), out):
        assert torch.equal(a, b)


def test_logits_past_32_bit_offsets(mpq):
    rows, v = 33000, 131073  # 4.3e9 logits
    l = torch.zeros(rows, v, dtype=BF, device="cuda")
    tail = torch.randn(2, v, generator=gen(8), device="cuda").to(BF)
    l[-2:] = tail
    tok = torch.full((rows,), 3, dtype=torch.int64, device="cuda")
    a, b = mpq.token_logprobs(l, tok, top=3), mpq.token_logprobs(tail, tok[:2], top=3)
    assert torch.equal(a["top_id"][-2:], b["top_id"]) and a["top_id"][0].tolist() == [0, 1, 2]
    # (one CTA a row there, eight here: other orders of the sums)
    close(a["logprob"][-2:], b["logprob"].double(), 2 * rel(v), "logprob")
    close(a["logprob"][:1], torch.full((1,), -math.log(v), dtype=torch.float64, device="cuda"), rel(v) + 50 * U, "uniform")
    d = mpq.topk_distill(l, a["top_logprob"], a["top_id"])
    e = mpq.topk_distill(tail, b["top_logprob"], b["top_id"])
    close(d["dlogits"][-2:], e["dlogits"].double(), 2 * half(BF) * e["dlogits"].double().abs() + 8 * U, "dlogits")


# ----------------------------------------------- a run of all, round a solve --
def test_a_solved_layer_calibrates_answers_and_trains(mpq):
    """norm -> solved projection -> the next layer's Gram; the answers of the
    solved model against the full one; gradients back to the norm."""
    g = gen(21)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    tokens, n, hidden, vocab = 600, 128, 192, 1000
    x = (rnd(tokens, n) * (1 + rnd(n).abs())).to(BF)
    gamma, beta = 1 + 0.1 * rnd(n), 0.1 * rnd(n)
    w1, head = rnd(hidden, n) / n ** 0.5, (rnd(vocab, hidden) / hidden ** 0.5 * 2).to(BF)
    h, mean, rstd = mpq.layer_norm(x, gamma, beta, stats=True)
    gram = mpq.Gram(n).accumulate(h.float())
    plan = mpq.Plan.from_gram(gram, 1, 16)
    w_hat = plan.solve(w1.contiguous(), 4, 1)["w_hat"].to(BF)

    nxt = mpq.linear(h, w_hat, activation="silu", out_dtype=F32)  # the next layer's calibration rows
    got = mpq.Gram(hidden).accumulate(nxt).matrix()
    ref = act = torch.nn.functional.silu(h.double() @ w_hat.double().T)
    ref = ref.T @ ref
    assert (got - ref).norm() <= 1e-5 * ref.norm()

    def model(w):
        z_in = mpq.linear(h, w, activation="silu", preact=True)
        return z_in, mpq.linear(z_in[0], head, out_dtype=F32)

    _, full = model(w1.to(BF))
    (a, z), quant = model(w_hat)
    target = full.argmax(-1)
    teacher = mpq.token_logprobs(full, target, top=16)
    student = mpq.token_logprobs(quant, target, top=1)
    assert torch.equal(teacher["top_id"][:, 0], target)
    assert float(student["logprob"].mean()) < float(teacher["logprob"].mean())  # the full model is surer of its own
    weight = torch.full((tokens,), 1.0 / tokens, device="cuda")
    d = mpq.topk_distill(quant, teacher["top_logprob"], teacher["top_id"], weight=weight)
    assert (d["loss"] >= -1e-5).all()
    da = mpq.linear_backward((d["dlogits"] * 1024).to(BF), None, head, dweight=False, dbias=False)["dx"]
    dh = mpq.linear_backward(da, None, w_hat, z, "silu", dweight=False)
    dn = mpq.layer_norm_backward(dh["dx"], x, mean, rstd, gamma)
    # the same chain by autograd in 64 bits from the same weights
    gl, bl = gamma.double().requires_grad_(), beta.double().requires_grad_()
    x64 = x.double()
    m = x64.mean(-1, keepdim=True)
    hn = (x64 - m) / torch.sqrt((x64 - m).square().mean(-1, keepdim=True) + 1e-5) * gl + bl
    logits = torch.nn.functional.silu(hn @ w_hat.double().T) @ head.double().T
    loss = distill64(logits, teacher["top_logprob"], teacher["top_id"], weight.double(), 1.0)[0]
    (loss * weight.double()).sum().backward()
    # five tensors on the way are rounded to bf16 (2^-8 of a value at most each):
    # h, the activations and z, and the two gradients
    for have, want in ((dn["dweight"], gl.grad), (dn["dbias"], bl.grad)):
        assert (have.double() / 1024 - want).norm() <= 5 * 2.0 ** -8 * 2 * want.norm()
    mpq.ops_status()
