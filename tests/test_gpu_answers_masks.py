"""token_logprobs and topk_distill on rows with finite masks of any size, against
plain 64-bit formulas with the tolerances of test_gpu_answers."""
import math

import pytest
import torch

from tests.test_gpu_answers import BF, F32, HF, LOWEST, U, check_logprobs, close, distill64, gen, half, rel, tiny

pytestmark = pytest.mark.gpu

MASKS = [(F32, -1e9), (F32, -1e10), (F32, -3e12), (F32, -1e30), (F32, -1e35), (F32, -3e38), (F32, LOWEST[F32]),
         (BF, -1e9), (BF, -1e10), (BF, -1e30), (BF, -1e35), (BF, LOWEST[BF]), (HF, -6e4), (HF, LOWEST[HF])]


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def masked(dtype, mask, many):
    """Rows with the mask in a prefix, a tail, a stretch, whole threads' columns, all but one column, everywhere, and
    in part next to -inf.  Few rows are shared by clusters of CTAs (1/8 of the columns each), many have one each."""
    v = 40000
    l = torch.randn(8, v, generator=gen(int(-mask) % 1000 + many), device="cuda") * 2
    cols = torch.arange(v, device="cuda")
    l[0, :8192] = mask                        # the first vectors of every thread
    l[1, v - 7000:] = mask                    # a padded vocabulary
    l[2, v // 8 * 3:v // 8 * 4] = mask        # one CTA's stretch
    l[3, (cols // 8) % 256 < 100] = mask      # all that some threads meet
    l[4] = mask
    l[4, 777] = 1.0                           # one left
    l[5] = mask                               # uniform
    l[6, :20000], l[6, 20000:] = mask, -math.inf
    l[7, ::2] = mask
    l = l.to(dtype)
    if many:
        l = l.repeat(40, 1)
    tok = torch.tensor([9000, 5, v // 2 - 9000, 850, 777, 11, 3, 1], device="cuda").repeat(40 if many else 1)
    return l, tok


def check_distill(mpq, l, tl, ids, w, temp):
    """As in test_gpu_answers, and with the powers that fp32's exponential takes as 0: 2^y below 2^-126, so that
    w / T (2^y / S) with S >= 1 is off by up to 2^-126 w / T (5e-39 at T = 2, 1e-35 at 0.001)."""
    out = mpq.topk_distill(l, tl, ids, weight=w, temperature=temp)
    loss, grad, q, logq, at, p = distill64(l, tl, ids, w.double(), temp)
    v = l.shape[-1]
    fin = lambda x: torch.nan_to_num(x, neginf=0.0, posinf=0.0)
    size = torch.where(q > 0, q * (1 + fin(logq).abs() + fin(at).abs()), 0.0).sum(-1)
    close(out["loss"], loss, 2 * rel(v) * size + 64 * U * size, "loss")
    big = p * (rel(v) + 2 * U * fin(p.log()).abs()) + 2.0 ** -126
    big = big.scatter_add(-1, ids.clamp_min(0), q * 256 * U)
    close(out["dlogits"], grad, half(l.dtype) * grad.abs() + tiny(l.dtype) + big * (w.double().abs() / temp)[..., None], "dlogits")
    assert torch.equal(mpq.topk_distill(l, tl, ids, weight=w, temperature=temp, grad=False)["loss"], out["loss"])
    return out


@pytest.mark.parametrize("many", [0, 1])
@pytest.mark.parametrize("dtype,mask", MASKS)
def test_logprobs_next_to_finite_masks(mpq, dtype, mask, many):
    l, tok = masked(dtype, mask, many)
    check_logprobs(mpq, l, tok, 20)
    out = check_logprobs(mpq, l, tok, 0)
    assert torch.isfinite(out["logprob"]).all() and torch.isfinite(out["entropy"]).all()
    masked_token = mpq.token_logprobs(l[:1], torch.zeros(1, dtype=torch.int64, device="cuda"))["logprob"]
    assert masked_token[0] <= l[0, 0].float() * 0.999  # the mask itself is the token


@pytest.mark.parametrize("many", [0, 1])
@pytest.mark.parametrize("temp", [1e-3, 0.7, 1.0, 2.0, 1e3])
@pytest.mark.parametrize("dtype,mask", MASKS)
def test_distill_next_to_finite_masks(mpq, dtype, mask, temp, many):
    l, tok = masked(dtype, mask, many)
    g = gen(7)
    # near the student's own temperature, so that several of the teacher's entries count at any
    tl = torch.randn(l.shape[0], 5, generator=g, device="cuda") * min(temp, 1.0)
    ids = torch.stack([tok, (tok + 1) % l.shape[1], (tok + 9) % l.shape[1], (tok + 30000) % l.shape[1], tok], -1)
    ids[..., 4] = -1
    for r in range(l.shape[0]):  # entries on logits of the row that are left (masked ones: below)
        if r % 8 == 4:
            ids[r, 1:] = -1
        elif r % 8 == 6:
            ids[r, 1:] = torch.tensor([1, 2, 7, -1])
    fine = l.gather(-1, ids.clamp_min(0)).float() > (mask * 0.99 if mask > -1e38 else -1e38)
    whole = torch.tensor([False] * 4 + [True] * 3 + [False], device="cuda").repeat(l.shape[0] // 8)
    ids = torch.where(fine | whole[:, None], ids, -1)
    w = torch.rand(l.shape[0], generator=g, device="cuda") + 0.5
    out = check_distill(mpq, l, tl, ids, w, temp)
    assert torch.isfinite(out["loss"]).all() and torch.isfinite(out["dlogits"].float()).all()


@pytest.mark.parametrize("temp", [0.7, 1.0])
def test_distill_of_a_masked_entry(mpq, temp):
    """The teacher has an entry where the student has a mask: a loss of the mask's size."""
    l, tok = masked(F32, -1e10, 0)
    ids = torch.stack([tok, torch.full_like(tok, 0)], -1)[:1]
    tl = torch.zeros(1, 2, device="cuda")
    check_distill(mpq, l[:1], tl, ids, torch.ones(1, device="cuda"), temp)


@pytest.mark.parametrize("many", [0, 1])
@pytest.mark.parametrize("size", [1e6, 1e8, 1e10, 1e30, 3e38])
def test_rows_of_large_logits(mpq, size, many):
    """Logits of any finite size, up to both ends of fp32 in one row."""
    v = 9001
    l = torch.randn(6, v, generator=gen(int(math.log10(size))), device="cuda")
    l[0] = (size + l[0].double() * size * 1e-6).float().clamp(max=3.4e38)  # a few steps of fp32 apart
    l[1] = (-size + l[1].double() * size * 1e-6).float().clamp(min=-3.4e38)
    l[2] = (l[2].double() * size).float().clamp(-3.4e38, 3.4e38)
    l[3] = size                                             # equal
    l[4, ::2], l[4, 1::2] = size, -size
    l[5, 100] = size
    tok = l.argmax(-1)
    if many:
        l, tok = l.repeat(60, 1), tok.repeat(60)
    out = check_logprobs(mpq, l, tok, 5)
    assert torch.isfinite(out["logprob"]).all() and torch.isfinite(out["entropy"]).all()
    for temp in (1e-3, 1.0, 1e3):
        ids = torch.stack([tok, (tok + 1) % v], -1)
        fine = l.gather(-1, ids) == l.max(-1, keepdim=True).values
        ids = torch.where(fine, ids, -1)
        check_distill(mpq, l, torch.zeros(*ids.shape, device="cuda"), ids, torch.ones(len(l), device="cuda"), temp)
    lost = mpq.topk_distill(l[4:5], torch.zeros(1, 1, device="cuda"), torch.ones(1, 1, dtype=torch.int64, device="cuda"),
                            temperature=1e3)["loss"]
    want = 2e-3 * float(torch.tensor(size)) + math.log((v + 1) // 2)  # log p of -size next to size, over T = 1000
    assert abs(float(lost) - want) <= 8 * U * want + 64 * U * math.log(v)


@pytest.mark.parametrize("rows", [1, 2, 300])
@pytest.mark.parametrize("v,top", [(9, 9), (700, 20), (20000, 9), (20000, 128), (90000, 100)])
@pytest.mark.parametrize("dtype", [BF, HF, F32])
def test_top_ids_of_masked_rows_with_nan(mpq, rows, v, top, dtype):
    """Of a row with a NaN the logits that are none are ranked, -inf among them (equal ones: lowest id first)."""
    g = gen(v + rows)
    l = torch.full((rows, v), -math.inf, device="cuda")
    for r in range(rows):
        kind = r % 4 if rows > 1 else 0
        l[r, 5] = math.nan                                   # a NaN among the first columns
        if kind == 1:                                        # and some all over, some finite logits
            l[r, torch.randint(0, v, (v // 50 + 1,), generator=g, device="cuda")] = math.nan
            l[r, torch.randint(0, v, (3,), generator=g, device="cuda")] = 1.5
        elif kind == 2:                                      # whole threads' columns
            l[r, : v // 3] = math.nan
        elif kind == 3:                                      # fewer logits than are asked for
            l[r] = math.nan
            l[r, v - 2:] = -math.inf
    l = l.to(dtype)
    out = mpq.token_logprobs(l, top=top)
    rank = torch.where(torch.isnan(l), torch.tensor(-1.0, device="cuda"), torch.where(l > -math.inf, 1.0, 0.0))
    val, idx = torch.sort(rank, dim=-1, descending=True, stable=True)  # (finite ones are all 1.5)
    want = torch.where(val[:, :top] < 0, -1, idx[:, :top])
    assert torch.equal(out["top_id"], want)
    # (among nine columns the finite logits may have taken the place of every NaN)
    has = torch.isnan(l).any(-1)
    assert torch.equal(torch.isnan(out["entropy"]), has) and torch.equal(torch.isnan(out["top_logprob"]).all(-1), has)


# Vectors of 8 columns belong to threads in turn (256 of them here); 40 threads hold large logits only, more than the
# candidate buffer's 4096.  They fill 20 of the 128 sets whose maxima bound the list, so that for more than 20
# alternatives all of them are candidates.  One CTA a row (300 rows), clusters of 8 (one row); many ties in 16 bits.
@pytest.mark.parametrize("rows,v,dtype", [(300, 80000, BF), (300, 80000, HF), (300, 40960, F32), (1, 8 * 8 * 256 * 20, BF),
                                          (1, 8 * 8 * 256 * 20, F32), (2, 8 * 8 * 256 * 15 + 5, HF)])
@pytest.mark.parametrize("top", [1, 64, 128])
def test_top_with_more_candidates_than_their_buffer(mpq, rows, v, dtype, top):
    assert v // (8 if rows < 9 else 1) // 8 // 256 * 8 * 40 > 4096
    l = torch.randn(rows, v, generator=gen(rows + top), device="cuda")
    cta = v // 8 if rows < 9 else v  # columns of a CTA
    cols = torch.arange(v, device="cuda") % cta
    l[:, ((cols // 8) % 256 >= 3) & ((cols // 8) % 256 < 43)] += 100
    check_logprobs(mpq, l.to(dtype), torch.zeros(rows, dtype=torch.int64, device="cuda"), top)
