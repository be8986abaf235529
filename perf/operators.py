"""Timed cases of the operators that run and judge a layer with its solved weights.

A solve gives w_hat; what follows it runs a model's layers with those weights and compares the model's answers
with the unquantised one's.  Four operators do that:

  linear          y = act(x W^T + b) + residual, and its backward pass (dx, dW, db)
  layer_norm      the norm whose outputs are a layer's calibration rows, and its backward pass
  token_logprobs  log probability of given tokens, entropy of each row, and the top alternatives
  topk_distill    KL divergence from a teacher's top logits, with the gradient of the student's logits

`run` computes a case in plain torch operations in 32 bits, or, where `own` is set, with the package's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
IGNORED = -100  # a token that is not scored (padding)
EPS = 1e-5


def listed():
    return [
        # one token of generation through a square projection
        {"name": "linear decode", "op": "linear", "rows": 1, "k": 4096, "n": 4096, "dtype": "bf16", "out": "bf16",
         "bias": True, "act": "silu", "residual": False},
        # a short ragged batch, sizes that no tile divides, fp32 rows for a Gram
        {"name": "linear ragged", "op": "linear", "rows": 777, "k": 1999, "n": 2051, "dtype": "fp16", "out": "fp32",
         "bias": True, "act": "gelu", "residual": True},
        # calibration: two sequences of 2048 tokens through the 14336-wide down projection, into the residual stream
        {"name": "linear calibration", "op": "linear", "rows": 4096, "k": 14336, "n": 4096, "dtype": "bf16",
         "out": "bf16", "bias": False, "act": "none", "residual": True},
        # recovery training of the wide projection: all three gradients
        {"name": "linear backward", "op": "linear_backward", "rows": 4096, "k": 4096, "n": 14336, "dtype": "bf16",
         "act": "gelu", "frozen": False},
        # one token's norm
        {"name": "norm decode", "op": "layer_norm", "rows": 1, "c": 4096, "dtype": "bf16", "param": "bf16"},
        # the norm of eight calibration sequences
        {"name": "norm calibration", "op": "layer_norm", "rows": 16384, "c": 4096, "dtype": "bf16", "param": "fp32"},
        # its training step
        {"name": "norm backward", "op": "layer_norm_backward", "rows": 16384, "c": 4096, "dtype": "bf16",
         "param": "fp32"},
        # odd sizes in full precision
        {"name": "norm backward odd", "op": "layer_norm_backward", "rows": 1003, "c": 1001, "dtype": "fp32",
         "param": "fp32"},
        # the answers of a generation step for eight requests, with five alternatives
        {"name": "logprobs decode", "op": "token_logprobs", "rows": 8, "v": 50001, "top": 5, "dtype": "fp32",
         "slack": 0},
        # perplexity and the teacher's alternatives over half a sequence of a large vocabulary
        {"name": "logprobs sequence", "op": "token_logprobs", "rows": 1024, "v": 131072, "top": 20, "dtype": "bf16",
         "slack": 0},
        # a small distillation batch, rows cut from a padded vocabulary
        {"name": "distill small", "op": "topk_distill", "rows": 63, "v": 32001, "top": 8, "dtype": "fp32",
         "slack": 63, "temperature": 1.0},
        # a training step's rows over a large vocabulary
        {"name": "distill sequence", "op": "topk_distill", "rows": 1024, "v": 131072, "top": 32, "dtype": "bf16",
         "slack": 0, "temperature": 2.0},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_backward", "layer_norm", "layer_norm_backward", "token_logprobs",
                     "topk_distill"])
    half = rng.choice(["bf16", "fp16"])
    if op in ("linear", "linear_backward"):
        k, n = _spread(rng, 64, 14336), _spread(rng, 64, 14336)
        if rng.random() < 0.7:  # widths of models are multiples of 8 more often than not
            k, n = max(64, k // 64 * 64), max(64, n // 8 * 8)
        rows = _spread(rng, 1, max(1, min(4096, 4096 * 4096 * 14336 // (k * n))))
        case = {"op": op, "rows": rows, "k": k, "n": n, "dtype": half, "act": rng.choice(ACTIVATIONS)}
        if op == "linear":
            case.update(out=rng.choice([half, "fp32"]), bias=rng.random() < 0.5, residual=rng.random() < 0.5)
        else:
            case.update(frozen=rng.random() < 0.5)
        return case
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if op in ("layer_norm", "layer_norm_backward"):
        c = _spread(rng, 16, 16384)
        rows = _spread(rng, 1, min(65536, 16384 * 4096 // c // (2 if dtype == "fp32" else 1)))
        return {"op": op, "rows": rows, "c": c, "dtype": dtype, "param": rng.choice([dtype, "fp32"])}
    v = _spread(rng, 1000, 200000)
    rows = _spread(rng, 1, min(4096, 1024 * 131072 // v // (2 if dtype == "fp32" else 1)))
    case = {"op": op, "rows": rows, "v": v, "top": rng.randint(1, 64), "dtype": dtype,
            "slack": rng.choice([0, 0, 1, 64])}
    if op == "token_logprobs" and rng.random() < 0.3:
        case["top"] = 0
    if op == "topk_distill":
        case["temperature"] = rng.choice([1.0, 1.0, 2.0, 0.7])
    return case


def work(case):
    """Each input once, each output once; products as 2 per multiply-add, exponentials and the like as one each."""
    op, r = case["op"], case["rows"]
    size = DTYPES[case["dtype"]].itemsize
    if op == "linear":
        k, n, o = case["k"], case["n"], DTYPES[case["out"]].itemsize
        moved = size * (r * k + n * k) + o * r * n * (2 if case["residual"] else 1) + (size * n if case["bias"] else 0)
        return {"bytes": moved, "flops": 2 * r * k * n}
    if op == "linear_backward":
        k, n = case["k"], case["n"]
        z = 0 if case["act"] == "none" else r * n
        moved = size * (r * n + z + n * k + r * k + n)
        if not case["frozen"]:
            moved += size * (r * k + n * k)
        return {"bytes": moved, "flops": (2 if case["frozen"] else 4) * r * k * n}
    if op == "layer_norm":
        c, p = case["c"], DTYPES[case["param"]].itemsize
        return {"bytes": 2 * r * c * size + 2 * c * p + 8 * r, "flops": 8 * r * c}
    if op == "layer_norm_backward":
        c, p = case["c"], DTYPES[case["param"]].itemsize
        return {"bytes": 3 * r * c * size + 3 * c * p + 8 * r, "flops": 14 * r * c}
    v, top = case["v"], case["top"]
    if op == "token_logprobs":
        return {"bytes": r * (v * size + 8 + 8 + top * 12), "flops": 5 * r * v}
    return {"bytes": r * (2 * v * size + top * 12 + 8), "flops": 6 * r * v}


def prepare(case, seed):
    """Inputs on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, r, dt = case["op"], case["rows"], DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, device="cuda", generator=g) * scale

    s = {"case": case}
    if op in ("linear", "linear_backward"):
        k, n = case["k"], case["n"]
        # activations with a few outlier channels, weights of a layer with rows of unequal size
        outlier = 1.0 + 9.0 * (torch.rand(k, device="cuda", generator=g) < 0.01)
        s["x"] = (normal(r, k) * outlier).to(dt)
        s["weight"] = (normal(n, k, scale=k ** -0.5) * torch.exp(0.5 * normal(n, 1))).to(dt)
        if op == "linear":
            out = DTYPES[case["out"]]
            s["bias"] = normal(n, scale=0.5).to(dt) if case["bias"] else None
            s["residual"] = normal(r, n, scale=2.0).to(out) if case["residual"] else None
            s["out"] = out
        else:
            s["dy"] = normal(r, n).to(dt)
            s["preact"] = None if case["act"] == "none" else (1.5 * normal(r, n)).to(dt)
    elif op in ("layer_norm", "layer_norm_backward"):
        c, pt = case["c"], DTYPES[case["param"]]
        x = normal(r, c) * (0.5 + 2.0 * torch.rand(r, 1, device="cuda", generator=g)) + 0.7 * normal(r, 1)
        s["x"] = x.to(dt)
        s["weight"] = (1.0 + 0.2 * normal(c)).to(pt)
        s["bias"] = (0.1 * normal(c)).to(pt)
        if op == "layer_norm_backward":
            s["dy"] = normal(r, c).to(dt)
            x64 = s["x"].double()
            s["mean"] = x64.mean(1).float()  # what the forward pass keeps
            s["rstd"] = (x64.var(1, unbiased=False) + EPS).rsqrt().float()
            del x64
    else:
        v, top = case["v"], case["top"]
        full = normal(r, v + case["slack"], scale=2.5)
        first = torch.randint(0, v, (r, 1), device="cuda", generator=g)
        peaks = (first + torch.arange(4, device="cuda") * (v // 5 + 1)) % v  # a model's few likely tokens
        full.scatter_add_(1, peaks, 8.0 + 2.0 * normal(r, 4))
        logits = full.to(dt)[:, :v]
        s["logits"] = logits
        if op == "token_logprobs":
            tokens = torch.where(torch.rand(r, device="cuda", generator=g) < 0.5, peaks[:, 0],
                                 torch.randint(0, v, (r,), device="cuda", generator=g))
            if r > 4:
                tokens[torch.rand(r, device="cuda", generator=g) < 0.05] = IGNORED
            s["tokens"] = tokens
        else:
            teacher = full[:, :v] + normal(r, v, scale=0.5)
            s["top_logits"], s["top_ids"] = (t.contiguous() for t in teacher.topk(top, dim=1))
            s["weight"] = torch.rand(r, device="cuda", generator=g) / r
            if r > 4:
                s["weight"][torch.rand(r, device="cuda", generator=g) < 0.05] = 0.0
    return s


# ------------------------------------------------------------- plain form --
def _act(z, name):
    if name == "relu":
        return z.clamp_min(0.0)
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, name):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * z * z)
    q = 1.0 / (1.0 + torch.exp(-z))  # silu
    return q * (1.0 + z * (1.0 - q))


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "linear":
        z = s["x"].float() @ s["weight"].float().T
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(s["out"])}
    if op == "linear_backward":
        dt = s["dy"].dtype
        dz = s["dy"].float()
        if s["preact"] is not None:
            dz = dz * _act_grad(s["preact"].float(), case["act"])
        out = {"dx": (dz @ s["weight"].float()).to(dt), "dbias": dz.sum(0).to(dt)}
        if not case["frozen"]:
            out["dweight"] = (dz.T @ s["x"].float()).to(dt)
        return out
    if op == "layer_norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "layer_norm_backward":
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["weight"].float()
        dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        pt = s["weight"].dtype
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0).to(pt), "dbias": dy.sum(0).to(pt)}
    if op == "token_logprobs":
        l = s["logits"].float()
        m = l.max(1, keepdim=True).values
        d = l - m
        e = torch.exp(d)
        total = e.sum(1, keepdim=True)
        lse = torch.log(total)
        entropy = lse[:, 0] - (e * d).sum(1) / total[:, 0]
        tok = s["tokens"]
        logp = d.gather(1, tok.clamp_min(0)[:, None])[:, 0] - lse[:, 0]
        out = {"logprob": torch.where(tok == IGNORED, torch.zeros_like(logp), logp), "entropy": entropy}
        if case["top"]:
            val, idx = torch.sort(l, dim=1, descending=True, stable=True)
            out["top_logprob"] = val[:, :case["top"]] - m - lse
            out["top_id"] = idx[:, :case["top"]].contiguous()
        return out
    x = s["logits"].float() / case["temperature"]
    t = s["top_logits"].float() / case["temperature"]
    t = t - t.max(1, keepdim=True).values
    logq = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    q = torch.exp(logq)
    d = x - x.max(1, keepdim=True).values
    logp = d - torch.log(torch.exp(d).sum(1, keepdim=True))
    loss = (q * (logq - logp.gather(1, s["top_ids"]))).sum(1)
    grad = torch.exp(logp).scatter_add_(1, s["top_ids"], -q) * (s["weight"] / case["temperature"])[:, None]
    return {"loss": loss, "dlogits": grad.to(s["logits"].dtype)}


# ------------------------------------------------------ the package's form --
def _kernels(s):
    import post_weight_quantization_row_b200 as mpq
    case = s["case"]
    op = case["op"]
    if op == "linear":
        return {"y": mpq.linear(s["x"], s["weight"], bias=s["bias"], residual=s["residual"], activation=case["act"],
                                out_dtype=s["out"])}
    if op == "linear_backward":
        return mpq.linear_backward(s["dy"], None if case["frozen"] else s["x"], s["weight"], preact=s["preact"],
                                   activation=case["act"], dweight=not case["frozen"])
    if op == "layer_norm":
        y, mean, rstd = mpq.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "layer_norm_backward":
        return mpq.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if op == "token_logprobs":
        return mpq.token_logprobs(s["logits"], s["tokens"], top=case["top"], ignore_index=IGNORED)
    return mpq.topk_distill(s["logits"], s["top_logits"], s["top_ids"], weight=s["weight"],
                            temperature=case["temperature"])


def run(state):
    if own:
        return _kernels(state)
    return _plain(state)


# --------------------------------------------- the definitions in 64 bits --
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    act = case.get("act")
    if op == "linear":
        z = torch.einsum("rk,nk->rn", f["x"], f["weight"]) + (f["bias"] if "bias" in f else 0.0)
        if act == "relu":
            z = torch.where(z > 0, z, 0.0)
        elif act == "gelu":  # z times the normal distribution function
            z = z * 0.5 * torch.special.erfc(-z / 2.0 ** 0.5)
        elif act == "gelu_tanh":  # (1 + tanh u) / 2 = 1 / (1 + e^-2u)
            z = z / (1.0 + torch.exp(-2.0 * (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
        elif act == "silu":
            z = z / (1.0 + torch.exp(-z))
        return {"y": z + (f["residual"] if "residual" in f else 0.0)}
    if op == "linear_backward":
        dz = f["dy"]
        if act != "none":
            z = f["preact"]
            if act == "relu":
                slope = torch.where(z > 0, 1.0, 0.0).double()
            elif act == "gelu":
                slope = 0.5 * torch.special.erfc(-z / 2.0 ** 0.5) + z * torch.exp(-z * z / 2.0) / (2.0 * math.pi) ** 0.5
            else:
                if act == "silu":
                    u, du = z, torch.ones_like(z)
                else:
                    a = 2.0 * (2.0 / math.pi) ** 0.5
                    u, du = a * (z + 0.044715 * z ** 3), a * (1.0 + 0.134145 * z ** 2)
                sig = 1.0 / (1.0 + torch.exp(-u))
                slope = sig + z * sig * (1.0 - sig) * du
            dz = dz * slope
        out = {"dx": torch.einsum("rn,nk->rk", dz, f["weight"]), "dbias": torch.einsum("rn->n", dz)}
        if not case["frozen"]:
            out["dweight"] = torch.einsum("rn,rk->nk", dz, f["x"])
        return out
    if op == "layer_norm":
        x = f["x"]
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        return {"y": (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * f["weight"] + f["bias"], "mean": mean,
                "rstd": rstd}
    if op == "layer_norm_backward":
        c = case["c"]
        xh = (f["x"] - f["mean"][:, None]) * f["rstd"][:, None]
        dxh = f["dy"] * f["weight"]
        along = (dxh * xh).sum(1, keepdim=True)
        return {"dx": f["rstd"][:, None] / c * (c * dxh - dxh.sum(1, keepdim=True) - xh * along),
                "dweight": torch.einsum("rc,rc->c", f["dy"], xh), "dbias": f["dy"].sum(0)}
    if op == "token_logprobs":
        logp = f["logits"] - torch.logsumexp(f["logits"], 1, keepdim=True)
        tok = s["tokens"]
        at = torch.arange(case["rows"], device=tok.device)
        own_p = logp[at, tok.clamp_min(0)]
        out = {"logprob": torch.where(tok == IGNORED, 0.0, own_p), "entropy": -(torch.exp(logp) * logp).sum(1)}
        if case["top"]:
            val, idx = torch.sort(logp, dim=1, descending=True, stable=True)
            out["top_logprob"], out["top_id"] = val[:, :case["top"]].contiguous(), idx[:, :case["top"]].contiguous()
        return out
    tau = case["temperature"]
    logp = f["logits"] / tau - torch.logsumexp(f["logits"] / tau, 1, keepdim=True)
    logq = f["top_logits"] / tau - torch.logsumexp(f["top_logits"] / tau, 1, keepdim=True)
    q = torch.exp(logq)
    loss = (q * logq).sum(1) - (q * torch.gather(logp, 1, s["top_ids"])).sum(1)
    grad = torch.exp(logp)
    grad.scatter_add_(1, s["top_ids"], -q)
    return {"loss": loss, "dlogits": grad * (f["weight"] / tau)[:, None]}
