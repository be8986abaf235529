"""The operators stand outside autograd, and say so where a gradient is expected
of them."""
import warnings

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def calls(mpq, t):
    """The forward calls, with `t` as each of their inputs in turn."""
    c = lambda *s, dt=torch.bfloat16: torch.ones(*s, dtype=dt, device="cuda")
    ids = torch.zeros(8, 2, dtype=torch.int64, device="cuda")
    b, v = t(c(8, 8)), t(c(8))
    f = t(c(8, 8, dt=torch.float32))
    return [("linear", lambda: mpq.linear(b, c(8, 8))), ("linear", lambda: mpq.linear(c(8, 8), b)),
            ("linear", lambda: mpq.linear(c(8, 8), c(8, 8), v)), ("linear", lambda: mpq.linear(c(8, 8), c(8, 8), residual=b)),
            ("layer_norm", lambda: mpq.layer_norm(b)), ("layer_norm", lambda: mpq.layer_norm(c(8, 8), v)),
            ("layer_norm", lambda: mpq.layer_norm(c(8, 8), bias=v)), ("token_logprobs", lambda: mpq.token_logprobs(f)),
            ("topk_distill", lambda: mpq.topk_distill(f, c(8, 2, dt=torch.float32), ids)),
            ("topk_distill", lambda: mpq.topk_distill(c(8, 8), t(c(8, 2, dt=torch.float32)), ids))]


def test_inputs_that_require_a_gradient_are_warned_of(mpq):
    for name, f in calls(mpq, lambda x: x.requires_grad_()):
        with pytest.warns(UserWarning, match=f"{name} takes no part in autograd") as said:
            out = f()
        assert said[0].filename == __file__  # the caller's line
        for r in out.values() if isinstance(out, dict) else [out]:
            assert not r.requires_grad


def test_no_warning_without_a_gradient_to_lose(mpq):
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for _, f in calls(mpq, lambda x: x):
            f()
        with torch.no_grad():
            for _, f in calls(mpq, lambda x: x.requires_grad_()):
                f()
        p = torch.nn.Parameter(torch.ones(8, 8, dtype=torch.bfloat16, device="cuda"))
        dy = torch.ones(3, 8, dtype=torch.bfloat16, device="cuda")
        mpq.linear_backward(dy, dy, p)  # the gradients themselves need no warning
