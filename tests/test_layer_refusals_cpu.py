"""The layer and answer operators refuse bad arguments before touching a GPU:
through the C ABI with pointers that are never read, and through the binding
with CPU tensors."""
import ctypes as C

import pytest
import torch

P = C.c_void_p(4096)


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def linear(lib, rows=4, n=8, k=8, dtype=1, bias=None, bdt=1, act=0, y=P, ydt=1, x=P, w=P, ldx=8, ldw=8, ws=None, wsb=0):
    return lib.mpq_linear(x, ldx, w, ldw, rows, n, k, dtype, bias, bdt, act, None, 0, None, y, ydt, ws, wsb, None)


def test_linear_refuses(mpq):
    lib = mpq.lib
    for kw in (dict(rows=-1), dict(rows=1 << 24), dict(n=0), dict(k=0), dict(n=1 << 23), dict(k=1 << 23), dict(dtype=0),
               dict(dtype=3), dict(act=5), dict(act=-1), dict(ydt=2), dict(bias=P, bdt=2), dict(x=None), dict(w=None),
               dict(y=None), dict(rows=6, ldx=9), dict(rows=6, ldw=4), dict(rows=6, x=C.c_void_p(4098))):
        assert linear(lib, **kw) == 1, kw
        assert b"linear" in lib.mpq_last_error()
    assert linear(lib, rows=0, x=None, w=None, y=None) == 0  # nothing to do
    # scratch: none for aligned rows or up to 2 of them; both operands' packed copies otherwise
    f = lib.mpq_linear_workspace_bytes
    assert f(P, 8, P, 8, 6, 8, 8) == 0 and f(P, 9, P, 8, 2, 8, 8) == 0 and f(C.c_void_p(4098), 9, P, 9, 1, 8, 8) == 0
    assert f(P, 9, P, 9, 6, 8, 9) == 256 + 256 and f(C.c_void_p(4098), 8, P, 8, 6, 8, 8) == 256
    assert f(P, 0, P, 8, 6, 8, 8) == 256  # rows that overlap
    # too little of it, and off its boundary
    assert linear(lib, rows=6, ldx=9, ws=P, wsb=255) == 1
    assert linear(lib, rows=6, ldx=9, ws=C.c_void_p(4100), wsb=4096) == 1


def test_linear_backward_refuses(mpq):
    lib = mpq.lib

    def back(rows=4, n=8, k=8, dtype=1, act=0, dy=P, x=P, w=P, z=None, dx=P, dw=P, db=P, dbt=1, ws=P, wsb=1 << 20):
        return lib.mpq_linear_backward(dy, n, x, k, w, k, z, n, rows, n, k, dtype, act, dx, dw, db, dbt, ws, wsb, None)

    for kw in (dict(rows=-1), dict(n=0), dict(k=0), dict(dtype=0), dict(act=9), dict(act=1), dict(dy=None), dict(x=None),
               dict(w=None), dict(dbt=2), dict(wsb=0), dict(ws=None), dict(ws=C.c_void_p(4100))):
        assert back(**kw) == 1, kw
    f = lib.mpq_linear_backward_workspace_bytes
    assert f(P, 8, P, 8, P, 8, 4, 8, 8, 0, 1, 1, 0) == 0
    assert f(P, 8, P, 8, P, 8, 4, 8, 8, 0, 1, 1, 1) == 256
    assert f(P, 8, P, 8, P, 8, 4, 8, 8, 2, 1, 1, 0) == 256
    assert f(P, 8, P, 8, P, 8, 4, 8, 8, 2, 0, 0, 0) == 0


def test_layer_norm_refuses(mpq):
    lib = mpq.lib

    def fwd(rows=2, n=8, dt=0, pdt=0, eps=1e-5, x=P, y=P, w=P):
        return lib.mpq_layer_norm(x, n, rows, n, dt, w, None, pdt, eps, y, None, None, None)

    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(n=0), dict(n=1 << 21), dict(dt=3), dict(dt=-1), dict(dt=1, pdt=2),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=1e-60), dict(x=None), dict(y=None)):
        assert fwd(**kw) == 1, kw
    assert fwd(rows=0, x=None, y=None) == 0

    def bwd(rows=2, n=8, dt=0, pdt=0, dy=P, x=P, m=P, r=P, ws=P, wsb=1 << 20):
        return lib.mpq_layer_norm_backward(dy, n, x, n, m, r, rows, n, dt, P, pdt, P, P, P, ws, wsb, None)

    for kw in (dict(rows=-1), dict(n=0), dict(dt=5), dict(dt=2, pdt=1), dict(dy=None), dict(x=None), dict(m=None),
               dict(r=None), dict(ws=None), dict(wsb=8), dict(ws=C.c_void_p(4097))):
        assert bwd(**kw) == 1, kw
    f = lib.mpq_layer_norm_backward_workspace_bytes
    assert f(2, 8, 0) == 0 and f(0, 8, 1) == 0 and f(2, 8, 1) >= 2 * 2 * 8 * 4


def test_answers_refuse(mpq):
    lib = mpq.lib

    def lp(rows=2, v=8, dt=0, top=2, tokens=P, out=P, tl=P, ti=P, l=P):
        return lib.mpq_token_logprobs(l, v, rows, v, dt, tokens, -100, top, out, P, tl, ti, None)

    for kw in (dict(rows=-1), dict(rows=1 << 25), dict(v=0), dict(v=1 << 25), dict(dt=3), dict(top=-1), dict(top=9),
               dict(v=1000, top=129), dict(tokens=None), dict(out=None), dict(tl=None), dict(ti=None), dict(l=None),
               dict(l=C.c_void_p(4097))):
        assert lp(**kw) == 1, kw
    assert lp(rows=0, l=None) == 0

    def kd(rows=2, v=8, dt=0, top=2, t=1.0, l=P, tl=P, ti=P, loss=P):
        return lib.mpq_topk_distill(l, v, rows, v, dt, tl, ti, top, None, t, loss, P, None)

    for kw in (dict(rows=-1), dict(v=0), dict(dt=3), dict(top=0), dict(top=129), dict(t=0.0), dict(t=float("nan")),
               dict(t=float("inf")), dict(l=None), dict(tl=None), dict(ti=None), dict(loss=None), dict(l=C.c_void_p(4098))):
        assert kd(**kw) == 1, kw
    assert kd(rows=0, l=None) == 0


def test_binding_refuses_cpu_tensors(mpq):
    b = torch.ones(2, 8, dtype=torch.bfloat16)
    for f in (lambda: mpq.linear(b, b), lambda: mpq.linear_backward(b, b, b), lambda: mpq.layer_norm(b),
              lambda: mpq.layer_norm_backward(b, b, b, b), lambda: mpq.token_logprobs(b),
              lambda: mpq.topk_distill(b, b, b)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
