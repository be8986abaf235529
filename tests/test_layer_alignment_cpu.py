"""The layer and answer operators refuse pointers that lie between two elements
(a misaligned access would fault on the device) before anything is launched."""
import ctypes as C

import pytest

ADDR, REFUSED = 1 << 20, 1


@pytest.fixture(scope="module")
def lib():
    import post_weight_quantization_row_b200 as m
    return m.lib


def refused(lib, call, names, good, size):
    """call(**pointers) is refused for each pointer in turn that is half an element further than a good one."""
    for name in names:
        for off in {1, size[name] // 2}:
            p = dict(good, **{name: C.c_void_p(ADDR + off)})
            assert call(p) == REFUSED, (name, off)
            assert b"aligned" in lib.mpq_last_error(), (name, off, lib.mpq_last_error())


@pytest.mark.parametrize("rows", [1, 2, 4])
@pytest.mark.parametrize("wide", [0, 1])  # fp32 bias, residual, result
def test_linear(lib, rows, wide):
    size = dict(x=2, w=2, bias=4 if wide else 2, residual=4 if wide else 2, preact=2, y=4 if wide else 2)
    good = {n: C.c_void_p(ADDR) for n in size}
    dt = 0 if wide else 1
    refused(lib, lambda p: lib.mpq_linear(p["x"], 8, p["w"], 8, rows, 8, 8, 1, p["bias"], dt, 0, p["residual"], 8,
                                          p["preact"], p["y"], dt, C.c_void_p(ADDR), 1 << 20, None), size, good, size)


@pytest.mark.parametrize("rows", [0, 3])
@pytest.mark.parametrize("wide", [0, 1])
def test_linear_backward(lib, rows, wide):
    size = dict(dy=2, x=2, w=2, z=2, dx=2, dw=2, db=4 if wide else 2)
    good = {n: C.c_void_p(ADDR) for n in size}
    refused(lib, lambda p: lib.mpq_linear_backward(p["dy"], 8, p["x"], 8, p["w"], 8, p["z"], 8, rows, 8, 8, 2, 2, p["dx"],
                                                   p["dw"], p["db"], 0 if wide else 2, C.c_void_p(ADDR), 1 << 20, None),
            size, good, size)


@pytest.mark.parametrize("dt,pt", [(0, 0), (1, 0), (2, 2)])
def test_layer_norm(lib, dt, pt):
    e, q = (4 if dt == 0 else 2), (4 if pt == 0 else 2)
    size = dict(x=e, w=q, b=q, y=e, mean=4, rstd=4)
    good = {n: C.c_void_p(ADDR) for n in size}
    refused(lib, lambda p: lib.mpq_layer_norm(p["x"], 8, 2, 8, dt, p["w"], p["b"], pt, 1e-5, p["y"], p["mean"], p["rstd"], None),
            size, good, size)
    size = dict(dy=e, x=e, mean=4, rstd=4, w=q, dx=e, dw=q, db=q)
    good = {n: C.c_void_p(ADDR) for n in size}
    for rows in (0, 2):
        refused(lib, lambda p: lib.mpq_layer_norm_backward(p["dy"], 8, p["x"], 8, p["mean"], p["rstd"], rows, 8, dt, p["w"],
                                                           pt, p["dx"], p["dw"], p["db"], C.c_void_p(ADDR), 1 << 20, None),
                size, good, size)


@pytest.mark.parametrize("dt", [0, 1, 2])
def test_answers(lib, dt):
    e = 4 if dt == 0 else 2
    size = dict(l=e, tok=8, lp=4, ent=4, tl=4, ti=8)
    good = {n: C.c_void_p(ADDR) for n in size}
    refused(lib, lambda p: lib.mpq_token_logprobs(p["l"], 8, 2, 8, dt, p["tok"], -100, 2, p["lp"], p["ent"], p["tl"], p["ti"],
                                                  None), size, good, size)
    size = dict(l=e, tl=4, ti=8, w=4, loss=4, d=e)
    good = {n: C.c_void_p(ADDR) for n in size}
    refused(lib, lambda p: lib.mpq_topk_distill(p["l"], 8, 2, 8, dt, p["tl"], p["ti"], 2, p["w"], 1.0, p["loss"], p["d"], None),
            size, good, size)
