"""The layer and answer operators called by several host threads at once, each
on a stream of its own."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def test_calls_of_several_threads(mpq):
    def inputs(i):
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
        return r(300 + i, 513), r(640, 513), r(640), r(3 + i, 30000)

    def step(x, w, b, l):
        h, mean, rstd = mpq.layer_norm(x, stats=True)
        y, z = mpq.linear(h, w, b, activation="silu", preact=True)
        d = mpq.linear_backward(y, h, w, z, "silu")
        e = mpq.layer_norm_backward(d["dx"], x, mean, rstd)
        p = mpq.token_logprobs(l, top=9)
        q = mpq.topk_distill(l, p["top_logprob"], p["top_id"])
        return [y, z, *d.values(), *e.values(), *p.values(), *q.values()]

    data = [inputs(i) for i in range(4)]
    want = [step(*d) for d in data]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(len(data))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait(60)
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step(*data[i])
                    stream.synchronize()
                    wrong.extend((i, k) for k, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
            mpq.ops_status()
        except Exception as e:  # (a thread's exception would be lost)
            wrong.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    # (a thread's first ops_status also tells of what another test let run out)
    assert not [w for w in wrong if not isinstance(w[1], mpq.MPQError)], wrong
