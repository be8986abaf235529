"""ops_status: a wait that ran out is reported to every thread, once, whatever
stream it ran on and whoever asked before."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mpq():
    import post_weight_quantization_row_b200 as m
    return m


def expire(mpq, stream):
    assert mpq.lib.mpq_ops_expire(stream.cuda_stream) == 0


def asked(mpq):
    """Whether ops_status reports a timeout."""
    try:
        mpq.ops_status()
        return False
    except mpq.MPQError as e:
        assert "wait" in str(e)
        return True


def in_thread(f):
    got = []
    t = threading.Thread(target=lambda: got.append(f()))
    t.start()
    t.join()
    return got[0]


def test_a_timeout_is_reported_once(mpq):
    asked(mpq)  # (what other tests of this process have left)
    assert not asked(mpq)
    expire(mpq, torch.cuda.current_stream())
    assert asked(mpq) and not asked(mpq)
    side = torch.cuda.Stream()
    expire(mpq, side)
    side.synchronize()
    assert asked(mpq) and not asked(mpq)


def test_no_thread_takes_anothers(mpq):
    asked(mpq)
    ready, go, seen = threading.Event(), threading.Event(), []

    def other():
        asked(mpq)
        seen.append(asked(mpq))
        ready.set()
        go.wait(60)
        seen.append(asked(mpq))
        seen.append(asked(mpq))

    t = threading.Thread(target=other)
    t.start()
    assert ready.wait(60)
    side = torch.cuda.Stream()
    expire(mpq, side)
    side.synchronize()
    assert asked(mpq)          # here first
    go.set()
    t.join()
    assert seen == [False, True, False]
    assert not asked(mpq)
    # a thread that asks for the first time hears of what was before it
    assert in_thread(lambda: (asked(mpq), asked(mpq))) == (True, False)


def test_a_timeout_between_two_calls_is_not_lost(mpq):
    asked(mpq)
    for _ in range(20):
        streams = [torch.cuda.Stream() for _ in range(4)]
        for s in streams:
            expire(mpq, s)
        first = asked(mpq)     # some, all or none of them have run
        for s in streams:
            s.synchronize()
        assert asked(mpq) or first
        assert not asked(mpq)


def test_status_of_good_calls(mpq):
    asked(mpq)
    x = torch.ones(300, 64, dtype=torch.bfloat16, device="cuda")
    mpq.linear(x, x[:64])
    assert not asked(mpq)
