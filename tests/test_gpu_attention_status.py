"""moe_attention_status: an error that a kernel recorded reaches every stream that asks, once, and none is lost."""
import threading

import pytest
import torch

from test_gpu_attention_decode import make

pytestmark = pytest.mark.gpu


def _state():
    c, q, table, n = make([20, 30], 4, 2, 64, 16, "bf16", 3)
    wrong = n.clone()
    wrong[1] = -1
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    return c, q, table, n, wrong, streams


def _heard(stream):
    """Whether the stream's report tells of an error."""
    from mxfp4_routed_expert_router_gb300 import attention as A, binding as B
    try:
        A.sync(stream)
    except B.MoeError as e:
        assert e.status == B.MOE_EDEVICE
        return True
    return False


def test_each_stream_hears_of_an_error_once():
    c, q, table, n, wrong, (a, b, other) = _state()
    for s in (a, b, other, None):
        _heard(s)  # (what came before)
    for _ in range(3):
        with torch.cuda.stream(a):
            c.decode(q, table, wrong)
        torch.cuda.synchronize()
        assert _heard(b)  # asks first
        assert _heard(a) and _heard(other) and _heard(None)
        assert not _heard(a) and not _heard(b) and not _heard(other) and not _heard(None)
    with torch.cuda.stream(b):
        c.decode(q, table, n)
    assert not any(_heard(s) for s in (a, b, other, None))


def test_a_replay_on_another_stream():
    c, q, table, n, wrong, (a, b, other) = _state()
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.decode(q, table, wrong, out=out)
    for s in (a, b, None):
        _heard(s)
    with torch.cuda.stream(b):
        g.replay()
    torch.cuda.synchronize()
    assert _heard(a) and _heard(b) and _heard(None) and not _heard(b)


def test_no_error_is_lost_between_reports():
    """Two threads, each with a stream: every one of their wrong calls is followed by a report that tells of it."""
    c, q, table, n, wrong, (a, b, _) = _state()
    missed = []

    def work(stream):
        torch.cuda.set_device(0)
        for _ in range(300):
            with torch.cuda.stream(stream):
                c.decode(q, table, wrong)
            if not _heard(stream):
                missed.append(stream)

    threads = [threading.Thread(target=work, args=(s,)) for s in (a, b)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not missed
    for s in (a, b, None):
        _heard(s)
    assert not any(_heard(s) for s in (a, b, None))


def test_many_reports_at_once_on_one_stream():
    c, q, table, n, wrong, (a, _, _) = _state()
    _heard(a)
    with torch.cuda.stream(a):
        c.decode(q, table, wrong)
    heard = []
    threads = [threading.Thread(target=lambda: heard.append(_heard(a))) for _ in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sum(heard) == 1
    _heard(None)
