"""Several threads' first calls through the binding at once: what a first call sets up is right whoever comes last."""
import builtins
import threading

import pytest
import torch


@pytest.fixture(scope="module")
def b():
    from mxfp4_routed_expert_router_gb300 import build
    build.build()
    from mxfp4_routed_expert_router_gb300 import binding
    return binding


def _at_once(monkeypatch, call, n=4):
    """Runs `call` in n threads that are all past its first look when the first of them goes on."""
    meet, real, errors = threading.Barrier(n, timeout=20), builtins.__import__, []

    def late(name, *args, **kw):
        if name == "torch" and threading.current_thread().name == "first call":
            meet.wait()
        return real(name, *args, **kw)

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    with monkeypatch.context() as m:
        m.setattr(builtins, "__import__", late)
        threads = [threading.Thread(target=work, name="first call") for _ in range(n)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not errors


@pytest.mark.parametrize("name,fill", [("_ATTN", "_attn"), ("_DTYPES", "_dtypes")])
def test_first_calls_of_several_threads(b, monkeypatch, name, fill):
    monkeypatch.setattr(b, name, type(getattr(b, name))())
    _at_once(monkeypatch, getattr(b, fill))
    got = tuple(getattr(b, name))
    assert got[:2] == ((torch.bfloat16, torch.int32) if name == "_ATTN" else (torch.float32, torch.int32))
    assert len(got) == (4 if name == "_ATTN" else 2)
    # and calls after them: refused for what is wrong with them
    z = torch.zeros
    with pytest.raises(b.MoeError) as e:
        if name == "_ATTN":
            b.moe_attention_prompt(z((3, 4, 64)), z((3, 2, 64)), z((3, 2, 64)), z(2), 0.1, z((3, 4, 64)))
        else:
            b.moe_route_grouped(z((2, 8)).half(), None, 2, 8, 2, 1, 1, 0, 0, True, 1.0, None, None)
    assert e.value.status == b.MOE_EINVAL
