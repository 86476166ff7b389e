"""Every value of moe_linear_forward on the GPU: none unwritten and none NaN that is not one.

Tolerances are those of test_gpu_linear (FP32 accumulation of exact products); a
value that is not a number is outside them, and outputs start as NaN.
"""
import inspect

import numpy as np
import pytest
import torch

import test_gpu_linear as base
from test_gpu_linear import FMTS, Weight, _x

pytestmark = pytest.mark.gpu


def close(got, x, W, out_bf16=False, base=None):
    got = got.float().cpu().numpy().astype(np.float64)
    sick = np.isnan(x).any(1)  # (E4M3 rows of randn * 100 hold a NaN where a value passes 448)
    assert np.isnan(got[sick]).all()
    got, x, base = got[~sick], x[~sick], None if base is None else base[~sick]
    ref = x @ W.w.T
    tol = (W.K / 16 + 32) * 2.0 ** -23 * (np.abs(x) @ W.terms.T)
    if base is not None:
        ref = ref + base
        tol = tol + 2.0 ** -23 * np.abs(ref)
    if out_bf16:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.isfinite(ref).all() and np.isfinite(tol).all()
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], ref[bad][:4])


def nan_out(lin, T, dtype=torch.float32):
    return torch.full((T, lin.N), float("nan"), dtype=dtype, device="cuda")


def value_tests():
    """The tests of test_gpu_linear that compare values, with each of their parameters."""
    for name, f in sorted(vars(base).items()):
        if name.startswith("test_") and "_check(" in inspect.getsource(f):
            sets = [{}]
            for m in getattr(f, "pytestmark", []):
                if m.name == "parametrize":
                    keys = [k.strip() for k in m.args[0].split(",")]
                    sets = [{**s, **dict(zip(keys, v if len(keys) > 1 else (v,)))} for s in sets for v in m.args[1]]
            for s in sets:
                yield pytest.param(f, s, id="-".join([name[5:]] + [str(v) for v in s.values()]))


@pytest.mark.parametrize("test,args", list(value_tests()))
def test_values_are_written_and_numbers(test, args, monkeypatch):
    """The value tests of test_gpu_linear, whose own comparison lets a NaN pass, with one that does not and with
    outputs that start as NaN."""
    B, Linear = base._mods()

    class Filled(Linear):
        def forward(self, x, x_scales=None, out=None, **kw):
            if out is None and not kw:
                out = nan_out(self, x.shape[0])
            return super().forward(x, x_scales, out=out, **kw)

    monkeypatch.setattr(base, "_check", close)
    monkeypatch.setattr(base, "_mods", lambda: (B, Filled))
    test(**args)
