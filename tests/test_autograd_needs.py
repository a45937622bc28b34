"""What packed_lora computes and returns when only some of its inputs need a gradient.

Tolerance: a bias gradient is a sum of fp32 dZ rounded to bf16 once (half a step, 2^-8 relative) after at most
rows 2^-24 of the magnitudes; dA and dB take the 2-norm bounds of test_epilogue."""
import pytest

import packed_lora_fine_b200 as pl
from test_epilogue import Problem, U, rel

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


@gpu
@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("needed", ["X", "A", "B", "bias", "R"])
def test_one_input_alone(needed, act, monkeypatch):
    p = Problem("bf16", 72, 72, [4, 3], [9, 150], seed=16)
    eng = p.engine()
    asked, call = [], pl.plora_backward_epilogue

    def watched(h, X, W, dY, dX, n, off, tab, saved, ep, *rest):
        asked.append((dX is not None, bool(ep.dbias)))
        return call(h, X, W, dY, dX, n, off, tab, saved, ep, *rest)
    monkeypatch.setattr(pl, "plora_backward_epilogue", watched)
    inputs = {"X": [p.X], "A": p.A, "B": p.B, "bias": p.bias, "R": [p.R]}
    for t in inputs[needed]:
        t.requires_grad_(True)
    Y = pl.packed_lora(eng, p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act, residual=p.R)
    Y.backward(p.dY)
    assert asked == [(needed == "X", needed == "bias")]
    for name, tensors in inputs.items():
        for t in tensors:
            assert (t.grad is not None) == (name == needed)
    Z = None if act == "none" else eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act)[2]
    ref = p.reference(act, None if Z is None else Z.detach())
    want = {"X": [ref["dX"]], "A": ref["dA"], "B": ref["dB"], "bias": ref["db"], "R": [p.dY]}[needed]
    most = {"X": 3 * U, "A": 3 * U, "B": 3 * U, "bias": U + 150 * 2.0 ** -20, "R": 0.0}[needed]
    for t, w in zip(inputs[needed], want):
        assert rel(t.grad, w) <= most, (needed, rel(t.grad, w))
    eng.close()
