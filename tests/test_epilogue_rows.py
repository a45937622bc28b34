"""The projection with its epilogue where the segment offsets and the rows of X differ: more rows in X than the last
adapter's end are left alone or zero, fewer are refused before anything is launched."""
import numpy as np
import pytest

import packed_lora_fine_b200 as pl

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


class NoLaunch(pl.PackedLoRA):
    """An engine without a handle: whatever passes the checks of the arguments fails the test."""

    def __init__(self, d_in, d_out):
        self.d_in, self.d_out, self.dtype, self.out_blocks, self.h = d_in, d_out, "bf16", None, None
        self.device = torch.device("cpu")

    def table(self, *a):
        raise AssertionError("not refused")


@pytest.mark.parametrize("off", [[0, 3, 9], [0, 8, 1 << 40]])
def test_offsets_past_the_rows_are_refused(off):
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    X, W, A, B, dY = t(8, 16), t(24, 16), [t(2, 16)] * 2, [t(24, 2)] * 2, t(8, 24)
    e = NoLaunch(16, 24)
    for off_ in (off, np.array(off)):
        for call in (lambda: e.forward_epilogue(X, W, off_, [1.0, 1.0], A, B),
                     lambda: e.forward_epilogue(X, W, off_, [1.0, 1.0], A, B, activation="silu", want_Z=False),
                     lambda: e.backward_epilogue(X, W, dY, off_, [1.0, 1.0], A, B, None),
                     lambda: pl.packed_lora(e, X, W, off_, [1.0, 1.0], A, B),
                     lambda: pl.packed_lora(e, X, W, off_, [1.0, 1.0], A, B, bias=t(24), residual=dY)):
            with pytest.raises(ValueError, match="off: the last adapter ends at row"):
                call()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("plain", [False, True])
def test_rows_behind_the_last_adapter(dtype, plain):
    """A padded batch: its rows are zero in Y and in the gradients, whatever they hold in X, residual and dY, and the
    other rows are as without them."""
    from test_epilogue import Problem
    p = Problem(dtype, 72, 264, [8, 3], [130, 21], extra=11, seed=90)
    eng = p.engine()
    kw = {} if plain else dict(bias=p.bias, activation="silu", residual=p.R)

    def run(rows):
        cut = lambda t: t[:rows].clone().requires_grad_(True)
        X, A, B = cut(p.X), [a.clone().requires_grad_(True) for a in p.A], [b.clone().requires_grad_(True) for b in p.B]
        R = None if plain else cut(p.R)
        trash = [torch.full((p.T + 11, n), float("nan"), dtype=X.dtype, device="cuda") for n in (p.d_in, p.d_out, p.d_out)]
        del trash          # what new tensors hold if nothing is written
        Y = pl.packed_lora(eng, X, p.W, p.off, p.scales, A, B, **(kw | ({} if plain else dict(residual=R))))
        Y.backward(p.dY[:rows])
        return [Y.detach(), X.grad] + ([] if plain else [R.grad]), [t.grad for t in A + B]
    whole, weights = run(p.T + 11)
    alone, same = run(p.T)
    for a, b in zip(whole, alone):
        assert torch.equal(a[:p.T], b) and not a[p.T:].any()
    assert all(torch.equal(a, b) for a, b in zip(weights, same))
    if not plain:
        Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, **kw)
        dX = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="silu")[0]
        assert not Y[p.T:].any() and not Z[p.T:].any() and not dX[p.T:].any()
        kept = torch.full_like(Y, 3.0)
        eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, Y=kept, **kw)
        assert torch.equal(kept[:p.T], Y[:p.T]) and bool((kept[p.T:] == 3).all())
    eng.close()
