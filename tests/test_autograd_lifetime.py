"""packed_lora's backward with gradients that are not contiguous: the copy that the kernels read lives until they are
launched, and the gradients are those of the contiguous one."""
import pytest

import packed_lora_fine_b200 as pl
from test_epilogue import Problem

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


@gpu
@pytest.mark.parametrize("plain", [True, False])
def test_a_gradient_that_is_not_contiguous(plain, monkeypatch):
    p = Problem("bf16", 72, 264, [8, 3], [130, 21], seed=91)
    eng = p.engine()
    name = "plora_backward" if plain else "plora_backward_epilogue"
    call, taken = getattr(pl, name), []

    def watched(h, X, W, dY, *rest):
        # what a second thread could be given while the call is made
        other = torch.empty((p.T, p.d_out), dtype=torch.bfloat16, device="cuda")
        taken.append(other.data_ptr() == dY)
        return call(h, X, W, dY, *rest)
    monkeypatch.setattr(pl, name, watched)

    def run(dY):
        leaves = [t.clone().requires_grad_(True) for t in [p.X, *p.A, *p.B]]
        Y = pl.packed_lora(eng, leaves[0], p.W, p.off, p.scales, leaves[1:3], leaves[3:], **({} if plain else dict(bias=p.bias, activation="silu")))
        Y.backward(dY)
        return [t.grad for t in leaves]
    wide = p.dY[:, :1].expand(p.T, p.d_out)
    turned = p.dY.t().contiguous().t()
    for dY in (wide, turned):
        assert not dY.is_contiguous()
        got, want = run(dY), run(dY.contiguous())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert len(taken) == 4 and not any(taken)
    eng.close()
