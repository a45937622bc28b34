"""Y of an inference call against a training call's on the same inputs, above the few-token kernels' 32 tokens.

Both take the same kernels and sums, so Y is equal to the bit; with relu a bf16 training call takes H' in two bf16 parts
where the inference call rounds it, half a step, U = 2^-8, of each |H'|, and both round Y: U |H'||B| + 2 U |Y|."""
import pytest

import packed_lora_fine_b200 as pl
from test_epilogue import ACTS, Problem, U, infer

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", ACTS)
def test_inference_gives_the_training_call_s_output(act, dtype):
    p = Problem(dtype, 136, 264, [8, 50], [40, 130], residual=False, seed=31)
    eng = p.engine()
    Y = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act)[0]
    Yi = infer(p, eng, act)
    if act != "relu" or dtype == "fp32":
        assert torch.equal(Y, Yi)
    else:
        low = torch.cat([p.scales[i] * (p.X[p.off[i]:p.off[i + 1]].double() @ p.A[i].double().T).abs() @ p.B[i].double().abs().T
                         for i in range(p.n)])
        # (an element whose H' rounds to itself differs by nothing, so U and a sixteenth covers the sums' drift)
        assert bool(((Y.double() - Yi.double()).abs() <= 17 / 16 * U * low + 2 * U * Y.double().abs()).all())
        assert not torch.equal(Y, Yi)
    eng.close()
