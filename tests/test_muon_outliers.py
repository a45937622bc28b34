"""The Muon step on gradients that one direction dominates: long-side columns, or a short-side row, far larger than
the rest, as an outlier input feature leaves them in dA_i = G_i^T X_i.  The orthogonalised matrix against float64.

Tolerance, relative to |O|_F.  What the dominating part leaves of the rest is summed by the tensor cores, which round an
accumulator by at most 2^-23 of it per step.  Gram: at most 64 steps before the sums go to float64, 64 2^-23 of G, half
of that in the singular values, and the polynomial's relative slope is at most 2: 128 2^-24.  Q X_0: eight products
of s / 16 steps, each rounding off half of 2^-23 in the mean: s / 2 2^-24.  With p = 0 and lr = 1 the step returns -O."""
import pytest

import packed_lora_fine_b200 as pl
from test_muon import orth64

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


def orthogonalised(eng, ranks, gA, gB):
    """O of every matrix (A's, then B's), by one step from zero."""
    z = lambda v: [torch.zeros_like(x) for x in v]
    pA, pB, mA, mB = z(gA), z(gB), z(gA), z(gB)
    ptr = lambda v: [x.data_ptr() for x in v]
    tab = pl.make_table(ranks, [1.0] * len(ranks), ptr(pA), ptr(pB), ptr(gA), ptr(gB))
    st = pl.make_muon_states([dict(lr=1.0, momentum=0.0, nesterov=False, scale="none")] * len(ranks), None, None, ptr(mA), ptr(mB))
    work = torch.full((pl.plora_muon_work_bytes(eng.h, len(ranks), tab),), 255, dtype=torch.uint8, device="cuda")
    pl.plora_muon_step(eng.h, len(ranks), tab, st, work.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert pl.plora_check(eng.h, 0) == pl.PLORA_OK
    return [-x for x in pA + pB]


@gpu
@pytest.mark.parametrize("d_in", [4104, 1000])
@pytest.mark.parametrize("kind", ["column", "columns", "row"])
@pytest.mark.parametrize("factor", [1, 30, 300, 1000, 3000])
def test_outliers(kind, factor, d_in):
    g = torch.Generator(device="cuda").manual_seed(factor)
    ranks = [16, 5, 64, 100, 128, 256]
    d_out = 2056
    gA = [torch.randn(r, d_in, generator=g, device="cuda") * 1e-3 for r in ranks]
    gB = [torch.randn(d_out, r, generator=g, device="cuda") * 1e-3 for r in ranks]
    for x in gA + [b.T for b in gB]:
        if kind == "column":
            x[:, 77] *= factor
        elif kind == "columns":
            x[:, 77::x.shape[1] // 5] *= factor
        else:
            x[3] *= factor
    eng = pl.PackedLoRA(d_in, d_out, "fp32", max_adapters=len(ranks), max_rank=256, max_tokens=16)
    for got, u in zip(orthogonalised(eng, ranks, gA, gB), gA + gB):
        o = orth64(u)
        err = float((got.double() - o).norm()) / float(o.norm())
        assert err <= (128 + min(u.shape) / 2) * 2.0 ** -24, (tuple(u.shape), err)
    eng.close()


@gpu
@pytest.mark.parametrize("largest", [1.7e38, 2.3e38, 3.4e38, 1e-20])
def test_the_largest_floats(largest):
    """u up to the end of fp32 (eps is nothing next to it, or, at 1e-20, everything): no scale overflows."""
    g = torch.Generator(device="cuda").manual_seed(5)
    ranks = [5, 100, 200]
    gA = [torch.randn(r, 1000, generator=g, device="cuda").clamp(-4, 4) * (largest / 4) for r in ranks]
    gB = [torch.randn(264, r, generator=g, device="cuda").clamp(-4, 4) * (largest / 4) for r in ranks]
    gA[0][1, 3] = gB[1][263, 99] = largest
    eng = pl.PackedLoRA(1000, 264, "fp32", max_adapters=len(ranks), max_rank=256, max_tokens=16)
    for got, u in zip(orthogonalised(eng, ranks, gA, gB), gA + gB):
        o = orth64(u)
        assert float((got.double() - o).norm()) <= (128 + min(u.shape) / 2) * 2.0 ** -24 * float(o.norm()), tuple(u.shape)
    eng.close()
