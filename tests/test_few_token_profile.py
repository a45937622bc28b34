"""Launch accounting of the few-token inference call, which takes no schedule slot: captured calls are counted and not
timed, later ones are timed again."""
import pytest

import packed_lora_fine_b200 as pl
from test_epilogue import Problem, infer

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


@gpu
def test_profile_around_a_capture():
    p = Problem("bf16", 136, 264, [4, 17], [1, 7], seed=97)
    eng = p.engine()
    tab = eng.table(p.scales, p.A, p.B)
    Y, saved = infer(p, eng, "silu"), torch.empty(eng.saved_bytes(p.off, tab), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pl.plora_profile_enable(eng.h, True)
    pl.plora_profile_read(eng.h)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        infer(p, eng, "silu", Y=Y, saved=saved)
    r = pl.plora_profile_read(eng.h)
    assert r["few_base"] == (1, 0.0) and r["few_shrink"] == (1, 0.0)
    g.replay()
    infer(p, eng, "silu")
    r = pl.plora_profile_read(eng.h)
    assert r["few_base"][0] == 1 and 0 < r["few_base"][1] < 100
    # a captured call that takes a slot, then a few tokens
    pl.plora_capture_reserve(eng.h, 1)
    h = torch.cuda.CUDAGraph()
    buf = torch.empty_like(Y)
    ep = pl.make_epilogue("none")
    with torch.cuda.graph(h):
        pl.plora_forward_epilogue(eng.h, p.X.data_ptr(), p.W.data_ptr(), buf.data_ptr(), 2, p.off, tab, saved.data_ptr(), ep,
                                  torch.cuda.current_stream().cuda_stream)
    infer(p, eng, "silu")
    r = pl.plora_profile_read(eng.h)
    assert r["few_base"][0] == 1 and 0 < r["few_base"][1] < 100
    del g, h
    pl.plora_capture_release(eng.h)
    eng.close()
