"""The epilogue calls on another stream than the current one: what they allocate comes from the current stream's memory,
so they wait for work there on what that memory held before, and it goes back only behind them."""
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
@pytest.mark.parametrize("call", ["forward", "inference", "backward"])
def test_memory_that_the_current_stream_still_uses(call):
    p = Problem("bf16", 264, 1032, [16, 8], [140, 57], seed=95)
    eng, side = p.engine(), torch.cuda.Stream()
    args = (p.X, p.W, p.off, p.scales, p.A, p.B)
    Y, saved, Z = eng.forward_epilogue(*args, bias=p.bias, activation="gelu")

    def run(stream=None):
        if call == "backward":
            r = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="gelu", want_dbias=True,
                                      stream=stream)
            return [r[0], *r[1], *r[2], *r[3]]
        r = eng.forward_epilogue(*args, bias=p.bias, activation="gelu", want_Z=call == "forward", stream=stream)
        return [t for t in (r[0], r[2]) if t is not None]
    want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    # given back with a write to come: blocks of every size that the call asks for
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in [1 << k for k in range(9, 22)] for _ in range(8)]
    torch.cuda._sleep(50_000_000)
    for t in held:
        t.fill_(255)
    del held, t
    got = run(side)
    # and the call's own blocks, given back before it has run
    other = [torch.empty_like(t).fill_(7) for t in run(side)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 7).all()) for t in other)
    eng.close()


@gpu
def test_captured_on_a_stream_that_is_not_current():
    p = Problem("bf16", 264, 1032, [16, 8], [10, 7], seed=96)
    eng, side = p.engine(), torch.cuda.Stream()
    args = (p.X, p.W, p.off, p.scales, p.A, p.B)
    Y = torch.empty_like(p.dY)
    saved = torch.empty(eng.saved_bytes(p.off, eng.table(p.scales, p.A, p.B)), dtype=torch.uint8, device="cuda")
    run = lambda s: eng.forward_epilogue(*args, bias=p.bias, activation="gelu", want_Z=False, Y=Y, saved=saved, stream=s)
    run(None)
    want = Y.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        g.capture_begin()
    run(side)
    with torch.cuda.stream(side):
        g.capture_end()
    Y.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Y, want)
    del g
    eng.close()
