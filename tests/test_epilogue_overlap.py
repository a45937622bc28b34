"""The epilogue calls refuse a buffer that they write where it overlaps any other buffer of the call, before anything is
launched: every written buffer over every other one, at its start and at its last 16 bytes."""
import numpy as np
import pytest

import packed_lora_fine_b200 as pl

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


D_IN, D_OUT, RANKS, COUNTS = 72, 264, [8, 3], [40, 30]
T = sum(COUNTS)
OFF = np.array([0, 40, 70], np.int64)


class Arena:
    """Every buffer of a call in one allocation, 4096 bytes apart."""

    def __init__(self, eng, call):
        tab = pl.make_table(RANKS, [1.0, 1.0], [16, 16], [16, 16])
        relu = pl.make_epilogue("relu", Z=4096)
        back = pl.make_epilogue("gelu", dbias=[16, 16], Z=4096)
        self.size = {"X": T * D_IN * 2, "W": D_OUT * D_IN * 2, "Y": T * D_OUT * 2, "Z": T * D_OUT * 2, "R": T * D_OUT * 2,
                     "dY": T * D_OUT * 2, "dX": T * D_IN * 2,
                     # (the backward reads the part of it that every forward has)
                     "saved": pl.plora_epilogue_saved_bytes(eng.h, 2, OFF, tab, relu) if call is forward
                     else pl.plora_saved_bytes(eng.h, 2, OFF, tab),
                     "work": pl.plora_epilogue_work_bytes(eng.h, 2, OFF, back)}
        for i, r in enumerate(RANKS):
            self.size |= {f"A{i}": r * D_IN * 2, f"B{i}": D_OUT * r * 2, f"dA{i}": r * D_IN * 4, f"dB{i}": D_OUT * r * 4,
                          f"b{i}": D_OUT * 2, f"db{i}": D_OUT * 4}
        self.at, end = {}, 4096
        for k, n in self.size.items():
            self.at[k] = end
            end += (n + 4095) // 4096 * 4096 + 4096
        self.mem = torch.zeros(end + max(self.size.values()), dtype=torch.uint8, device="cuda")

    def pointers(self, moved=None, to=0):
        p = {k: self.mem.data_ptr() + a for k, a in self.at.items()}
        if moved:
            p[moved] = to
        return p


def forward(eng, p, act="relu"):
    tab = pl.make_table(RANKS, [1.0, 1.0], [p["A0"], p["A1"]], [p["B0"], p["B1"]])
    ep = pl.make_epilogue(act, bias=[p["b0"], p["b1"]], residual=p["R"], Z=p["Z"])
    return pl.plora_forward_epilogue(eng.h, p["X"], p["W"], p["Y"], 2, OFF, tab, p["saved"], ep, 0, check=False)


def backward(eng, p):
    tab = pl.make_table(RANKS, [1.0, 1.0], [p["A0"], p["A1"]], [p["B0"], p["B1"]], [p["dA0"], p["dA1"]], [p["dB0"], p["dB1"]])
    ep = pl.make_epilogue("gelu", dbias=[p["db0"], p["db1"]], Z=p["Z"], work=p["work"])
    return pl.plora_backward_epilogue(eng.h, p["X"], p["W"], p["dY"], p["dX"], 2, OFF, tab, p["saved"], ep, 0, check=False)


FORWARD = (["Y", "Z", "saved"], ["X", "W", "Y", "Z", "saved", "R", "A0", "A1", "B0", "B1", "b0", "b1"])
BACKWARD = (["dX", "work", "dA0", "dA1", "dB0", "dB1", "db0", "db1"],
            ["X", "W", "dY", "Z", "saved", "dX", "work", "A0", "A1", "B0", "B1", "dA0", "dA1", "dB0", "dB1", "db0", "db1"])


@gpu
@pytest.mark.parametrize("call, lists", [(forward, FORWARD), (backward, BACKWARD)])
def test_no_written_buffer_overlaps_another(call, lists):
    eng = pl.PackedLoRA(D_IN, D_OUT, "bf16", max_adapters=2, max_rank=8, max_tokens=T)
    a = Arena(eng, call)
    align = {"saved": 256, "work": 256}
    for written in lists[0]:
        for other in lists[1]:
            if other == written:
                continue
            start = a.mem.data_ptr() + a.at[other]
            for at in (start, start + (a.size[other] - 1) // 256 * 256):
                if at % align.get(written, 16) or (written, other, at) == ("Y", "R", start):    # (in place)
                    continue
                assert call(eng, a.pointers(written, at)) == pl.PLORA_ERR_INVALID_ARG, (written, other, at - start)
                assert "overlaps" in pl.plora_last_error(eng.h)
    torch.cuda.synchronize()
    assert not a.mem.any()
    assert call(eng, a.pointers()) == pl.PLORA_OK
    if call is forward:
        p = a.pointers()
        p["R"] = p["Y"]
        assert call(eng, p) == pl.PLORA_OK
        p["B1"] = p["B0"]                   # two adapters may read one factor
        assert call(eng, p) == pl.PLORA_OK
    torch.cuda.synchronize()
    assert pl.plora_check(eng.h, 0) == pl.PLORA_OK
    eng.close()
