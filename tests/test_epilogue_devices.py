"""The epilogue calls refuse tensors that are not on the engine's device, before anything is launched (their pointers would
reach its kernels)."""
import pytest

import packed_lora_fine_b200 as pl

torch = pytest.importorskip("torch")
from test_epilogue_rows import NoLaunch  # noqa: E402


@pytest.mark.parametrize("where", ["X", "W", "A", "B", "bias", "residual", "Y", "dY", "Z"])
def test_another_device_is_refused(where):
    here, there = torch.device("cpu"), torch.device("meta")
    t = lambda name, *s: torch.zeros(s, dtype=torch.bfloat16, device=there if name == where else here)
    X, W, A, B = t("X", 8, 16), t("W", 24, 16), [t("A", 2, 16)], [t("B", 24, 2)]
    kw = dict(bias=t("bias", 24), residual=t("residual", 8, 24))
    e = NoLaunch(16, 24)
    with pytest.raises(ValueError, match="on meta"):
        if where in ("dY", "Z"):
            e.backward_epilogue(X, W, t("dY", 8, 24), [0, 8], [1.0], A, B, None, Z=t("Z", 8, 24), activation="silu")
        else:
            e.forward_epilogue(X, W, [0, 8], [1.0], A, B, activation="silu", Y=t("Y", 8, 24), **kw)
    if where not in ("Y", "dY", "Z"):
        with pytest.raises(ValueError, match="on meta"):
            pl.packed_lora(e, X, W, [0, 8], [1.0], A, B, activation="silu", **kw)


def test_the_engine_knows_its_device(monkeypatch):
    monkeypatch.setattr(pl, "plora_create", lambda *a: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    assert pl.PackedLoRA(16, 24).device == torch.device("cuda", 3)
