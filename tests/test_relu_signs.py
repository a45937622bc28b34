"""relu's training forward on the tensor cores: Z's sign is the formula's, since relu's derivative jumps with it.

The signs are compared with float64's without a tolerance: a Z that the library computes anew is off by the float64
sums' own roundings, (K + 8) 2^-53 of its products' magnitudes, and no |Z| of these inputs is below 2^-40.  Gradients
take the tolerances of test_epilogue, with the derivative at float64's Z."""
import numpy as np
import pytest

import packed_lora_fine_b200 as pl
from test_epilogue import Problem, U, bounds, inside, rel

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


def forward(p, eng, residual=None):
    Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="relu", residual=residual)
    torch.cuda.synchronize()
    assert pl.plora_check(eng.h, 0) == pl.PLORA_OK
    return Y, saved, Z


def z64(p):
    d = lambda v: [None if t is None else t.double() for t in v]
    return p.z64(p.X.double(), d(p.A), d(p.B), d(p.biases()))


# d_in, d_out, ranks, counts, blocks, bias: long sums over adapters of 1 to 20 rows (and one of many)
LONG = [
    (8192, 2056, [1, 4, 16, 64, 3] * 4, list(range(1, 21)), 1, "each"),
    (10808, 1544, [1] * 16, [1, 2, 3, 5] * 4, 1, "none"),
    (14336, 1032, [256, 100], [700, 9], 1, "shared"),
    (8200, 2304, [8, 24, 3], [7, 130, 1], 3, "some"),
    (264, 4104, [17, 1], [1000, 3], 1, "each"),
]


@gpu
@pytest.mark.parametrize("k", range(len(LONG)))
def test_signs_and_gradients_of_long_sums(k):
    d_in, d_out, ranks, counts, blocks, bias = LONG[k]
    p = Problem("bf16", d_in, d_out, ranks, counts, blocks=blocks, bias=bias, residual=False, seed=50 + k)
    if k == 1:
        p.scales = [16.0] * p.n
    eng = p.engine()
    Y, saved, Z = forward(p, eng)
    z = z64(p)
    assert float(z.abs().min()) > 2.0 ** -40
    assert int(((Z > 0) != (z > 0)).sum()) == 0
    assert torch.equal(Y > 0, Z > 0)
    want = [b is not None for b in p.biases()]
    dX, dA, dB, db = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="relu",
                                           want_dbias=want)
    ref = p.reference("relu")
    b = bounds(p, ref, None, "relu", (max(d_in, d_out, p.T) + 8) * 2.0 ** -24 + U)
    assert inside(dX, ref["dX"], b["dX"]) and rel(dX, ref["dX"]) <= 3 * U
    for i in range(p.n):
        assert inside(dA[i], ref["dA"][i], b["dA"][i]), i
        assert inside(dB[i], ref["dB"][i], b["dB"][i]) and rel(dB[i], ref["dB"][i]) <= 2 * U, i
        if want[i]:       # sums of unrounded dY in fp32
            assert float((db[i].double() - ref["db"][i]).abs().max()) <= 2.0 ** -22 * counts[i] * 8, i
    again = forward(p, eng)
    assert torch.equal(again[0], Y) and torch.equal(again[2], Z)
    eng.close()


@gpu
@pytest.mark.parametrize("residual", [False, True])
def test_sums_that_cancel(residual):
    """Every Z is what is left of long sums that cancel: +-2^-14 or 0 of products up to 1, in every column of every tile,
    with a low-rank part that the bias takes back (1.5 = s x a, exactly).  2^-14 is below the drift of 8192 products."""
    K, N = 8192, 264
    p = Problem("bf16", K, N, [1, 20], [140, 3], bias="each", residual=residual, seed=60)
    g = torch.Generator().manual_seed(61)
    half = torch.rand(N, K // 2 - 4, generator=g).bfloat16().float()
    at = torch.randperm(K - 8, generator=g)
    W = torch.zeros(N, K)
    W[:, at] = torch.cat([half, -half], 1)
    sign = (torch.arange(N) % 3 - 1).float()              # -1, 0, 1
    W[:, K - 1] = sign * 2.0 ** -14
    p.W, p.X = W.bfloat16().cuda(), torch.ones_like(p.X)
    p.scales = [1.5, 1.5]
    for i in range(2):
        p.A[i].zero_()
        p.A[i][0, K - 2] = 1
        p.B[i].zero_()
        p.B[i][:, 0] = 1
        p.bias[i].fill_(-1.5)
    eng = p.engine()
    Y, saved, Z = forward(p, eng, p.R)
    want = (sign * 2.0 ** -14).cuda().expand(p.T, N)
    assert torch.equal(Z.float(), want)
    if not residual:
        assert torch.equal(Y.float(), want.clamp(min=0))
    else:                 # Y is what the sums gave: within their drift and its rounding of the residual
        assert float((Y.double() - p.R.double() - want.clamp(min=0)).abs().max()) <= 2.0 ** -8 * float(p.R.abs().max()) + 2.0 ** -9
    db = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="relu", want_dbias=True)[3]
    for i in range(2):
        t = slice(int(p.off[i]), int(p.off[i + 1]))
        ref = (p.dY[t].double() * (want[t] > 0)).sum(0)
        assert float((db[i].double() - ref).abs().max()) <= 2.0 ** -22 * 8 * (t.stop - t.start)
    eng.close()


@gpu
@pytest.mark.parametrize("blocks", [1, 3])
def test_a_low_rank_part_that_two_parts_do_not_hold(blocks):
    """s x a = 1 + 2^-9 + 2^-20 has more bits than two bf16 parts; W takes the first two terms back, so Z is 2^-20 (or, in
    every other column, twice W's share past it: -2^-20), which only A itself shows."""
    K, N = 136, 768
    p = Problem("bf16", K, N, [5, 40], [30, 131], blocks=blocks, bias="none", residual=False, seed=70)
    p.X = torch.ones_like(p.X)
    p.W.zero_()
    p.W[:, 3] = -1
    p.W[:, 70] = -2.0 ** -9
    p.W[1::2, 9] = -2.0 ** -19
    p.scales = [1.0, 1.0]
    for i in range(2):
        r = p.ranks[i]
        p.A[i].zero_()
        p.B[i].zero_()
        for b in range(blocks):
            row = b * r + (r - 1)
            p.A[i][row, 5], p.A[i][row, 66], p.A[i][row, 130] = 1, 2.0 ** -9, 2.0 ** -20
        p.B[i][:, r - 1] = 1
    eng = p.engine()
    Y, _, Z = forward(p, eng)
    want = torch.full((N,), 2.0 ** -20, device="cuda")
    want[1::2] = -2.0 ** -20
    assert torch.equal(Z.float(), want.expand(p.T, N)) and torch.equal(Y.float(), want.clamp(min=0).expand(p.T, N))
    eng.close()


@gpu
def test_rows_of_zeros_and_special_values():
    """A row of zeros has the bias for Z, exactly; a NaN or an infinity stays in its row; nothing waits on them."""
    p = Problem("bf16", 2056, 520, [8, 3], [140, 5], bias="each", residual=False, seed=80)
    p.X[7] = 0
    p.bias[0][11] = 0
    clean = forward(p, p.engine())[2]
    assert torch.equal(clean[7], p.bias[0])
    p.X[9, 5] = float("nan")
    p.X[10, 5] = float("inf")
    p.X[11] *= 2.0 ** 100
    p.X[12] *= 2.0 ** -100
    Z = forward(p, p.engine())[2]
    rows = [t for t in range(p.T) if t not in (9, 10, 11, 12)]
    assert torch.equal(Z[rows], clean[rows])
    assert bool(Z[9].isnan().all()) and not bool(Z[10].isfinite().any()) and bool(Z[11].isfinite().all())


@gpu
def test_captured_and_replayed():
    p = Problem("bf16", 4104, 520, [8, 3], [140, 5], bias="each", residual=False, seed=81)
    eng = p.engine()
    Y0, s0, Z0 = forward(p, eng)
    Y, Z, saved = torch.empty_like(Y0), torch.empty_like(Z0), torch.empty_like(s0)
    tab = eng.table(p.scales, p.A, p.B)
    ep = pl.make_epilogue("relu", bias=[b.data_ptr() for b in p.bias], Z=Z.data_ptr())
    assert pl.plora_epilogue_saved_bytes(eng.h, p.n, p.off, tab, ep) == saved.numel()
    pl.plora_capture_reserve(eng.h, 1)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        pl.plora_forward_epilogue(eng.h, p.X.data_ptr(), p.W.data_ptr(), Y.data_ptr(), p.n, p.off, tab, saved.data_ptr(), ep,
                                  s.cuda_stream)
    for _ in range(2):
        saved.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, Y0) and torch.equal(Z, Z0)
    p.X.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(Z, forward(p, eng)[2])
    del g
    pl.plora_capture_release(eng.h)
    eng.close()
