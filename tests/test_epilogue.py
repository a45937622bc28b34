"""The projection with bias, activation and residual (plora_forward_epilogue, plora_backward_epilogue,
PackedLoRA.forward_epilogue / backward_epilogue, packed_lora) against the formulas in float64.

Tolerances.  With U = 2^-8 (half a bf16 step) the library rounds H' = s X A, G = s dZ B^T, dZ, Z and the
results once each, so element by element, to first order, with |.| the products of the magnitudes,
    Z: U (|H'||B| + |Z|)      Y: U (1.13 |H'||B| + |Y|)      (1.13: the activations' largest slope)
    G: 2 U |s dZ||B|          dX: U (|dZ||W| + 2 |s dZ||B||A| + |dX|)
    dA: 2 U |X|^T |s dZ||B|   dB: 2 U |dZ|^T |H'|
where |dZ| stands for |dZ| + 2^-13 |dY| with an activation (act' cancels where it crosses zero: its fp32
form is then off by up to 2^-21 = 2^-13 U absolutely) and |H'| for |H'| + (K + 8) 2^-16 s |X||A| (the fp32
sum that H' rounds, off by (K + 8) 2^-24 = (K + 8) 2^-16 U of its magnitudes).  The other fp32 add K 2^-24 of the same magnitudes, less than U / 16 for the K here.  On an fp32 handle U is
(K + 8) 2^-24 with K the longest sum.  db sums fp32 values from the unrounded dZ.  Where the sums are long
the errors average out, and the bf16 results of a whole call are also held to the 2-norm of their
roundings: a rounding moves a tensor by at most U of itself, so Y and Z (H', Y) 2 U, dX (dZ, G, dX) 3 U, all
dA together (dZ, G) 2 U, all dB (dZ, H') 2 U."""
import ctypes
import math

import numpy as np
import pytest

import packed_lora_fine_b200 as pl

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
U = 2.0 ** -8
ACTS = list(pl.ACTIVATIONS)


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


# ------------------------------------------------------------------ the formulas in float64
def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


class Problem:
    """Random inputs of one call; off bounds the adapters' rows, extra rows follow the last one."""

    def __init__(self, dtype, d_in, d_out, ranks, counts, blocks=1, bias="each", residual=True, extra=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype, self.d_in, self.d_out, self.ranks, self.n = dtype, d_in, d_out, ranks, len(ranks)
        self.blocks = blocks
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)
        self.T, rows = int(self.off[-1]), int(self.off[-1]) + extra

        def rand(*s, std=1.0):
            return (torch.randn(s, generator=g) * std).to(dt).cuda()
        self.X, self.dY, self.W = rand(rows, d_in), rand(rows, d_out), rand(d_out, d_in, std=d_in ** -0.5)
        self.A = [rand(blocks * r, d_in, std=d_in ** -0.5) for r in ranks]
        self.B = [rand(d_out, r, std=0.3) for r in ranks]
        self.scales = [0.5 + 0.25 * i for i in range(self.n)]
        self.bias = {"none": None, "shared": rand(d_out), "each": [rand(d_out) for _ in ranks],
                     "some": [rand(d_out) if i % 2 else None for i in range(self.n)]}[bias]
        self.R = rand(rows, d_out) if residual else None

    def engine(self, **kw):
        return pl.PackedLoRA(self.d_in, self.d_out, self.dtype, max_adapters=max(1, self.n), max_rank=max(self.ranks),
                             max_tokens=max(1, self.T),
                             out_blocks=[self.d_out // self.blocks] * self.blocks if self.blocks > 1 else None, **kw)

    def biases(self):
        return self.bias if isinstance(self.bias, list) else [self.bias] * self.n

    def z64(self, X, A, B, bias):
        z = X[:self.T] @ self.W.double().T
        parts, w = [], self.d_out // self.blocks
        for i in range(self.n):
            r, x = self.ranks[i], X[self.off[i]:self.off[i + 1]]
            low = [(x @ A[i][b * r:(b + 1) * r].T) @ B[i][b * w:(b + 1) * w].T for b in range(self.blocks)]
            parts.append(self.scales[i] * torch.cat(low, 1) + (0.0 if bias[i] is None else bias[i]))
        return z + torch.cat(parts)

    def reference(self, act, Z=None):
        """Y, Z and every gradient in float64 (the activation's derivative taken at Z if it is given)."""
        leaf = lambda t: None if t is None else t.detach().double().requires_grad_(True)
        X, A, B, b = leaf(self.X), [leaf(a) for a in self.A], [leaf(x) for x in self.B], [leaf(x) for x in self.biases()]
        z = self.z64(X, A, B, b)
        y = act64(z, act) + (0.0 if self.R is None else self.R[:self.T].double())
        dY = self.dY[:self.T].double()
        if Z is not None:
            q = Z[:self.T].double().requires_grad_(True)
            dZ, = torch.autograd.grad(act64(q, act), q, dY)
        else:
            dZ, = torch.autograd.grad(act64(z, act), z, dY, retain_graph=True)
        wanted = [X, *A, *B, *[x for x in b if x is not None]]
        g = list(torch.autograd.grad(z, wanted, dZ))
        k = 1 + 2 * self.n
        db = iter(g[k:])
        return dict(Y=y.detach(), Z=z.detach(), dX=g[0][:self.T], dA=g[1:1 + self.n], dB=g[1 + self.n:k],
                    db=[None if x is None else next(db) for x in b])


def rel(got, ref):
    got, ref = got.detach().double(), ref.detach().double()
    assert got.shape == ref.shape
    if ref.numel() == 0:
        return 0.0
    d, n = float((got - ref).norm()), float(ref.norm())
    return d / n if n else (0.0 if d == 0 else math.inf)


def bounds(p, ref, Z, act, u):
    """The elementwise bounds of the module's docstring (u: U with its share for the fp32 sums)."""
    w = p.d_out // p.blocks
    q = (ref["Z"] if Z is None else Z[:p.T].double()).requires_grad_(True)
    dZ = torch.autograd.grad(act64(q, act), q, p.dY[:p.T].double())[0].abs()
    if act != "none":
        dZ = dZ + 2.0 ** -13 * p.dY[:p.T].double().abs()
    X, W = p.X[:p.T].double().abs(), p.W.double().abs()
    low, gx, dA, dB = [], [], [], []
    for i in range(p.n):
        t, r, s = slice(p.off[i], p.off[i + 1]), p.ranks[i], p.scales[i]
        A, B = p.A[i].double().abs(), p.B[i].double().abs()
        H = [s * ((p.X[t].double() @ p.A[i][b * r:(b + 1) * r].double().T).abs()
                  + (p.d_in + 8) * 2.0 ** -16 * X[t] @ A[b * r:(b + 1) * r].T) for b in range(p.blocks)]
        G = [s * dZ[t, b * w:(b + 1) * w] @ B[b * w:(b + 1) * w] for b in range(p.blocks)]
        low.append(torch.cat([H[b] @ B[b * w:(b + 1) * w].T for b in range(p.blocks)], 1))
        gx.append(sum(G[b] @ A[b * r:(b + 1) * r] for b in range(p.blocks)))
        dA.append(2 * u * torch.cat([G[b].T @ X[t] for b in range(p.blocks)]))
        dB.append(2 * u * torch.cat([dZ[t, b * w:(b + 1) * w].T @ H[b] for b in range(p.blocks)]))
    low, gx, res = torch.cat(low), torch.cat(gx), 0.0 if p.R is None else p.R[:p.T].double().abs()
    # the fp32 base sums' share enters with the products' magnitudes
    base = (u - U if p.dtype == "bf16" else u) * (X @ W.T)
    return dict(Z=u * (low + ref["Z"].abs()) + base, Y=u * (1.13 * low + ref["Y"].abs() + res) + 1.13 * base,
                dX=u * (dZ @ W + 2 * gx + ref["dX"].abs()), dA=dA, dB=dB)


def inside(got, ref, bound):
    return bool(((got.double() - ref).abs() <= bound + 1e-30).all())


def check(p, act, eng=None, averaged=True):
    own = eng is None
    eng = eng or p.engine()
    f32 = p.dtype == "fp32"
    Y, saved, Z = eng.forward_epilogue(p.X[:p.T], p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act,
                                       residual=None if p.R is None else p.R[:p.T])
    want = [b is not None for b in p.biases()]
    dX, dA, dB, db = eng.backward_epilogue(p.X[:p.T], p.W, p.dY[:p.T], p.off, p.scales, p.A, p.B, saved, Z=Z,
                                           activation=act, want_dbias=want)
    torch.cuda.synchronize()
    assert pl.plora_check(eng.h, 0) == pl.PLORA_OK
    ref = p.reference(act, Z)
    longest = max(p.d_in, p.d_out, p.T)
    b = bounds(p, ref, Z, act, (longest + 8) * 2.0 ** -24 + (0.0 if f32 else U))
    assert (Z is None) == (act == "none")
    assert inside(Y, ref["Y"], b["Y"]) and (Z is None or inside(Z, ref["Z"], b["Z"]))
    assert inside(dX, ref["dX"], b["dX"])
    for i in range(p.n):
        assert inside(dA[i], ref["dA"][i], b["dA"][i]), i
        assert inside(dB[i], ref["dB"][i], b["dB"][i]), i
        if ref["db"][i] is not None:
            rows = int(p.off[i + 1] - p.off[i])
            # the sums may cancel: bound the error by the sum of magnitudes, rows * max|dZ| <= 8 rows here
            assert float((db[i].double() - ref["db"][i]).abs().max()) <= 2.0 ** -22 * max(1, rows) * 8, i
    if averaged and not f32:
        flat = lambda v: torch.cat([x.reshape(-1) for x in v])
        assert rel(Y, ref["Y"]) <= 2 * U and (Z is None or rel(Z, ref["Z"]) <= 2 * U)
        assert rel(dX, ref["dX"]) <= 3 * U
        assert rel(flat(dA), flat(ref["dA"])) <= 2 * U and rel(flat(dB), flat(ref["dB"])) <= 2 * U
    if own:
        eng.close()


SHAPES = [
    # d_in, d_out, ranks, counts: one token; an odd last column block; an empty adapter; straddled tiles
    (64, 8, [1], [1]),
    (136, 264, [4, 17, 1], [1, 300, 7]),
    (264, 392, [16, 8, 3, 64], [130, 0, 257, 60]),
    (72, 1032, [2] * 20, [5, 1, 0, 9, 3] * 4),
    (1000, 520, [128, 200], [513, 255]),
]


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("k", range(len(SHAPES)))
def test_bf16_matches_the_formulas(k, act):
    d_in, d_out, ranks, counts = SHAPES[k]
    check(Problem("bf16", d_in, d_out, ranks, counts, bias=("each", "some", "shared")[k % 3], residual=k % 2 == 0, seed=k), act,
          averaged=k > 0)


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_fp32_matches_the_formulas(act):
    check(Problem("fp32", 72, 264, [4, 17, 1], [1, 140, 0], bias="some", seed=3), act)


@gpu
@pytest.mark.parametrize("ranks, counts", [([1], [136]), ([17, 80, 2], [100, 0, 36]), ([3] * 17, [8] * 17)])
def test_relu_sees_what_a_rounded_h_would_lose(ranks, counts):
    """relu's derivative jumps with Z's sign, so its training forward takes H' in two bf16 parts.  Here X is the
    identity, H' = 1.5 A (at most 10 bits), B = 1 and W the negative of H' rounded to 8 bits, so that Z is what that
    rounding left, without a rounding of its own: it is 0 with H' in one part."""
    p = Problem("bf16", 136, 264, ranks, counts, bias="none", residual=False, seed=40)
    p.scales = [1.5] * p.n
    p.X[:] = torch.eye(136, device="cuda")
    h = torch.empty(136, device="cuda")
    for i in range(p.n):
        p.A[i][1:] = 0
        p.B[i][:] = 0
        p.B[i][:, 0] = 1
        h[int(p.off[i]):int(p.off[i + 1])] = 1.5 * p.A[i][0, int(p.off[i]):int(p.off[i + 1])].float()
    p.W[:] = -h.bfloat16()
    left = h - h.bfloat16().float()
    assert int((left != 0).sum()) > 40
    eng = p.engine()
    Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, activation="relu")
    want = left[:, None].expand(136, 264)
    assert torch.equal(Z.float(), want) and torch.equal(Y.float(), want.clamp(min=0))
    dX = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="relu")[0]
    # the derivative at 0 is 0, and W and the factors cancel in dX: the elementwise bound of the module's docstring
    dZ = p.dY.double() * (want > 0)
    for i in range(p.n):
        t, B, A, W = slice(int(p.off[i]), int(p.off[i + 1])), p.B[i].double(), p.A[i].double(), p.W.double()
        ref = dZ[t] @ W + 1.5 * (dZ[t] @ B) @ A
        bound = dZ[t].abs() @ W.abs() + 2 * 1.5 * (dZ[t].abs() @ B.abs()) @ A.abs() + ref.abs()
        assert inside(dX[t], ref, (U + (264 + 8) * 2.0 ** -24) * bound)
    # the low parts need room in `saved`, and none without Z
    tab, ep = eng.table(p.scales, p.A, p.B), pl.make_epilogue("relu", Z=Z.data_ptr())
    size = lambda e: pl.plora_epilogue_saved_bytes(eng.h, p.n, p.off, tab, e)
    plain = eng.saved_bytes(p.off, tab)
    assert size(ep) > plain == size(pl.make_epilogue("relu")) == size(pl.make_epilogue("silu", Z=Z.data_ptr()))
    eng.close()


@gpu
@pytest.mark.parametrize("act, bias, residual", [("none", "none", True), ("none", "each", False), ("silu", "none", False)])
def test_each_part_alone(act, bias, residual):
    check(Problem("bf16", 136, 328, [8, 24], [200, 77], bias=bias, residual=residual, seed=5), act)


@gpu
def test_output_blocks():
    check(Problem("bf16", 200, 768, [8, 24], [150, 70], blocks=3, seed=6), "gelu")


@gpu
def test_an_empty_epilogue_is_the_plain_call_bit_for_bit():
    p = Problem("bf16", 264, 392, [16, 3], [130, 257], bias="none", residual=False, seed=7)
    eng = p.engine()
    Y0, s0 = eng.forward(p.X, p.W, p.off, p.scales, p.A, p.B)
    g0 = eng.backward(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, s0)
    Y1, s1, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B)
    g1 = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, s1)
    torch.cuda.synchronize()
    assert Z is None and g1[3] is None
    assert torch.equal(Y0, Y1) and torch.equal(g0[0], g1[0])
    for a, b in zip(g0[1] + g0[2], g1[1] + g1[2]):
        assert torch.equal(a, b)
    eng.close()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_residual_in_place_and_rows_behind_the_last_adapter(dtype):
    p = Problem(dtype, 72, 328, [8, 5], [190, 101], extra=13, seed=8)
    eng = p.engine()
    Y, _, _ = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="silu", residual=p.R)
    Yi = p.R.clone()
    if dtype == "fp32":     # the fp32 path builds Z in Y, so the residual has to be another buffer
        with pytest.raises(pl.PloraError) as err:
            eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, residual=Yi, Y=Yi)
        assert err.value.status == pl.PLORA_ERR_INVALID_ARG
        eng.close()
        return
    Y2, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="silu",
                                        residual=Yi, Y=Yi)
    torch.cuda.synchronize()
    assert Y2 is Yi and torch.equal(Yi[:p.T], Y[:p.T])
    assert torch.equal(Yi[p.T:], p.R[p.T:])          # rows behind the last adapter are left as they were
    eng.close()


@gpu
def test_special_values_stay_with_their_rows_and_adapters():
    p = Problem("bf16", 72, 264, [8, 5, 2], [140, 130, 33], seed=9)
    eng = p.engine()
    run = lambda: eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="gelu", residual=p.R)[0]
    clean = run()
    p.bias[1][3] = math.inf
    p.bias[1][9] = math.nan
    p.R[5, 7] = math.nan
    p.R[6, 7] = -math.inf
    Y = run()
    torch.cuda.synchronize()
    rows = slice(int(p.off[1]), int(p.off[2]))
    assert torch.isposinf(Y[rows, 3]).all() and torch.isnan(Y[rows, 9]).all()
    assert torch.isnan(Y[5, 7]) and torch.isneginf(Y[6, 7])
    Y[rows, 3], Y[rows, 9], Y[5, 7], Y[6, 7] = clean[rows, 3], clean[rows, 9], clean[5, 7], clean[6, 7]
    assert torch.equal(Y, clean)
    eng.close()


@gpu
def test_activations_at_their_borders():
    # X W + low rank is zero, so Z is the bias: large, tiny, signed zeros and infinities
    vals = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3.0, -3.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4, 1e30, math.inf, math.nan, 0.5])
    for act in ACTS:
        p = Problem("fp32", 16, 16, [2], [3], residual=False, seed=10)
        p.X.zero_()
        p.bias = [vals.cuda()]
        eng = p.engine()
        Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act)
        ref = act64(vals.double(), act)
        got = Y[0].double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), act
        ok = torch.isfinite(ref)
        assert torch.equal(got[~ok & ~torch.isnan(ref)], ref[~ok & ~torch.isnan(ref)]), act
        # the functions' fp32 forms cancel near 0 and -inf (1 + erf, 1 + tanh): absolute 2^-22 of |z|
        assert ((got - ref).abs()[ok] <= 2.0 ** -22 * vals.double().abs()[ok]).all(), act
        if act != "none":
            ones = torch.ones_like(Y)
            dX, dA, dB, db = eng.backward_epilogue(p.X, p.W, ones, p.off, p.scales, p.A, p.B, saved, Z=Z, activation=act,
                                                   want_dbias=True)
            q = vals.double().clone().requires_grad_(True)
            fin = torch.isfinite(vals) & (vals.abs() <= 1e4)
            g, = torch.autograd.grad(act64(q[fin], act).sum(), q)
            if act == "relu":
                g[vals == 0] = 0.0          # the documented derivative at 0
            assert ((db[0].double().cpu() / 3 - g).abs()[fin] <= 2.0 ** -20).all(), act
        eng.close()


@gpu
@pytest.mark.parametrize("act", ACTS)
def test_bf16_activations_at_their_borders(act):
    # as above: rounded once, the functions within 2^-21 of |z| and the derivatives within 2^-19 absolute.
    # The fast exponential is off by (2 + 1.16 |x|) ulps and the fast division by 2, of terms z^k exp(-|z|) and
    # z^k exp(-z^2 / 2) whose (1 + |x|)-fold stays below 4; erf's polynomial by 1.5e-7
    vals = torch.cat([torch.linspace(-12, 12, 113), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30.0, -30.0, 60.0, -60.0, 100.0,
                      -100.0, 1e4, -1e4, 1e30, -1e30, math.inf, math.nan])]).bfloat16()
    n = (vals.numel() + 7) // 8 * 8
    vals = torch.cat([vals, torch.zeros(n - vals.numel(), dtype=torch.bfloat16)])
    p = Problem("bf16", 16, n, [2], [3], residual=False, seed=10)
    p.X.zero_()
    p.bias = [vals.cuda()]
    eng = p.engine()
    Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act)
    ref = act64(vals.double(), act)
    got = Y[0].double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    ok = torch.isfinite(ref)
    assert torch.equal(got[~ok & ~torch.isnan(ref)], ref[~ok & ~torch.isnan(ref)])
    assert ((got - ref).abs()[ok] <= U * ref.abs()[ok] + 2.0 ** -21 * vals.double().abs()[ok].clamp(max=100.0)).all()
    if act != "none":
        db = eng.backward_epilogue(p.X, p.W, torch.ones_like(Y), p.off, p.scales, p.A, p.B, saved, Z=Z, activation=act,
                                   want_dbias=True)[3]
        q = vals.double().clone().requires_grad_(True)
        fin = torch.isfinite(vals) & (vals.abs() <= 1e4)
        g, = torch.autograd.grad(act64(q[fin], act).sum(), q)
        if act == "relu":
            g[vals == 0] = 0.0
        got = db[0].double().cpu() / 3
        assert ((got - g).abs()[fin] <= 2.0 ** -19).all()
        far = vals.abs() == torch.tensor(1e30).bfloat16()
        assert torch.equal(got[far], (vals[far] > 0).double())
    eng.close()


@gpu
def test_gradients_against_differences():
    p = Problem("fp32", 24, 40, [3, 2], [6, 5], seed=11)
    eng = p.engine()

    def loss(act):
        Y, _, _ = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act, residual=p.R)
        return float((Y.double() * p.dY.double()).sum())
    for act in ("none", "gelu", "gelu_tanh", "silu"):
        _, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act, residual=p.R)
        dX, dA, dB, db = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation=act,
                                               want_dbias=True)
        for t, g, at in ((p.X, dX, (3, 7)), (p.A[1], dA[1], (1, 5)), (p.B[0], dB[0], (9, 2)), (p.bias[1], db[1], (4,)),
                         (p.R, p.dY, (10, 3))):
            old, h = float(t[at]), 2.0 ** -6
            t[at] = old + h
            up = loss(act)
            t[at] = old - h
            down = loss(act)
            t[at] = old
            # h^2/6 of the third derivatives (sums of up to 40 terms of order one) and the loss's rounding / h
            assert abs((up - down) / (2 * h) - float(g[at])) <= 40 * h * h / 6 + 440 * 2.0 ** -22 / h, (act, at)
    eng.close()


@gpu
def test_no_tokens_and_only_empty_adapters():
    p = Problem("bf16", 64, 72, [4, 2], [0, 0], seed=12)
    eng = p.engine()
    Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="silu", residual=p.R)
    dX, dA, dB, db = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="silu",
                                           want_dbias=True)
    torch.cuda.synchronize()
    assert Y.shape == (0, 72)
    assert not any(bool(t.any()) for t in dA + dB + db)
    eng.close()


@gpu
def test_packed_equals_alone_and_repeats_bit_for_bit():
    p = Problem("bf16", 136, 328, [8, 24, 3], [200, 77, 130], seed=13)
    eng = p.engine()

    def run(i=None):
        s = slice(0, p.T) if i is None else slice(int(p.off[i]), int(p.off[i + 1]))
        k = list(range(p.n)) if i is None else [i]
        off = p.off if i is None else np.array([0, s.stop - s.start])
        pick = lambda v: [v[j] for j in k]
        X, dY, R = p.X[s].contiguous(), p.dY[s].contiguous(), p.R[s].contiguous()
        Y, saved, Z = eng.forward_epilogue(X, p.W, off, pick(p.scales), pick(p.A), pick(p.B), bias=pick(p.bias),
                                           activation="silu", residual=R)
        out = eng.backward_epilogue(X, p.W, dY, off, pick(p.scales), pick(p.A), pick(p.B), saved, Z=Z, activation="silu",
                                    want_dbias=True)
        return [Y, Z, out[0]], out[3]
    a, da = run()
    b, db = run()
    for x, y in zip(a + da, b + db):
        assert torch.equal(x, y)
    for i in range(p.n):
        c, dc = run(i)
        rows = slice(int(p.off[i]), int(p.off[i + 1]))
        assert all(torch.equal(x[rows], y) for x, y in zip(a, c)) and torch.equal(da[i], dc[0])
    eng.close()


@gpu
def test_capture_replays_and_runs_on_another_stream():
    p = Problem("bf16", 136, 328, [8, 24], [200, 77], seed=14)
    eng = p.engine()
    tf = eng.table(p.scales, p.A, p.B)
    new = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")
    dA, dB = [new(*a.shape, dt=torch.float32) for a in p.A], [new(*b.shape, dt=torch.float32) for b in p.B]
    tb = eng.table(p.scales, p.A, p.B, dA, dB)
    Y, Z, dX = new(p.T, p.d_out), new(p.T, p.d_out), new(p.T, p.d_in)
    db = [new(p.d_out, dt=torch.float32) for _ in range(2)]
    saved = new(eng.saved_bytes(p.off, tf), dt=torch.uint8)
    ef = pl.make_epilogue("gelu", bias=[b.data_ptr() for b in p.bias], residual=p.R.data_ptr(), Z=Z.data_ptr())
    eb = pl.make_epilogue("gelu", dbias=[b.data_ptr() for b in db], Z=Z.data_ptr())
    work = new(pl.plora_epilogue_work_bytes(eng.h, 2, p.off, eb), dt=torch.uint8)
    eb.work = work.data_ptr()

    def step(st):
        pl.plora_forward_epilogue(eng.h, p.X.data_ptr(), p.W.data_ptr(), Y.data_ptr(), 2, p.off, tf, saved.data_ptr(), ef, st)
        pl.plora_backward_epilogue(eng.h, p.X.data_ptr(), p.W.data_ptr(), p.dY.data_ptr(), dX.data_ptr(), 2, p.off, tb,
                                   saved.data_ptr(), eb, st)
    outs = [Y, Z, dX, *dA, *dB, *db]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(s.cuda_stream)
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    pl.plora_capture_reserve(eng.h, 4)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(s.cuda_stream)
        graphs.append(g)
    for g in graphs + graphs:
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    del graphs, g
    pl.plora_capture_release(eng.h)
    eng.close()


# ------------------------------------------------------------------ inference, a few tokens
def infer(p, eng, act, residual=True, **kw):
    Y, saved, Z = eng.forward_epilogue(p.X[:p.T], p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation=act, want_Z=False,
                                       residual=p.R[:p.T] if residual and p.R is not None else None, **kw)
    assert saved is None and Z is None
    return Y


FEW = [
    # d_in, d_out, ranks, counts, output blocks: one token; eight; nine; ranks that are no multiple of 8, adapters
    # without tokens, columns past a block's 16; K ending inside a slice; the most tokens; one more than that
    (64, 8, [1], [1], 1),
    (136, 264, [4, 17, 64], [1, 0, 7], 1),
    (1000, 520, [128, 200], [5, 4], 1),
    (200, 768, [8, 24, 3], [2, 0, 14], 3),
    (72, 1032, [2] * 20, [1, 2] * 10, 1),
    (4104, 136, [16, 256], [1, 31], 1),
    (136, 264, [4, 17], [1, 32], 1),
]


@gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("k", range(len(FEW)))
def test_few_tokens_match_the_formulas(k, act):
    d_in, d_out, ranks, counts, blocks = FEW[k]
    p = Problem("bf16", d_in, d_out, ranks, counts, blocks=blocks, bias=("each", "some", "shared")[k % 3], residual=k % 2 == 0,
                seed=20 + k)
    eng = p.engine()
    Y = infer(p, eng, act)
    assert pl.plora_check(eng.h, 0) == pl.PLORA_OK
    ref = p.reference(act)
    b = bounds(p, ref, None, act, (max(d_in, max(ranks)) + 8) * 2.0 ** -24 + U)
    assert inside(Y, ref["Y"], b["Y"])
    assert torch.equal(Y, infer(p, eng, act))
    eng.close()


@gpu
def test_few_tokens_alone_in_place_and_captured():
    p = Problem("bf16", 264, 392, [16, 3, 40], [9, 1, 15], extra=5, seed=30)
    eng = p.engine()
    Y = infer(p, eng, "silu")
    for i in range(p.n):               # an adapter's rows alone, which take another number of tokens at a time
        s = slice(int(p.off[i]), int(p.off[i + 1]))
        y, _, _ = eng.forward_epilogue(p.X[s].contiguous(), p.W, np.array([0, s.stop - s.start]), p.scales[i:i + 1],
                                       p.A[i:i + 1], p.B[i:i + 1], bias=p.bias[i:i + 1], activation="silu",
                                       residual=p.R[s].contiguous(), want_Z=False)
        assert torch.equal(y, Y[s])
    R = p.R.clone()                    # the residual is Y itself; rows behind the last adapter stay
    eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="silu", residual=R, Y=R, want_Z=False)
    assert torch.equal(R[:p.T], Y) and torch.equal(R[p.T:], p.R[p.T:])
    out, saved = torch.empty_like(Y), torch.empty(eng.saved_bytes(p.off, eng.table(p.scales, p.A, p.B)), dtype=torch.uint8,
                                                  device="cuda")
    bad = p.X.clone()                  # a token's NaN and infinity stay in its row
    bad[9] = math.nan
    bad[10, 3] = math.inf
    keep, p.X = p.X, bad
    got = infer(p, eng, "silu")
    p.X = keep
    rows = [t for t in range(p.T) if t not in (9, 10)]
    assert torch.equal(got[rows], Y[rows]) and bool(got[9].isnan().all()) and not bool(got[10].isfinite().any())
    side = torch.cuda.Stream()         # another stream than the current one, behind work of its own
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = p.X * 2
    y, _, _ = eng.forward_epilogue(x, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="silu", residual=p.R, want_Z=False,
                                   stream=side)
    keep, p.X = p.X, p.X * 2
    torch.cuda.synchronize()
    assert torch.equal(y[:p.T], infer(p, eng, "silu"))
    p.X = keep
    graph = torch.cuda.CUDAGraph()     # no schedule slot is reserved
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        infer(p, eng, "silu", Y=out, saved=saved)
        infer(p, eng, "silu", Y=out, saved=saved)
    p.X.neg_()
    graph.replay()
    want = infer(p, eng, "silu")
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not torch.equal(out, Y)
    del graph
    eng.close()


@gpu
def test_inference_keeps_nothing():
    p = Problem("bf16", 72, 264, [8, 5], [40, 30], seed=31)      # more than a few tokens: the training kernels
    eng = p.engine()
    Y, _, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="gelu", residual=p.R)
    assert torch.equal(infer(p, eng, "gelu"), Y)
    tab, saved = eng.table(p.scales, p.A, p.B), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    ep = pl.make_epilogue("gelu", Z=Z.data_ptr(), inference=True)
    assert pl.plora_forward_epilogue(eng.h, p.X.data_ptr(), p.W.data_ptr(), Y.data_ptr(), 2, p.off, tab, saved.data_ptr(), ep, 0,
                                     check=False) == pl.PLORA_ERR_INVALID_ARG
    eng.close()
    p = Problem("fp32", 72, 264, [8, 5], [4, 3], seed=32)
    eng = p.engine()
    Y, _, _ = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="gelu", residual=p.R)
    assert torch.equal(infer(p, eng, "gelu"), Y)
    eng.close()


# ------------------------------------------------------------------ autograd
@gpu
@pytest.mark.parametrize("shared", [False, True])
def test_autograd(shared):
    p = Problem("bf16", 136, 264, [4, 17, 2], [60, 130, 7], bias="shared" if shared else "each", seed=15)
    eng = p.engine()
    leaf = lambda t: t.requires_grad_(True)
    X = leaf(p.X.t().contiguous().t())                # not contiguous
    A, B = [leaf(a) for a in p.A], [leaf(b) for b in p.B]
    bias = leaf(p.bias) if shared else [leaf(b) for b in p.bias]
    R = leaf(p.R)
    Y = pl.packed_lora(eng, X, p.W, p.off, p.scales, A, B, bias=bias, activation="silu", residual=R)
    Y.backward(p.dY)
    ref = p.reference("silu")
    assert rel(Y, ref["Y"]) <= 2 * U
    assert torch.equal(R.grad, p.dY)
    # Z's own rounding moves act'(Z) by at most sup|z act''(z)| 2^-8 <= 2^-8 (silu): one more rounding
    assert rel(X.grad, ref["dX"]) <= 4 * U
    for i in range(3):
        assert rel(A[i].grad, ref["dA"][i]) <= 4 * U and rel(B[i].grad, ref["dB"][i]) <= 4 * U
    got = [bias.grad] if shared else [b.grad for b in bias]
    want = [sum(ref["db"])] if shared else ref["db"]
    for g, w in zip(got, want):
        assert g.dtype == torch.bfloat16 and rel(g, w) <= 2 * U
    eng.close()


@gpu
def test_autograd_asks_only_for_what_is_needed():
    p = Problem("bf16", 72, 72, [4], [9], seed=16)
    eng = p.engine()
    p.bias[0].requires_grad_(True)
    Y = pl.packed_lora(eng, p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="relu")
    g, = torch.autograd.grad(Y, p.bias, p.dY)
    assert rel(g, p.reference("relu")["db"][0]) > 0 and g.shape == (72,)
    eng.close()


# ------------------------------------------------------------------ refusals
def test_refusals_without_a_device():
    lib, out, ep = pl.load(), ctypes.c_size_t(7), pl.make_epilogue("gelu")
    a = ctypes.addressof
    assert lib.plora_epilogue_work_bytes(None, 0, None, a(ep), ctypes.byref(out)) == pl.PLORA_ERR_INVALID_ARG
    assert lib.plora_epilogue_saved_bytes(None, 0, None, None, a(ep), ctypes.byref(out)) == pl.PLORA_ERR_INVALID_ARG
    assert lib.plora_forward_epilogue(None, None, None, None, 0, None, None, None, a(ep), None) == pl.PLORA_ERR_INVALID_ARG
    assert lib.plora_backward_epilogue(None, None, None, None, None, 0, None, None, None, a(ep), None) == pl.PLORA_ERR_INVALID_ARG
    assert ctypes.sizeof(pl.plora_epilogue) == 48
    with pytest.raises(ValueError):
        pl.make_epilogue("swish")
    ep = pl.make_epilogue("silu", bias=[4096, None], Z=8192)
    assert ep.activation == pl.PLORA_ACT_SILU and ep.Z == 8192 and not ep.dbias and not ep.work
    assert list((ctypes.c_void_p * 2).from_address(ep.bias)) == [4096, None]


@gpu
def test_refusals_leave_the_outputs_alone():
    p = Problem("bf16", 72, 264, [8, 5], [40, 30], seed=17)
    eng = p.engine()
    tab = eng.table(p.scales, p.A, p.B)
    Y = torch.zeros((p.T, p.d_out), dtype=torch.bfloat16, device="cuda")
    Z = torch.zeros_like(Y)
    saved = torch.zeros(eng.saved_bytes(p.off, tab), dtype=torch.uint8, device="cuda")
    dA, dB = [torch.zeros(a.shape, device="cuda") for a in p.A], [torch.zeros(b.shape, device="cuda") for b in p.B]
    db = [torch.zeros(p.d_out, device="cuda") for _ in range(2)]
    tabg = eng.table(p.scales, p.A, p.B, dA, dB)
    work = torch.zeros(pl.plora_epilogue_work_bytes(eng.h, 2, p.off, pl.make_epilogue("gelu", dbias=[b.data_ptr() for b in db])),
                       dtype=torch.uint8, device="cuda")
    assert work.numel() == 70 * 264 * 2 + 256 - 70 * 264 * 2 % 256 + 2 * 264 * 4
    host = np.zeros(1 << 20, np.uint8)

    def fwd(ep, e=eng):
        return pl.plora_forward_epilogue(e.h, p.X.data_ptr(), p.W.data_ptr(), Y.data_ptr(), 2, p.off, tab, saved.data_ptr(),
                                         ep, 0, check=False)

    def bwd(ep):
        return pl.plora_backward_epilogue(eng.h, p.X.data_ptr(), p.W.data_ptr(), p.dY.data_ptr(), None, 2, p.off, tabg,
                                          saved.data_ptr(), ep, 0, check=False)
    bad = pl.PLORA_ERR_INVALID_ARG
    m = pl.make_epilogue
    b0 = p.bias[0].data_ptr()
    for ep in (m(5), m(-1), m("gelu", Z=Z.data_ptr() + 8), m(bias=[b0 + 2, None]), m(bias=[host.ctypes.data, None]),
               m(residual=host.ctypes.data), m("gelu", Z=host.ctypes.data),
               m("gelu", Z=Y.data_ptr()),                     # Z over Y
               m(residual=Y.data_ptr() + 16),                 # the residual overlaps Y without being it
               m("gelu", residual=Z.data_ptr(), Z=Z.data_ptr())):
        assert fwd(ep) == bad
    ep = m("gelu")
    ep.inference = 2
    assert fwd(ep) == bad and "inference" in pl.plora_last_error(eng.h)
    dbp = [b.data_ptr() for b in db]
    for ep in (m("gelu", work=work.data_ptr()),                                        # no Z
               m("gelu", Z=Z.data_ptr()),                                              # no work
               m("gelu", dbias=dbp, Z=Z.data_ptr(), work=work.data_ptr() + 16),
               m("gelu", Z=Z.data_ptr(), work=p.dY.data_ptr()),                        # work over dY
               m(dbias=[dbp[0], dbp[0]], work=work.data_ptr()),                        # one db for two adapters
               m(dbias=[dbp[0] + 4, None], work=work.data_ptr()), m(dbias=dbp)):
        assert bwd(ep) == bad
    torch.cuda.synchronize()
    for t in (Y, Z, saved, *dA, *dB, *db):
        assert not t.any()
    for kw in (dict(simt=True), dict(unfused=True), dict(base_pair=True)):
        e = p.engine(**kw)
        assert fwd(m("gelu", Z=Z.data_ptr()), e) == pl.PLORA_ERR_UNSUPPORTED
        e.close()
    args = (p.X, p.W, p.off, p.scales, p.A, p.B)
    for kw in (dict(bias=p.bias[:1]), dict(bias=p.bias[0][:8]), dict(residual=p.R[:, :8]), dict(residual=p.R.float()),
               dict(activation="swish"), dict(residual=p.R.t().contiguous().t())):
        with pytest.raises(ValueError):
            eng.forward_epilogue(*args, **kw)
    eng.close()
