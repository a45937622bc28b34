"""The packed Muon step (plora_muon_step) against its formula in float64.

Tolerances.  m is one fused multiply-add, 2^-24 relative.  O = Q X_0 is formed in fp32 from Q (rounded from
64 bits) and X_0: with s products per element its 2-norm error is within s 2^-24 |Q|_F |X_0|_2 <=
s 2^-24 sqrt(s) 3.4445^n; the tests' spectra keep |Q X_0| of order sqrt(s), and a bound of
1e-6 + 2^-24 * 3.4445^n = 3e-5 (n = 5) relative to |O|_F covers a sum of s random roundings of entries of Q
that its largest directions do not need.  p = p0 (1 - lr wd) - lr k O adds two roundings."""
import ctypes
import math

import numpy as np
import pytest

import packed_lora_fine_b200 as pl

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
A_, B_, C_ = pl.MUON_COEFFS
O_TOL = 3e-5


@pytest.fixture(scope="module", autouse=True)
def built():
    from packed_lora_fine_b200 import build as plbuild
    plbuild.build()


def orth64(u, eps=1e-7, steps=5, coeffs=pl.MUON_COEFFS):
    a, b, c = coeffs
    tall = u.shape[0] > u.shape[1]
    x = (u.T if tall else u).double()
    x = x / (torch.linalg.matrix_norm(x) + eps)
    for _ in range(steps):
        q = x @ x.T
        x = a * x + (b * q + c * q @ q) @ x
    return x.T if tall else x


def shape_factor(rule, rows, cols):
    return {"none": 1.0, "rows": math.sqrt(max(1.0, rows / cols)), "rms": 0.2 * math.sqrt(max(rows, cols))}[rule]


class Job:
    """Adapters' factors, gradients and state; spectrum shapes every matrix's singular values."""

    def __init__(self, dtype, d_in, d_out, ranks, blocks=1, spectrum="noise", seed=0, hp=None):
        g = torch.Generator().manual_seed(seed)
        self.n, self.dtype, self.blocks, self.d_in, self.d_out, self.ranks = len(ranks), dtype, blocks, d_in, d_out, ranks
        self.hp = hp or [dict(lr=0.02, weight_decay=0.01)] * self.n

        def mat(rows, cols, scale):
            x = torch.randn((rows, cols), generator=g, dtype=torch.float64)
            s = min(rows, cols)
            i = torch.arange(1, s + 1, dtype=torch.float64)
            w = {"noise": None, "power": 1 / i, "low rank": (i <= max(1, s // 4)).double(), "one": (i == 1).double()}[spectrum]
            if w is not None:
                q = torch.linalg.qr(torch.randn((s, s), generator=g, dtype=torch.float64))[0]
                x = (q * w) @ x if rows <= cols else x @ (q * w).T
            return (x * scale).float()

        def stack(side, r, scale):
            if side == 0:
                return torch.cat([mat(r, d_in, scale) for _ in range(blocks)]).cuda()
            return torch.cat([mat(d_out // blocks, r, scale) for _ in range(blocks)]).cuda()
        self.g = [[stack(s, r, 1e-3) for r in ranks] for s in (0, 1)]
        # the momentum in the gradient's directions, so that the spectrum is u's as well
        self.m = [[x * 5.0 for x in v] for v in self.g]
        self.p = [[(torch.randn(x.shape, generator=g) * 0.02).cuda() for x in v] for v in self.g]
        self.out = [[x.to(torch.bfloat16) for x in v] for v in self.p] if dtype == "bf16" else None

    def matrices(self, side, i):
        """(slice of rows) of every matrix of adapter i's A (side 0) or B (side 1)."""
        h = self.ranks[i] if side == 0 else self.d_out // self.blocks
        return [slice(b * h, (b + 1) * h) for b in range(self.blocks)]

    def engine(self):
        return pl.PackedLoRA(self.d_in, self.d_out, self.dtype, max_adapters=self.n, max_rank=max(self.ranks), max_tokens=16,
                             out_blocks=[self.d_out // self.blocks] * self.blocks if self.blocks > 1 else None)

    def args(self, eng):
        ptr = lambda v: [x.data_ptr() for x in v]
        lay = self.out or self.p
        tab = pl.make_table(self.ranks, [1.0] * self.n, ptr(lay[0]), ptr(lay[1]), ptr(self.g[0]), ptr(self.g[1]))
        bf = self.dtype == "bf16"
        st = pl.make_muon_states(self.hp, ptr(self.p[0]) if bf else None, ptr(self.p[1]) if bf else None, ptr(self.m[0]),
                                 ptr(self.m[1]))
        work = torch.full((pl.plora_muon_work_bytes(eng.h, self.n, tab),), 255, dtype=torch.uint8, device="cuda")
        return tab, st, work

    def step(self, eng, times=1):
        tab, st, work = self.args(eng)
        for _ in range(times):
            pl.plora_muon_step(eng.h, self.n, tab, st, work.data_ptr(), torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert pl.plora_check(eng.h, 0) == pl.PLORA_OK

    def tensors(self):
        return sum(self.p + self.m + (self.out or []), [])


def check(job, tol=O_TOL, eng=None):
    g = [[x.double() for x in v] for v in job.g]
    m0, p0 = [[x.double() for x in v] for v in job.m], [[x.double() for x in v] for v in job.p]
    own = eng or job.engine()
    job.step(own)
    for side in (0, 1):
        for i in range(job.n):
            hp = job.hp[i]
            mu, nest = hp.get("momentum", 0.95), hp.get("nesterov", True)
            m = mu * m0[side][i] + g[side][i]
            # (the hyper-parameters reach the kernel as fp32)
            assert float((job.m[side][i].double() - m).norm()) <= 2.0 ** -22 * float(m.norm()), (side, i)
            u = g[side][i] + mu * m if nest else m
            for rows in job.matrices(side, i):
                o = orth64(u[rows], hp.get("eps", 1e-7), hp.get("ns_steps", 5), hp.get("coeffs", pl.MUON_COEFFS))
                k = hp["lr"] * shape_factor(hp.get("scale", "rows"), *o.shape)
                want = p0[side][i][rows] * (1 - hp["lr"] * hp.get("weight_decay", 0.0)) - k * o
                err = float((job.p[side][i][rows].double() - want).norm())
                assert err <= k * tol * float(o.norm()) + 2.0 ** -22 * float(want.norm()), (side, i, err / max(1e-300, k * float(o.norm())))
            if job.out:
                assert torch.equal(job.out[side][i], job.p[side][i].to(torch.bfloat16))
    if eng is None:
        own.close()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d_in, d_out, ranks", [
    (264, 392, [1, 16, 64, 3]),          # odd ranks, one row
    (8, 16, [3, 8, 13, 40]),             # ranks above both sizes: the short side is d_in or d_out
    (2056, 1032, [17, 128]),             # more than one Gram chunk, a ragged one
    (520, 264, [129, 200, 256]),         # the largest ranks
    (16384, 8, [128, 128, 100, 17]),     # matrices of one tile between long ones, in the same block's run
])
def test_matches_the_formula(dtype, d_in, d_out, ranks):
    check(Job(dtype, d_in, d_out, ranks, seed=len(ranks) + d_in))


@gpu
@pytest.mark.parametrize("spectrum", ["power", "low rank", "one"])
def test_spectra_that_a_gram_matrix_squares(spectrum):
    # one direction alone: Q is 3.4445^5 on every other direction, and its fp32 rounding enters in full,
    # 2^-24 * 485 * sqrt(s) <= 4.6e-4 relative to |O| = 1 at s = 256
    check(Job("bf16", 520, 1032, [8, 64, 130, 256], spectrum=spectrum, seed=3), tol=4.6e-4 if spectrum == "one" else O_TOL)


@gpu
def test_hyper_parameters():
    hp = [dict(lr=1e-3, momentum=0.0, nesterov=False, scale="none"), dict(lr=0.1, momentum=0.5, nesterov=True, scale="rms"),
          dict(lr=0.02, ns_steps=1), dict(lr=0.02, ns_steps=3, coeffs=(1.875, -1.25, 0.375), eps=1e-2),
          dict(lr=0.02, ns_steps=12, coeffs=(1.5, -0.5, 0.0), weight_decay=0.1)]
    check(Job("bf16", 136, 264, [8, 24, 5, 40, 2], hp=hp, seed=4))


@gpu
def test_output_blocks():
    check(Job("bf16", 136, 768, [8, 24], blocks=3, seed=5))


@gpu
def test_zero_and_non_finite_gradients():
    job = Job("bf16", 136, 264, [8, 24, 5], seed=6)
    job.g[0][0].zero_(); job.m[0][0].zero_()
    job.g[1][1][3, 2] = math.nan
    job.g[0][2][1, 1] = math.inf
    p0 = [[x.clone() for x in v] for v in job.p]
    clean = Job("bf16", 136, 264, [8, 24, 5], seed=6)
    e = job.engine()
    job.step(e), clean.step(e)
    decay = 1 - 0.02 * 0.01
    assert torch.allclose(job.p[0][0], p0[0][0] * decay, rtol=2.0 ** -22, atol=0)      # X = 0: only the decay
    assert torch.isnan(job.p[1][1]).all() and torch.isnan(job.p[0][2]).all()
    assert int(torch.isnan(job.m[1][1]).sum()) == 1 and int(torch.isinf(job.m[0][2]).sum()) == 1
    for side, i in ((0, 1), (1, 0), (1, 2)):
        assert torch.equal(job.p[side][i], clean.p[side][i])
    e.close()


@gpu
@pytest.mark.parametrize("scale", [1e-25, 1e-12, 1e12])
def test_gradient_scale_does_not_matter(scale):
    # u's norm cancels as long as eps is small next to it; at 1e-25 eps decides (X = u / eps, tiny)
    job = Job("fp32", 136, 264, [8, 24], seed=7)
    for v in job.g + job.m:
        for x in v:
            x.mul_(scale)
    check(job)


@gpu
def test_packed_equals_alone_and_repeats_bit_for_bit():
    a, b = Job("bf16", 1048, 264, [8, 130, 17], seed=8), Job("bf16", 1048, 264, [8, 130, 17], seed=8)
    e = a.engine()
    a.step(e), b.step(e)
    assert all(torch.equal(x, y) for x, y in zip(a.tensors(), b.tensors()))
    one = Job("bf16", 1048, 264, [8, 130, 17], seed=8)
    for side in (0, 1):
        for v in (one.g, one.m, one.p, one.out):
            v[side] = v[side][1:2]
    one.ranks, one.n, one.hp = [130], 1, one.hp[:1]
    one.step(e)
    for side in (0, 1):
        assert torch.equal(one.p[side][0], a.p[side][1]) and torch.equal(one.m[side][0], a.m[side][1])
    e.close()


@gpu
def test_two_captured_steps_and_another_stream():
    ref, job = Job("bf16", 264, 392, [5, 64], seed=9), Job("bf16", 264, 392, [5, 64], seed=9)
    e = job.engine()
    ref.step(e, times=3)
    tab, st, work = job.args(e)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pl.plora_muon_step(e.h, 2, tab, st, work.data_ptr(), s.cuda_stream)
    torch.cuda.synchronize()
    pl.plora_capture_reserve(e.h, 2)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pl.plora_muon_step(e.h, 2, tab, st, work.data_ptr(), s.cuda_stream)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref.tensors(), job.tensors()))
    del graphs, g
    pl.plora_capture_release(e.h)
    e.close()


@gpu
def test_a_training_step_of_the_set():
    """Forward with epilogue, its backward and the Muon step on its gradients, as a training loop runs
    them: the updated factors against the same chain in float64 on the library's gradients."""
    from test_epilogue import Problem
    p = Problem("bf16", 264, 392, [16, 8, 3], [130, 1, 57], seed=20)
    eng = p.engine()
    job = Job("bf16", 264, 392, [16, 8, 3], seed=21)
    for side, lay in ((0, p.A), (1, p.B)):
        job.out[side] = lay
        job.p[side] = [x.float() for x in lay]
    for _ in range(2):
        Y, saved, Z = eng.forward_epilogue(p.X, p.W, p.off, p.scales, p.A, p.B, bias=p.bias, activation="silu", residual=p.R)
        dX, dA, dB, db = eng.backward_epilogue(p.X, p.W, p.dY, p.off, p.scales, p.A, p.B, saved, Z=Z, activation="silu",
                                               want_dbias=True)
        ref = p.reference("silu", Z)
        for i in range(3):
            assert float((dA[i].double() - ref["dA"][i]).norm()) <= 2 * 2.0 ** -8 * float(ref["dA"][i].norm())
        job.g = [dA, dB]
        job.m = [[torch.zeros_like(x) for x in v] for v in job.g]
        check(job, tol=4.6e-4, eng=eng)     # adapter 1 has one token: its gradients have one direction
    eng.close()


# ------------------------------------------------------------------ refusals
def test_refusals_without_a_device():
    lib, out = pl.load(), ctypes.c_size_t(7)
    assert lib.plora_muon_work_bytes(None, 0, None, ctypes.byref(out)) == pl.PLORA_ERR_INVALID_ARG
    assert lib.plora_muon_step(None, 0, None, None, None, None) == pl.PLORA_ERR_INVALID_ARG
    assert ctypes.sizeof(pl.plora_muon_state) == 80
    st = pl.make_muon_states([dict(lr=0.5)], [16], [32], [48], [64])
    assert st[0].ns_steps == 5 and st[0].nesterov == 1 and st[0].scale == pl.PLORA_MUON_SCALE_ROWS and st[0].mB == 64
    with pytest.raises(KeyError):
        pl.make_muon_states([dict(lr=0.5, scale="cols")], [16], [32], [48], [64])


@gpu
def test_refusals_leave_the_state_alone():
    job = Job("bf16", 64, 72, [8, 4], seed=10)
    e = job.engine()
    before = [x.clone() for x in job.tensors()]
    bad = pl.PLORA_ERR_INVALID_ARG

    def status(change=None, work_off=0, hp=None, n=2, work=True):
        if hp:
            job.hp = [dict(lr=0.02) | hp] * 2
        tab, st, w = job.args(e)
        job.hp = [dict(lr=0.02)] * 2
        if change:
            change(tab, st)
        return pl.plora_muon_step(e.h, n, tab, st, w.data_ptr() + work_off if work else 0, 0, check=False)
    for hp in (dict(momentum=1.0), dict(momentum=-0.1), dict(eps=0.0), dict(eps=math.inf), dict(lr=math.nan), dict(ns_steps=0),
               dict(ns_steps=17), dict(coeffs=(1.0, math.inf, 0.0)), dict(weight_decay=math.nan)):
        assert status(hp=hp) == bad, hp
    host = np.zeros(1 << 16, np.uint8)

    def put(where, field, value):
        def f(tab, st):
            setattr((tab if where == "tab" else st)[0], field, value)
        return f
    other = job.m[0][1].data_ptr()
    for c in (put("st", "nesterov", 2), put("st", "scale", 3), put("st", "reserved", 1), put("st", "mA", None),
              put("st", "mA", job.m[0][0].data_ptr() + 4), put("st", "A_master", None), put("tab", "dA", host.ctypes.data),
              put("tab", "rank", 0), put("tab", "rank", 9),
              put("st", "mA", other),                              # two adapters with one momentum
              put("st", "mA", job.g[0][0].data_ptr()),             # the momentum over the gradient
              put("st", "B_master", job.p[0][0].data_ptr())):
        assert status(c) == bad
    assert status(work_off=16) == bad and status(work=False) == bad and status(n=3) == bad
    assert "max_adapters" in pl.plora_last_error(e.h)
    assert status(n=0) == pl.PLORA_OK
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, job.tensors()))
    f = Job("fp32", 64, 72, [8], seed=11)
    ef = f.engine()
    tab, st, w = f.args(ef)
    st[0].A_master = f.p[0][0].data_ptr()
    assert pl.plora_muon_step(ef.h, 1, tab, st, w.data_ptr(), 0, check=False) == bad
    ef.close()
    e.close()
