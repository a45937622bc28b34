"""Measured cases of two operators of the packed LoRA library.

* ``fwd`` and ``train``: the packed projection with bias, activation and residual in its epilogue,
  ``Z_i = X_i W + s_i (X_i A_i) B_i + b_i``, ``Y = act(Z) + R`` over N adapters' contiguous row
  segments; ``train`` adds the backward (dX, dA_i, dB_i, db_i, dR).
* ``muon``: one Muon step for every adapter's A_i and B_i: ``m <- mu m + g``, ``u = g + mu m``,
  ``X = u / (|u|_F + eps)``, five times ``X <- a X + (b X X^T + c (X X^T)^2) X``, and
  ``p <- p (1 - lr wd) - lr sqrt(max(1, rows / cols)) X``, with p also rounded to bf16.

With ``own`` false, ``run`` is the plain form in elementary torch operations, in fp32.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
MU, LR, WD, EPS = 0.95, 0.02, 0.01, 1e-7


# ------------------------------------------------------------------------------------ cases
def _layer(name, kind, d_in, d_out, n, tokens, rank_lo, rank_hi, act, bias, residual, dtype="bf16"):
    """tokens: all rows of the packed buffer; bias: "none", "shared" (one frozen vector) or "each" (one
    trained vector per adapter)."""
    return {"name": name, "kind": kind, "d_in": d_in, "d_out": d_out, "n": n, "tokens": tokens, "rank_lo": rank_lo,
            "rank_hi": rank_hi, "act": act, "bias": bias, "residual": residual, "dtype": dtype}


def _muon(name, d_in, d_out, n, rank_lo, rank_hi, blocks=1, dtype="bf16"):
    return {"name": name, "kind": "muon", "d_in": d_in, "d_out": d_out, "n": n, "rank_lo": rank_lo,
            "rank_hi": rank_hi, "blocks": blocks, "dtype": dtype}


def listed():
    return [
        # one new token for each of 8 adapters through a query projection with a frozen bias
        _layer("fwd decode q 8x1", "fwd", 3584, 3584, 8, 8, 8, 64, "none", "shared", False),
        # evaluation of 8 adapters over a few ragged batches each
        _layer("fwd q ragged", "fwd", 3584, 3584, 8, 4001, 8, 64, "none", "each", False),
        # an MLP's first projection with its activation, whole evaluation batches
        _layer("fwd up silu 16k", "fwd", 4096, 14336, 16, 16384, 8, 128, "silu", "none", False),
        # an MLP's last projection, added to the residual stream
        _layer("fwd down residual", "fwd", 14336, 4096, 16, 8192, 8, 128, "none", "shared", True),
        # a small fp32 job: the library's debug-precision type
        _layer("train fp32 small", "train", 256, 256, 4, 320, 4, 16, "gelu", "each", True, "fp32"),
        # query projections fine-tuned with one trained bias per adapter
        _layer("train q lora bias", "train", 3584, 3584, 8, 16384, 8, 64, "none", "each", False),
        # a GELU MLP's first projection, odd sizes, ragged segments
        _layer("train up gelu odd", "train", 1048, 4296, 5, 3001, 1, 40, "gelu", "each", True),
        # an MLP's first projection, the largest training call
        _layer("train up silu 16k", "train", 4096, 14336, 16, 16384, 8, 128, "silu", "each", False),
        # a small job's four adapters
        _muon("muon fp32 small", 256, 256, 4, 4, 16, dtype="fp32"),
        # stacked query, key and value projections of one adapter set
        _muon("muon qkv blocks", 4096, 6144, 16, 16, 16, blocks=3),
        # the benchmark's adapter mix: 32 ranks between 8 and 128
        _muon("muon up mix", 4096, 14336, 32, 8, 128),
        # the largest rank the library takes
        _muon("muon rank 256", 4096, 4096, 8, 256, 256),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("fwd", "train", "muon"))
    d_in = 8 * _log_int(rng, 8, 1792)
    d_out = 8 * _log_int(rng, 8, 1792)
    lo = _log_int(rng, 1, 128)
    hi = min(256, lo + _log_int(rng, 1, 128))
    if kind == "muon":
        n = _log_int(rng, 1, 32)
        while n > 1 and n * hi * (d_in + d_out) * (64 + hi) > 32 * 68 * 18432 * 132:
            n //= 2
        blocks = 1
        if hi <= 64 and rng.random() < 0.3:
            blocks, d_out = 3, 768 * max(1, d_out // 768)
        return _muon("drawn", d_in, d_out, n, lo, hi, blocks, rng.choice(("bf16", "bf16", "fp32")))
    n = _log_int(rng, 1, 16)
    tokens = _log_int(rng, 1, 16384)
    dtype = "fp32" if rng.random() < 0.1 else "bf16"
    while tokens > 1 and tokens * (d_in * d_out + 3 * hi * (d_in + d_out)) > (16384 * 4096 * 14336 if dtype == "bf16" else 1 << 30):
        tokens //= 2
    return _layer("drawn", kind, d_in, d_out, n, tokens, lo, hi, rng.choice(("none", "relu", "gelu", "gelu_tanh", "silu")),
                  rng.choice(("none", "shared", "each")), rng.random() < 0.5, dtype)


def _ranks(case):
    """Ranks spread evenly over [rank_lo, rank_hi]."""
    n, lo, hi = case["n"], case["rank_lo"], case["rank_hi"]
    return [lo + ((hi - lo) * i) // max(1, n - 1) for i in range(n)]


def _offsets(case):
    """Segment bounds of a long-tailed mix: adapter i's share of the rows falls by a tenth each step."""
    n, t = case["n"], case["tokens"]
    w = [0.9 ** i for i in range(n)]
    off, run_, total = [0], 0.0, sum(w)
    for x in w:
        run_ += x
        off.append(int(round(t * run_ / total)))
    return off


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _prepare_layer(case, seed):
    g, n, di, do = _gen(seed), case["n"], case["d_in"], case["d_out"]
    t, train = case["tokens"], case["kind"] == "train"
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    ranks, off = _ranks(case), _offsets(case)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    def uniform(*shape, lim=1.0):
        return ((torch.rand(shape, generator=g, device="cuda") * 2 - 1) * lim).to(dt)

    s = {"case": case, "off": off, "ranks": ranks, "scales": [16.0 / r for r in ranks]}
    s["X"] = normal(t, di)
    s["W"] = normal(do, di, std=0.02)
    s["A"] = [uniform(r, di, lim=math.sqrt(6 / di)) for r in ranks]
    s["B"] = [normal(do, r, std=0.01) for r in ranks]
    s["bias"] = None if case["bias"] == "none" else [normal(do, std=0.2) for _ in range(n if case["bias"] == "each" else 1)]
    s["R"] = normal(t, do) if case["residual"] else None
    s["dY"] = normal(t, do) if train else None
    s["seg"] = torch.repeat_interleave(torch.arange(n, device="cuda"), torch.tensor([off[i + 1] - off[i] for i in range(n)], device="cuda"))
    if train:
        s["leaves"] = [s["X"]] + s["A"] + s["B"] + (s["bias"] if case["bias"] == "each" else []) + ([s["R"]] if case["residual"] else [])
        for x in s["leaves"]:
            x.requires_grad_(True)
    if own:
        import packed_lora_fine_b200 as pl
        s["engine"] = pl.PackedLoRA(di, do, case["dtype"], max_adapters=n, max_rank=max(ranks), max_tokens=max(1, t))
    return s


def _matrices(case):
    """(rows, cols) of every matrix of the step, A's then B's: with output blocks A_i stacks one
    [r][d_in] matrix per block and B_i's rows split into the blocks' rows."""
    p = case["blocks"]
    a = [(r, case["d_in"]) for r in _ranks(case) for _ in range(p)]
    b = [(case["d_out"] // p, r) for r in _ranks(case) for _ in range(p)]
    return a, b


def _prepare_muon(case, seed):
    g = _gen(seed)
    ms = sum(_matrices(case), [])
    total = sum(r * c for r, c in ms)

    def gradients(scale):
        """Gaussian noise plus four directions that stand out of it, as token sums leave them."""
        x = torch.randn(total, generator=g, device="cuda")
        at = 0
        for r, c in ms:
            m = x[at:at + r * c].view(r, c)
            k = min(4, r, c)
            u, v = torch.randn(r, k, generator=g, device="cuda"), torch.randn(k, c, generator=g, device="cuda")
            m += u @ (v * (2.0 / torch.arange(1, k + 1, device="cuda"))[:, None])
            at += r * c
        return x * scale

    n_a = sum(r * c for r, c in _matrices(case)[0])
    p = torch.empty(total, device="cuda")
    p[:n_a] = (torch.rand(n_a, generator=g, device="cuda") * 2 - 1) * math.sqrt(6 / case["d_in"])
    p[n_a:] = torch.randn(total - n_a, generator=g, device="cuda") * 0.01
    s = {"case": case, "ms": ms, "g": gradients(1e-3), "m": gradients(1e-2), "p": p}
    s["out"] = p.to(torch.bfloat16) if case["dtype"] == "bf16" else None
    if own:
        import packed_lora_fine_b200 as pl
        n, di, do, blocks, ranks = case["n"], case["d_in"], case["d_out"], case["blocks"], _ranks(case)
        if case["dtype"] == "fp32" and blocks > 1:
            # the library's output blocks are bf16's; in fp32 each block's A and B are an adapter's of their own
            n, do, blocks, ranks = n * blocks, do // blocks, 1, [r for r in ranks for _ in range(blocks)]
        eng = pl.PackedLoRA(di, do, case["dtype"], max_adapters=n, max_rank=max(ranks), max_tokens=16,
                            out_blocks=[do // blocks] * blocks if blocks > 1 else None)
        sizes = [r * blocks * di for r in ranks] + [do * r for r in ranks]
        at = [sum(sizes[:k]) for k in range(2 * n)]

        def ptrs(t):
            q = [t.data_ptr() + t.element_size() * o for o in at]
            return q[:n], q[n:]

        lay = s["out"] if case["dtype"] == "bf16" else s["p"]
        pa, pb = ptrs(s["p"])
        ma, mb = ptrs(s["m"])
        tab = pl.make_table(ranks, [1.0] * n, *ptrs(lay), *ptrs(s["g"]))
        hp = [dict(lr=LR, momentum=MU, nesterov=True, weight_decay=WD, eps=EPS, ns_steps=NS_STEPS, coeffs=NS, scale="rows")] * n
        master = case["dtype"] == "bf16"
        st = pl.make_muon_states(hp, pa if master else None, pb if master else None, ma, mb)
        work = torch.empty(pl.plora_muon_work_bytes(eng.h, n, tab), dtype=torch.uint8, device="cuda")
        s |= {"engine": eng, "adapters": n, "tab": tab, "states": st, "work": work}
    return s


def prepare(case, seed):
    return _prepare_muon(case, seed) if case["kind"] == "muon" else _prepare_layer(case, seed)


# ------------------------------------------------------------------------------------ plain forms
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 + z * (1 - sg))


@torch.no_grad()
def _plain_layer(s):
    case, off, dt = s["case"], s["off"], s["X"].dtype
    X, W = s["X"].float(), s["W"].float()
    A, B = [a.float() for a in s["A"]], [b.float() for b in s["B"]]
    n, rows = case["n"], [slice(off[i], off[i + 1]) for i in range(case["n"])]
    Z = X @ W.T
    H = [s["scales"][i] * (X[rows[i]] @ A[i].T) for i in range(n)]
    for i in range(n):
        Z[rows[i]] += H[i] @ B[i].T
    if s["bias"] is not None:
        b = torch.stack(s["bias"]).float()
        Z += b[s["seg"]] if case["bias"] == "each" else b
    Y = _act(Z, case["act"])
    if s["R"] is not None:
        Y = Y + s["R"].float()
    Y = Y.to(dt)
    if case["kind"] == "fwd":
        return Y
    dZ = s["dY"].float()
    if case["act"] != "none":
        dZ = dZ * _act_grad(Z, case["act"])
    G = [s["scales"][i] * (dZ[rows[i]] @ B[i]) for i in range(n)]
    dX = dZ @ W
    for i in range(n):
        dX[rows[i]] += G[i] @ A[i]
    out = [Y, dX.to(dt)]
    out += [(G[i].T @ X[rows[i]]).to(dt) for i in range(n)]
    out += [(dZ[rows[i]].T @ H[i]).to(dt) for i in range(n)]
    if case["bias"] == "each":
        out += [dZ[rows[i]].sum(0).to(dt) for i in range(n)]
    if s["R"] is not None:
        out.append(s["dY"])
    return out


def _orthogonalise(u, eps):
    """Newton-Schulz on the side that makes X X^T the smaller of the two squares."""
    tall = u.shape[0] > u.shape[1]
    x = u.T if tall else u
    x = x / (torch.sqrt((x * x).sum()) + eps)
    for _ in range(NS_STEPS):
        q = x @ x.T
        x = NS[0] * x + (NS[1] * q + NS[2] * (q @ q)) @ x
    return x.T if tall else x


@torch.no_grad()
def _plain_muon(s):
    g, m, p = s["g"], s["m"], s["p"]
    m.mul_(MU).add_(g)
    u, at = g + MU * m, 0
    p.mul_(1 - LR * WD)
    for r, c in s["ms"]:
        p[at:at + r * c].view(r, c).sub_(LR * math.sqrt(max(1.0, r / c)) * _orthogonalise(u[at:at + r * c].view(r, c), EPS))
        at += r * c
    if s["out"] is not None:
        s["out"].copy_(p)
    return {"p": p, "m": m} | ({"out": s["out"]} if s["out"] is not None else {})


# ------------------------------------------------------------------------------------ one pass
def _own_layer(s):
    import packed_lora_fine_b200 as pl
    case, eng = s["case"], s["engine"]
    bias = None if s["bias"] is None else s["bias"] if case["bias"] == "each" else s["bias"][0]
    if case["kind"] == "fwd":
        return eng.forward_epilogue(s["X"], s["W"], s["off"], s["scales"], s["A"], s["B"], bias=bias,
                                    activation=case["act"], residual=s["R"], want_Z=False)[0]
    Y = pl.packed_lora(eng, s["X"], s["W"], s["off"], s["scales"], s["A"], s["B"], bias=bias, activation=case["act"],
                       residual=s["R"])
    return [Y.detach(), *torch.autograd.grad(Y, s["leaves"], s["dY"])]


def _own_muon(s):
    import packed_lora_fine_b200 as pl
    pl.plora_muon_step(s["engine"].h, s["adapters"], s["tab"], s["states"], s["work"].data_ptr(),
                       torch.cuda.current_stream().cuda_stream)
    return {"p": s["p"], "m": s["m"]} | ({"out": s["out"]} if s["out"] is not None else {})


def run(state):
    muon = state["case"]["kind"] == "muon"
    if own:
        return _own_muon(state) if muon else _own_layer(state)
    return _plain_muon(state) if muon else _plain_layer(state)


# ------------------------------------------------------------------------------------ work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    di, do, ranks = case["d_in"], case["d_out"], _ranks(case)
    if case["kind"] == "muon":
        a, b = _matrices(case)
        elems = sum(r * c for r, c in a + b)
        # half a Gram product (it is symmetric) and one small-by-long product per matrix
        flops = sum(3 * min(r, c) * r * c for r, c in a + b)
        return {"bytes": (22 if case["dtype"] == "bf16" else 20) * elems, "flops": flops}
    off, t = _offsets(case), case["tokens"]
    low = sum(2 * (off[i + 1] - off[i]) * ranks[i] * (di + do) for i in range(case["n"]))
    factors = sum(ranks) * (di + do)
    biases = do * (0 if case["bias"] == "none" else 1 if case["bias"] == "shared" else case["n"])
    nbytes = es * (t * di + di * do + factors + biases + t * do * (2 if case["residual"] else 1))
    flops = 2 * t * di * do + low
    if case["kind"] == "train":
        # dY in, dX, dA, dB and db out, on the inputs the forward has read
        nbytes += es * (t * do + t * di + factors + (biases if case["bias"] == "each" else 0))
        flops += 2 * t * di * do + 2 * low
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------------------------ 64 bits
def _exact_layer(case, seed):
    s = _prepare_layer(case, seed)
    n, off = case["n"], s["off"]
    d = {k: (None if s[k] is None else s[k].detach().double()) for k in ("X", "W", "R", "dY")}
    A, B = [a.detach().double() for a in s["A"]], [b.detach().double() for b in s["B"]]
    bias = None if s["bias"] is None else [b.detach().double() for b in s["bias"]]
    train = case["kind"] == "train"
    leaves = [d["X"], *A, *B] + (bias if case["bias"] == "each" else []) + ([d["R"]] if case["residual"] else [])
    if train:
        for x in leaves:
            x.requires_grad_(True)
    parts = []
    for i in range(n):
        x = d["X"][off[i]:off[i + 1]]
        z = torch.nn.functional.linear(x, d["W"] + s["scales"][i] * (B[i] @ A[i]))
        parts.append(z if bias is None else z + bias[i if case["bias"] == "each" else 0])
    z = torch.cat(parts)
    f = torch.nn.functional
    y = {"none": lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"),
         "silu": f.silu}[case["act"]](z)
    if case["residual"]:
        y = y + d["R"]
    if not train:
        return y
    return [y.detach(), *torch.autograd.grad(y, leaves, d["dY"])]


@torch.no_grad()
def _exact_muon(case, seed):
    s = _prepare_muon(case, seed)
    g, m, p = s["g"].double(), s["m"].double(), s["p"].double()
    m = MU * m + g
    u, parts, at = g + MU * m, [], 0
    for r, c in s["ms"]:
        # singular values through the polynomial, from the eigenvalues of the small Gram matrix
        x = u[at:at + r * c].view(r, c)
        x = x / (torch.linalg.matrix_norm(x) + EPS)
        w = x if r <= c else x.T
        lam, q = torch.linalg.eigh(w @ w.T)
        gain = torch.ones_like(lam)
        for _ in range(NS_STEPS):
            f = NS[0] + NS[1] * lam + NS[2] * lam * lam
            gain, lam = gain * f, lam * f * f
        o = (q * gain) @ (q.T @ w)
        o = o if r <= c else o.T
        parts.append((math.sqrt(max(1.0, r / c)) * o).reshape(-1))
        at += r * c
    p = p * (1 - LR * WD) - LR * torch.cat(parts)
    return {"p": p, "m": m} | ({"out": p} if s["out"] is not None else {})


def exact(case, seed):
    return _exact_muon(case, seed) if case["kind"] == "muon" else _exact_layer(case, seed)
