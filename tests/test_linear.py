"""Matrix product with bias, activation and residual in its epilogue (mok_linear_forward /
_backward) against the formula in fp64, and its refusals.

Tolerances: products of bf16 or fp32 values are exact or one rounding off in fp32, and an fp32
sum of K of them, in whatever order, is within K * 2^-24 of the sum of magnitudes; the errors
of rounding are of either sign, so sqrt(K) * 4 * 2^-24 of it is allowed (K * 2^-24 for K <= 16).
A bf16 output adds half a step, 2^-8 of the value, and the backward's operand dp half a step of
each product: 2^-8 of the sum of magnitudes, of which random signs leave 5 / sqrt(K) of the root
sum of squares. The activations' slopes are below 1.13, their fp32 forms within 2^-20 of the terms
that they add (Case.dp_terms)."""
import ctypes

import pytest
import torch

DEV = "cuda"


def _mok():
    from mixture_experts_layer_stable_amd import mok
    return mok


def act64(epi, p):
    N = p.shape[1] // 2
    if epi == "none":
        return p
    if epi == "silu":
        return p * torch.sigmoid(p)
    if epi == "gelu":
        return p * torch.special.ndtr(p)
    return p[:, :N] * torch.sigmoid(p[:, :N]) * p[:, N:]


def sum_tol(K):
    return 2.0**-24 * (K if K <= 16 else max(16, 4 * K**0.5))


def near(got, want, tol, name):
    assert torch.isfinite(got).all(), name
    half = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}[got.dtype] * 1.01
    off = (got.double().cpu() - want).abs()
    lim = tol + half * (want.abs() + tol) + 1e-30
    assert (off <= lim).all(), (name, float((off / lim).max()), int((off > lim).sum()))


class Case:
    def __init__(self, M, N, K, act, epi, seed=0, wgrad_f32=False):
        mok = self.mok = _mok()
        self.t = t = mok.TORCH_DTYPE[mok.DTYPES[act]]
        self.d = d = mok.LinearDesc(M, N, K, act=mok.DTYPES[act], epi=mok.EPILOGUES[epi],
                                    flags=mok.FLAG_WGRAD_F32 if wgrad_f32 else 0)
        self.epi, self.wt = epi, torch.float32 if wgrad_f32 else t
        g = torch.Generator().manual_seed(seed + M * 31 + N * 7 + K)
        n = lambda *s: torch.randn(*s, generator=g)
        P = d.P
        self.x, self.w = n(M, K).to(t), (n(P, K) * K**-0.5).to(t)
        self.bias, self.res, self.dy = n(P), n(M, N).to(t), n(M, N).to(t)
        self.pre = (1.5 * n(M, P)).to(t)
        self.dx_add, self.dw_add = n(M, K).to(t), n(P, K).to(self.wt)
        sz = mok.linear_workspace_query(d)
        self.fws, self.bws = (torch.full((max(v, 16),), 255, dtype=torch.uint8, device=DEV)
                              for v in (sz["fwd_ws"], sz["bwd_ws"]))

    def new(self, *s, dtype=None):
        return torch.full(s, float("nan"), dtype=dtype or self.t, device=DEV)

    def forward(self, bias=True, res=True, pre=True):
        d, dev = self.d, lambda v: v.to(DEV)
        y, p = self.new(d.M, d.N), self.new(d.M, d.P) if pre else None
        self.mok.linear_forward(d, dev(self.x), dev(self.w), y, bias=dev(self.bias) if bias else None,
                                res=dev(self.res) if res else None, pre=p, ws=self.fws)
        return y, p

    def check_forward(self, bias=True, res=True):
        y, pre = self.forward(bias, res)
        x, w = self.x.double(), self.w.double()
        p = x @ w.t() + (self.bias.double() if bias else 0)
        size = x.abs() @ w.abs().t() + (self.bias.double().abs() if bias else 0)
        e = sum_tol(self.d.K) * size
        near(pre, p, e, "pre")
        f, N = act64(self.epi, p), self.d.N
        if self.epi == "swiglu":
            ef = 1.13 * e[:, :N] * p[:, N:].abs() + p[:, :N].abs() * e[:, N:]
        else:
            ef = 1.13 * e
        near(y, f + (self.res.double() if res else 0), ef + 2.0**-20 * (f.abs() + (self.res.double().abs() if res else 0)), "y")

    def backward(self, add=True, dx=True, dw=True, db=True):
        d, dev = self.d, lambda v: v.to(DEV)
        gx, gw = self.new(d.M, d.K) if dx else None, self.new(d.P, d.K, dtype=self.wt) if dw else None
        gb = self.new(d.P, dtype=torch.float32) if db else None
        self.mok.linear_backward(d, dev(self.dy), dev(self.x) if dw else None, dev(self.w) if dx else None, dx=gx, dw=gw,
                                 db=gb, pre=None if self.epi == "none" else dev(self.pre),
                                 dx_add=dev(self.dx_add) if add and dx else None,
                                 dw_add=dev(self.dw_add) if add and dw else None, ws=self.bws)
        return gx, gw, gb

    def dp64(self):
        dy = self.dy.double()
        if self.epi == "none":
            return dy
        p = self.pre.double().requires_grad_()
        return torch.autograd.grad(act64(self.epi, p), p, dy)[0]

    def dp_terms(self):
        """What dp's fp32 errors are relative to: f' = sig (1 + p (1 - sig)) of SiLU has a zero near p = -1.28, where the
        two terms, each rounded to 2^-24 of itself, cancel (GELU's Phi + p phi likewise), so the error there is
        relative to the terms' magnitudes and not to f'."""
        dy, p, N = self.dy.double().abs(), self.pre.double(), self.d.N
        silu = lambda v: torch.sigmoid(v) * (1 + v.abs() * torch.sigmoid(-v))
        if self.epi == "none":
            return dy
        if self.epi == "silu":
            return dy * silu(p)
        if self.epi == "gelu":
            return dy * (torch.special.ndtr(p) + p.abs() * torch.exp(-p * p / 2) / 2.5066282746)
        a, u = p[:, :N], p[:, N:]
        return torch.cat([dy * u.abs() * silu(a), dy * (a * torch.sigmoid(a)).abs()], 1)

    def check_backward(self, add=True):
        gx, gw, gb = self.backward(add)
        dp, x, w = self.dp64(), self.x.double(), self.w.double()
        terms = self.dp_terms()
        rnd = 0.0 if self.epi == "none" else {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-20}[self.t]
        for name, got, a, b, more, t in (("dx", gx, dp, w, self.dx_add, terms), ("dw", gw, dp.t(), x, self.dw_add, terms.t())):
            more = more.double() if add else torch.zeros(())
            size = a.abs() @ b.abs()
            root = (a.square() @ b.square()).sqrt()
            e = sum_tol(a.shape[1]) * (size + more.abs()) + rnd * torch.minimum(size, 5 * root) + 2.0**-20 * (t @ b.abs())
            near(got, a @ b + more, e, name)
        near(gb, dp.sum(0), (sum_tol(self.d.M) + 2.0**-18) * terms.sum(0), "db")


SMALL = [(1, 8, 8), (3, 16, 24), (5, 64, 136), (17, 40, 72), (64, 128, 128), (65, 136, 264), (130, 264, 1032), (300, 72, 40),
         (33, 1000, 520), (257, 256, 256), (129, 384, 2048), (31, 512, 7168), (1, 4096, 2048), (16, 200, 16), (700, 520, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("epi", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_forward(act, epi):
    for M, N, K in SMALL:
        print("case linear fwd", M, N, K, act, epi, flush=True)
        c = Case(M, N, K, act, epi)
        c.check_forward()
        c.check_forward(bias=False, res=False)


@pytest.mark.gpu
@pytest.mark.parametrize("epi", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_backward(act, epi):
    for M, N, K in SMALL:
        print("case linear bwd", M, N, K, act, epi, flush=True)
        c = Case(M, N, K, act, epi)
        c.check_backward()
        c.check_backward(add=False)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(2048, 1024, 512), (1000, 2048, 1536), (4100, 264, 1032), (520, 776, 4096), (8, 2048, 7168),
                                   (48, 7168, 2048), (100, 1032, 7168), (6000, 384, 1024)])
def test_larger_bf16(M, N, K):
    for epi in ("none", "swiglu"):
        print("case linear", M, N, K, epi, flush=True)
        c = Case(M, N, K, "bf16", epi)
        c.check_forward(bias=epi == "none")
        c.check_backward(add=epi == "none")


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 8), (1, 24, 1000), (2, 4104, 2056), (5, 2056, 4104), (15, 40, 72), (16, 1000, 520),
                                   (17, 8, 2048), (31, 264, 1032), (32, 1032, 136), (33, 520, 264), (1, 16, 40000)])
def test_few_rows(M, N, K, act):
    """Single tokens and small batches of them; K shorter and longer than a round of pieces, odd ends."""
    for epi in ("none", "silu", "gelu", "swiglu"):
        print("case linear few", M, N, K, act, epi, flush=True)
        c = Case(M, N, K, act, epi)
        c.check_forward()
        c.check_forward(bias=False, res=False)


@pytest.mark.gpu
def test_fp32_weight_gradients():
    for M, N, K in ((40, 24, 136), (1030, 384, 256)):
        c = Case(M, N, K, "bf16", "none", wgrad_f32=True)
        c.check_backward()


@pytest.mark.gpu
def test_in_place_addends_and_repeats():
    """y over res, dx over dx_add, dw over dw_add; parts of the backward alone; the same bits each time."""
    for M, N, K in ((70, 136, 264), (1024, 512, 1024), (9, 256, 2048)):
        c = Case(M, N, K, "bf16", "swiglu")
        y, pre = c.forward()
        gx, gw, gb = c.backward()
        r, ax, aw = c.res.to(DEV), c.dx_add.to(DEV), c.dw_add.to(DEV)
        c.mok.linear_forward(c.d, c.x.to(DEV), c.w.to(DEV), r, bias=c.bias.to(DEV), res=r, ws=c.fws)
        c.mok.linear_backward(c.d, c.dy.to(DEV), c.x.to(DEV), c.w.to(DEV), dx=ax, dw=aw, pre=c.pre.to(DEV), dx_add=ax,
                              dw_add=aw, ws=c.bws)
        assert torch.equal(r, y) and torch.equal(ax, gx) and torch.equal(aw, gw)
        assert torch.equal(c.backward(dw=False, db=False)[0], gx)
        assert torch.equal(c.backward(dx=False, db=False)[1], gw)
        assert torch.equal(c.backward(dx=False, dw=False)[2], gb)


@pytest.mark.gpu
def test_rows_do_not_touch_each_other():
    """A NaN or infinity in one row of x or w reaches that row or column only; guard bytes around
    every output stay."""
    M, N, K = 150, 200, 88
    c = Case(M, N, K, "bf16", "none")
    clean = c.forward(bias=False, res=False)[0]
    c.x[7, 3] = float("nan")
    c.w[11, 80] = float("inf")
    big = torch.full((M + 2, N), 3.0, dtype=torch.bfloat16, device=DEV)
    y = big[1:-1]
    c.mok.linear_forward(c.d, c.x.to(DEV), c.w.to(DEV), y, ws=c.fws)
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[7] = False
    keep[:, 11] = False
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
    assert not torch.isfinite(y.cpu()[~keep]).any()
    assert (big[0] == 3).all() and (big[-1] == 3).all()


@pytest.mark.gpu
def test_captured_and_replayed():
    c = Case(200, 264, 520, "bf16", "swiglu")
    x, w, dy, pre, ax, aw = (v.to(DEV) for v in (c.x, c.w, c.dy, c.pre, c.dx_add, c.dw_add))
    y, p, dx, dw, db = c.new(200, 264), c.new(200, 528), c.new(200, 520), c.new(528, 520), c.new(528, dtype=torch.float32)

    def step():
        c.mok.linear_forward(c.d, x, w, y, pre=p, ws=c.fws)
        c.mok.linear_backward(c.d, dy, x, w, dx=dx, dw=dw, db=db, pre=p, dx_add=ax, dw_add=aw, ws=c.bws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.mul_(0.75)
        step()
        outs = (y, p, dx, dw, db)
        want = [v.clone() for v in outs]
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.gpu
def test_no_rows():
    c = Case(0, 64, 128, "bf16", "swiglu")
    c.forward()
    gx, gw, gb = c.backward()
    assert torch.equal(gw.cpu(), c.dw_add) and (gb == 0).all()
    assert (c.backward(add=False)[1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_offsets_past_32_bits(act):
    """Rows whose elements lie past 2^31 of x, y and dx, and a weight gradient over all of them."""
    mok = _mok()
    t = mok.TORCH_DTYPE[mok.DTYPES[act]]
    M, N, K = (1 << 27) + 77, 24, 24
    print("case linear large", M, N, K, act, flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(M, K, dtype=t, device=DEV).normal_(generator=g)
    w = torch.randn(N, K, generator=g, device=DEV).to(t)
    d = mok.LinearDesc(M, N, K, act=mok.DTYPES[act], flags=mok.FLAG_WGRAD_F32)
    sz = mok.linear_workspace_query(d)
    ws = torch.empty(max(sz["fwd_ws"], sz["bwd_ws"], 16), dtype=torch.uint8, device=DEV)
    y, dw = torch.empty(M, N, dtype=t, device=DEV), torch.empty(N, K, device=DEV)
    mok.linear_forward(d, x, w, y, ws=ws)
    for sl in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        near(y[sl], (x[sl].double() @ w.double().t()).cpu(), 24 * 2.0**-24 * (x[sl].double().abs() @ w.double().abs().t()).cpu(), "y")
    x[:] = 0            # the weight gradient of a few rows at both ends
    x[5], x[-3] = 1.0, 2.0
    y[:] = 0
    y[5, 1], y[-3, 2] = 3.0, 4.0
    mok.linear_backward(d, y, x, w, dw=dw, ws=ws)
    want = torch.zeros(N, K, device=DEV)
    want[1], want[2] = 3.0, 8.0
    assert torch.equal(dw, want)
    mok.linear_backward(d, y, x, w, dx=x, ws=ws)   # x itself is not read for dx
    assert torch.equal(x[-3].double(), (4 * w[2].double()).to(t).double()) and (x[:5] == 0).all() and (x[-2:] == 0).all()


# ---- refusals (no GPU needed) ----

@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 3), (dict(M=1 << 31), 3), (dict(N=0), 3), (dict(N=12), 3), (dict(K=4), 3), (dict(K=(1 << 20) + 8), 3),
    (dict(N=(1 << 20) + 8), 3), (dict(M=1 << 30, N=1 << 12), 3), (dict(N=1 << 20, K=1 << 20), 3), (dict(act=2), 4),
    (dict(epi=4), 4), (dict(epi=-1), 4), (dict(flags=4), 3),
])
def test_descriptor_refusals(kw, status):
    mok = _mok()
    with pytest.raises(mok.MokError) as ei:
        mok.linear_workspace_query(mok.LinearDesc(**{**dict(M=4, N=16, K=8), **kw}))
    assert ei.value.status == status


def test_pointer_refusals():
    mok = _mok()
    lib, ok, odd = mok._lib, ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    d = mok.LinearDesc(300, 16, 4096, epi=mok.EPI_SILU)
    sz = mok.linear_workspace_query(d)
    args = [ok] * 7
    for i in (0, 1, 4):
        assert lib.mok_linear_forward(d.c(), *args[:i], None, *args[i + 1:], sz["fwd_ws"], None) == 1, i
    for i in range(6):
        assert lib.mok_linear_forward(d.c(), *args[:i], odd, *args[i + 1:], sz["fwd_ws"], None) == 2, i
    if sz["fwd_ws"]:
        assert lib.mok_linear_forward(d.c(), *args, sz["fwd_ws"] - 1, None) == 6
    args = [ok] * 10
    assert lib.mok_linear_backward(d.c(), *args, sz["bwd_ws"] - 1, None) == 6
    for i in (0, 1, 2, 3, 9):
        assert lib.mok_linear_backward(d.c(), *args[:i], None, *args[i + 1:], sz["bwd_ws"], None) == 1, i
    for i in (4, 5, 6, 7, 8):
        assert lib.mok_linear_backward(d.c(), *args[:i], odd, *args[i + 1:], sz["bwd_ws"], None) == 2, i


def test_binding_refusals():
    mok = _mok()
    d = mok.LinearDesc(4, 16, 8)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    good = dict(x=z(4, 8), w=z(16, 8), y=z(4, 16))
    for bad in (dict(w=z(8, 16).t()), dict(x=z(4, 8).float()), dict(y=z(4, 8)), dict(x=None), dict(bias=z(16)), dict(res=z(16, 4)), dict()):
        with pytest.raises(ValueError):
            mok.linear_forward(d, **{**good, **bad})
    with pytest.raises(ValueError):
        mok.linear_backward(d, z(4, 16), z(4, 8), z(16, 8), dw=z(16, 8), dx_add=z(4, 8))
