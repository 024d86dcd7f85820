"""Matrix products grouped by expert (mok_grouped_forward / _backward) against the formula in fp64, and their refusals.

Every row is held to what test_linear.py derives for one matrix: fp32 sums of K terms, in whatever order, within
sum_tol(K) of the sum of magnitudes, half a step of the output's type, and the backward's operand dp half a step of each
product. Rows in no group hold NaN in every input, and outputs' rows there have to stay as they were."""
import ctypes

import pytest
import torch

from test_linear import DEV, _mok, act64, near, sum_tol

KEEP = 77.0  # what outputs hold before a call


class Case:
    def __init__(self, counts, N, K, act, epi, lead=0, tail=0, seed=0, wgrad_f32=False):
        mok = self.mok = _mok()
        self.t = t = mok.TORCH_DTYPE[mok.DTYPES[act]]
        E, M = len(counts), lead + sum(counts) + tail
        self.d = d = mok.GroupedDesc(M, N, K, E, act=mok.DTYPES[act], epi=mok.EPILOGUES[epi],
                                     flags=mok.FLAG_WGRAD_F32 if wgrad_f32 else 0)
        self.epi, self.wt = epi, torch.float32 if wgrad_f32 else t
        self.off = [lead]
        for n in counts:
            self.off.append(self.off[-1] + n)
        g = torch.Generator().manual_seed(seed + M * 31 + N * 7 + K + E)
        n = lambda *s: torch.randn(*s, generator=g)
        P = d.P
        self.x, self.w = n(M, K).to(t), (n(E, P, K) * K**-0.5).to(t)
        self.bias, self.res, self.dy = n(E, P), n(M, N).to(t), n(M, N).to(t)
        self.pre = (1.5 * n(M, P)).to(t)
        self.dx_add, self.dw_add = n(M, K).to(t), n(E, P, K).to(self.wt)
        self.out = torch.ones(M, dtype=torch.bool)
        self.out[self.off[0]:self.off[-1]] = False
        for v in (self.x, self.res, self.dy, self.pre, self.dx_add):
            v[self.out] = float("nan")
        sz = mok.grouped_workspace_query(d)
        self.fws, self.bws = (torch.full((max(v, 16),), 255, dtype=torch.uint8, device=DEV)
                              for v in (sz["fwd_ws"], sz["bwd_ws"]))
        self.goff = torch.tensor(self.off, dtype=torch.int32, device=DEV)

    def groups(self):
        return [(e, slice(a, b)) for e, (a, b) in enumerate(zip(self.off, self.off[1:]))]

    def new(self, *s, dtype=None):
        return torch.full(s, KEEP, dtype=dtype or self.t, device=DEV)

    def forward(self, bias=True, res=True, pre=True):
        d, dev = self.d, lambda v: v.to(DEV)
        y, p = self.new(d.M, d.N), self.new(d.M, d.P) if pre else None
        self.mok.grouped_forward(d, dev(self.x), dev(self.w), self.goff, y, bias=dev(self.bias) if bias else None,
                                 res=dev(self.res) if res else None, pre=p, ws=self.fws)
        return y, p

    def check_forward(self, bias=True, res=True):
        y, pre = (v.cpu() for v in self.forward(bias, res))
        assert (y[self.out] == KEEP).all() and (pre[self.out] == KEEP).all()
        N = self.d.N
        for e, r in self.groups():
            x, w = self.x[r].double(), self.w[e].double()
            p = x @ w.t() + (self.bias[e].double() if bias else 0)
            err = sum_tol(self.d.K) * (x.abs() @ w.abs().t() + (self.bias[e].double().abs() if bias else 0))
            near(pre[r], p, err, ("pre", e))
            f = act64(self.epi, p)
            ef = 1.13 * err[:, :N] * p[:, N:].abs() + p[:, :N].abs() * err[:, N:] if self.epi == "swiglu" else 1.13 * err
            add = self.res[r].double() if res else torch.zeros(())
            near(y[r], f + add, ef + 2.0**-20 * (f.abs() + add.abs()), ("y", e))

    def backward(self, add=True, dx=True, dw=True, db=True):
        d, dev = self.d, lambda v: v.to(DEV)
        gx = self.new(d.M, d.K) if dx else None
        gw = self.new(d.E, d.P, d.K, dtype=self.wt) if dw else None
        gb = self.new(d.E, d.P, dtype=torch.float32) if db else None
        self.mok.grouped_backward(d, dev(self.dy), dev(self.x) if dw else None, dev(self.w) if dx else None, self.goff,
                                  dx=gx, dw=gw, db=gb, pre=None if self.epi == "none" else dev(self.pre),
                                  dx_add=dev(self.dx_add) if add and dx else None,
                                  dw_add=dev(self.dw_add) if add and dw else None, ws=self.bws)
        return gx, gw, gb

    def dp64(self, r):
        """dp of rows r, and what its fp32 errors are relative to (test_linear.Case.dp_terms)."""
        from test_linear import Case as Linear
        one = Linear.__new__(Linear)
        one.epi, one.dy, one.pre, one.d = self.epi, self.dy[r], self.pre[r], self.d
        return one.dp64(), one.dp_terms()

    def check_backward(self, add=True):
        gx, gw, gb = (v.cpu() for v in self.backward(add))
        assert (gx[self.out] == KEEP).all()
        rnd = 0.0 if self.epi == "none" else {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-20}[self.t]
        for e, r in self.groups():
            dw_add = self.dw_add[e].double() if add else torch.zeros(())
            if r.start == r.stop:
                assert (gw[e].double() == dw_add).all() and (gb[e] == 0).all(), e
                continue
            dp, terms = self.dp64(r)
            x, w = self.x[r].double(), self.w[e].double()
            dx_add = self.dx_add[r].double() if add else torch.zeros(())
            for name, got, a, b, more, t in (("dx", gx[r], dp, w, dx_add, terms), ("dw", gw[e], dp.t(), x, dw_add, terms.t())):
                size = a.abs() @ b.abs()
                root = (a.square() @ b.square()).sqrt()
                err = sum_tol(a.shape[1]) * (size + more.abs()) + rnd * torch.minimum(size, 5 * root) + 2.0**-20 * (t @ b.abs())
                near(got, a @ b + more, err, (name, e))
            near(gb[e], dp.sum(0), (sum_tol(r.stop - r.start) + 2.0**-18) * terms.sum(0), ("db", e))


# rows of the groups, N, K, rows before the first and behind the last group
SMALL = [([1], 8, 8, 0, 0), ([0], 8, 16, 0, 3), ([0, 0, 5, 0], 24, 40, 2, 0), ([3, 1, 0, 2], 64, 136, 1, 4), ([17] * 5, 40, 72, 0, 0),
         ([64, 65, 0, 63, 1], 128, 128, 5, 5), ([130, 7, 300], 72, 264, 0, 9), ([1] * 70, 136, 40, 0, 1),
         ([0] * 100 + [9] + [0] * 91, 16, 200, 3, 3), ([31, 0, 33, 32] * 20, 264, 88, 0, 0), ([257, 256, 255], 256, 256, 0, 0),
         ([700, 0, 2], 520, 8, 0, 0), ([2, 1, 0, 3, 1, 1], 200, 2048, 0, 0), ([40] * 12, 384, 1032, 0, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("epi", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_forward(act, epi):
    for counts, N, K, lead, tail in SMALL:
        print("case grouped fwd", len(counts), sum(counts), N, K, act, epi, flush=True)
        c = Case(counts, N, K, act, epi, lead, tail)
        c.check_forward()
        c.check_forward(bias=False, res=False)


@pytest.mark.gpu
@pytest.mark.parametrize("epi", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_backward(act, epi):
    for counts, N, K, lead, tail in SMALL:
        print("case grouped bwd", len(counts), sum(counts), N, K, act, epi, flush=True)
        c = Case(counts, N, K, act, epi, lead, tail)
        c.check_backward()
        c.check_backward(add=False)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", [([1000, 24, 0, 1024], 1024, 512), ([4100], 264, 1032), ([37] * 111, 128, 256),
                                        ([2500, 3000], 776, 520), ([3] * 300, 256, 264), ([12000, 40], 64, 136)])
def test_larger(counts, N, K):
    for act, epi in (("bf16", "none"), ("bf16", "swiglu"), ("f32", "gelu")):
        print("case grouped", len(counts), sum(counts), N, K, act, epi, flush=True)
        c = Case(counts, N, K, act, epi, tail=3)
        c.check_forward(bias=epi == "none")
        c.check_backward(add=epi == "none")


@pytest.mark.gpu
@pytest.mark.parametrize("N,K,epi", [(2048, 1024, "none"), (1024, 2048, "silu"), (1032, 1032, "swiglu")])
def test_tiles_as_high_as_their_groups(N, K, epi):
    """Groups of one row up to a few tiles, at both sides of every height that a tile of 256 rows is cut to."""
    counts = [1, 63, 64, 65, 127, 128, 129, 0, 191, 192, 193, 255, 256, 257, 320, 384, 385, 511, 512, 513, 700, 769, 20, 300]
    print("case grouped heights", N, K, epi, flush=True)
    c = Case(counts, N, K, "bf16", epi, lead=1, tail=4)
    c.check_forward(res=epi == "none")
    c.check_backward(add=epi == "none")


@pytest.mark.gpu
@pytest.mark.parametrize("E", [63, 64, 65, 1000, 1024])
def test_many_groups(E):
    """A lane of the search holds one group, or up to 16; runs of empty ones."""
    g = torch.Generator().manual_seed(E)
    counts = torch.randint(0, 4, (E,), generator=g)
    counts[E // 3: E // 2] = 0
    print("case grouped many", E, int(counts.sum()), flush=True)
    for act, epi in (("bf16", "swiglu"), ("f32", "none")):
        c = Case(counts.tolist(), 24, 40, act, epi, lead=2, tail=2)
        c.check_forward()
        c.check_backward()


@pytest.mark.gpu
def test_one_group_has_every_row():
    for e in (0, 5, 31):
        counts = [0] * 32
        counts[e] = 1500
        c = Case(counts, 128, 264, "bf16", "swiglu")
        print("case grouped hot", e, flush=True)
        c.check_forward()
        c.check_backward()


@pytest.mark.gpu
def test_fp32_weight_gradients():
    for counts in ([20, 0, 21], [1030, 5]):
        c = Case(counts, 24, 136, "bf16", "none", wgrad_f32=True)
        c.check_backward()


@pytest.mark.gpu
def test_one_group_is_the_dense_product():
    """The same tiles give the same bits as mok_linear_forward where both take them (128 x 128 and larger)."""
    mok = _mok()
    c = Case([2048], 1024, 512, "bf16", "swiglu")
    y, pre = c.forward()
    d = mok.LinearDesc(2048, 1024, 512, epi=mok.EPI_SWIGLU)
    y2, pre2 = torch.empty_like(y), torch.empty_like(pre)
    ws = torch.empty(max(mok.linear_workspace_query(d)["fwd_ws"], 16), dtype=torch.uint8, device=DEV)
    mok.linear_forward(d, c.x.to(DEV), c.w[0].to(DEV), y2, bias=c.bias[0].to(DEV), res=c.res.to(DEV), pre=pre2, ws=ws)
    assert torch.equal(y, y2) and torch.equal(pre, pre2)


@pytest.mark.gpu
def test_in_place_addends_and_repeats():
    for counts, N, K in (([30, 0, 40], 136, 264), ([500, 524], 512, 1024), ([9], 256, 2048)):
        c = Case(counts, N, K, "bf16", "swiglu")
        y, pre = c.forward()
        gx, gw, gb = c.backward()
        dev = lambda v: v.to(DEV)
        r, ax, aw = dev(c.res).clone(), dev(c.dx_add).clone(), dev(c.dw_add).clone()
        c.mok.grouped_forward(c.d, dev(c.x), dev(c.w), c.goff, r, bias=dev(c.bias), res=r, ws=c.fws)
        c.mok.grouped_backward(c.d, dev(c.dy), dev(c.x), dev(c.w), c.goff, dx=ax, dw=aw, pre=dev(c.pre), dx_add=ax,
                               dw_add=aw, ws=c.bws)
        assert torch.equal(r, y) and torch.equal(ax, gx) and torch.equal(aw, gw)
        assert torch.equal(c.backward(dw=False, db=False)[0], gx)
        assert torch.equal(c.backward(dx=False, db=False)[1], gw)
        assert torch.equal(c.backward(dx=False, dw=False)[2], gb)


@pytest.mark.gpu
def test_groups_do_not_touch_each_other():
    """A NaN in one group's rows or weights reaches that group only, in every output, also where groups share a tile's
    rows; guard rows around the outputs stay."""
    counts = [5, 40, 3, 100]
    for act in ("bf16", "f32"):
        c = Case(counts, 72, 88, act, "none", lead=1, tail=1)
        clean, grads = c.forward(bias=False, res=False)[0].cpu(), [v.cpu() for v in c.backward(add=False)]
        lo, hi = c.off[1], c.off[2]
        c.x[lo:hi] = float("nan")
        c.w[1] = float("inf")
        c.dy[lo:hi] = float("nan")
        c.pre[lo:hi] = float("nan")
        got, bad = c.forward(bias=False, res=False)[0].cpu(), [v.cpu() for v in c.backward(add=False)]
        keep = torch.ones(c.d.M, dtype=torch.bool)
        keep[lo:hi] = False
        assert torch.equal(got[keep], clean[keep]) and torch.equal(bad[0][keep], grads[0][keep])
        others = [0, 2, 3]
        assert torch.equal(bad[1][others], grads[1][others]) and torch.equal(bad[2][others], grads[2][others])


@pytest.mark.gpu
def test_offsets_that_descend_or_pass_the_rows_stay_inside():
    """Unspecified results, but nothing outside the arrays is written."""
    M, N, K, E = 60, 40, 72, 6
    mok = _mok()
    for off in ([-5, 70, 10, 200, -1, 3, 1 << 30], [60, 50, 40, 30, 20, 10, 0], [-(1 << 31)] * 7, [(1 << 31) - 1] * 7,
                [0, (1 << 31) - 1, 0, (1 << 31) - 1, 0, (1 << 31) - 1, 0]):
        print("case grouped bad offsets", off, flush=True)
        for epi in (mok.EPI_NONE, mok.EPI_SWIGLU):
            d = mok.GroupedDesc(M, N, K, E, epi=epi)
            new = lambda *s, dtype=torch.bfloat16: torch.ones(s[0] + 2, *s[1:], dtype=dtype, device=DEV)
            x, dy, pre, w = (torch.zeros(*s, dtype=torch.bfloat16, device=DEV) for s in ((M, K), (M, N), (M, d.P), (E, d.P, K)))
            y, p, dx, dw, db = new(M, N), new(M, d.P), new(M, K), new(E, d.P, K), new(E, d.P, dtype=torch.float32)
            ws = torch.empty(max(mok.grouped_workspace_query(d)["bwd_ws"], 16), dtype=torch.uint8, device=DEV)
            o = torch.tensor(off, dtype=torch.int32, device=DEV)
            mok.grouped_forward(d, x, w, o, y[1:-1], pre=p[1:-1], ws=ws)
            mok.grouped_backward(d, dy, x, w, o, dx=dx[1:-1], dw=dw[1:-1], db=db[1:-1], ws=ws,
                                 pre=None if epi == mok.EPI_NONE else pre)
            for v in (y, p, dx, dw, db):
                assert (v[0] == 1).all() and (v[-1] == 1).all()


@pytest.mark.gpu
def test_captured_and_replayed():
    """Two graphs that share a workspace, replayed between eager steps with other offsets in the same array."""
    c = Case([50, 0, 100, 30], 264, 520, "bf16", "swiglu", tail=20)
    dev = lambda v: torch.nan_to_num(v).to(DEV)
    x, w, dy, b = dev(c.x), dev(c.w), dev(c.dy), dev(c.bias)
    M, E, P = c.d.M, c.d.E, c.d.P
    y, p, dx, dw, db = c.new(M, 264), c.new(M, P), c.new(M, 520), c.new(E, P, 520), c.new(E, P, dtype=torch.float32)

    def fwd():
        c.mok.grouped_forward(c.d, x, w, c.goff, y, bias=b, pre=p, ws=c.fws)

    def bwd():
        c.mok.grouped_backward(c.d, dy, x, w, c.goff, dx=dx, dw=dw, db=db, pre=p, ws=c.bws)

    fwd(), bwd()
    torch.cuda.synchronize()
    graphs = []
    for f in (fwd, bwd):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for off in ([0, 10, 10, 150, 200], [5, 5, 5, 6, 190], [0, 200, 200, 200, 200], [0, 0, 0, 0, 0]):
        c.goff.copy_(torch.tensor(off, dtype=torch.int32))
        x.mul_(0.75)
        outs = (y, p, dx, dw, db)
        for v in outs:
            v.fill_(KEEP)
        fwd(), bwd()
        want = [v.clone() for v in outs]
        for v in outs:
            v.fill_(KEEP)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs)), off


@pytest.mark.gpu
def test_on_another_stream():
    c = Case([33, 100, 0, 64], 128, 256, "bf16", "swiglu")
    want = [*c.forward(), *c.backward()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [*c.forward(), *c.backward()]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.gpu
def test_no_rows():
    c = Case([0, 0, 0], 64, 128, "bf16", "swiglu")
    c.forward()
    gx, gw, gb = c.backward()
    assert torch.equal(gw.cpu(), c.dw_add) and (gb == 0).all()
    assert (c.backward(add=False)[1] == 0).all()


@pytest.mark.gpu
def test_gradients_against_differences():
    """dx, dw and db of a fp32 layer against central differences of the forward: of f(x) + O(h^2), here exact for the
    product (bilinear) and within h^2/6 max|f'''| < h^2 of GELU; each side's fp32 forward off by its tolerance."""
    c = Case([6, 0, 9], 16, 24, "f32", "gelu", tail=2)
    mok, d = c.mok, c.d
    live = ~c.out
    dy = torch.where(live[:, None], c.dy, torch.zeros(()))
    x, w, b = c.x.clone(), c.w.clone(), c.bias.clone()
    x[~live] = 0

    def loss(x, w, b):
        y = c.new(d.M, d.N)
        p = c.new(d.M, d.P)
        mok.grouped_forward(d, x.to(DEV), w.to(DEV), c.goff, y, bias=b.to(DEV), pre=p)
        return (y.double().cpu()[live] * dy.double()[live]).sum(), p

    _, p = loss(x, w, b)
    dx, dw, db = c.new(d.M, d.K), c.new(d.E, d.P, d.K), c.new(d.E, d.P)
    mok.grouped_backward(d, dy.to(DEV), x.to(DEV), w.to(DEV), c.goff, dx=dx, dw=dw, db=db, pre=p, ws=c.bws)
    g = torch.Generator().manual_seed(3)
    h = 2.0**-6
    for name, at, grad in (("x", 0, dx), ("w", 1, dw), ("b", 2, db)):
        args = [x, w, b]
        v = torch.randn(args[at].shape, generator=g)
        if at == 0:
            v[~live] = 0
        v /= v.norm()
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + h * v, args[at] - h * v
        num = (loss(*up)[0] - loss(*dn)[0]) / (2 * h)
        ana = (grad.double().cpu()[live] * v[live].double()).sum() if at == 0 else (grad.double().cpu() * v.double()).sum()
        # fp32 forwards: each of the 15 x 16 outputs off by 2^-20 of about 2, with |dy| about 1, over 2 h
        tol = h * h * float(dy.abs().sum()) * 0.25 + 2.0**-20 * 2 * float(dy.abs().sum()) / h
        assert abs(num - ana) < tol, (name, float(num), float(ana), tol)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_offsets_past_32_bits(act):
    """Rows whose elements lie past 2^31 of x, y and dx, in the last groups, and weights past 2^31 elements."""
    mok = _mok()
    t = mok.TORCH_DTYPE[mok.DTYPES[act]]
    M, N, K, E = (1 << 27) + 77, 24, 24, 3
    print("case grouped large", M, N, K, act, flush=True)
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.empty(M, K, dtype=t, device=DEV).normal_(generator=g)
    w = torch.randn(E, N, K, generator=g, device=DEV).to(t)
    cut = [0, 1000, M - 400, M]
    off = torch.tensor(cut, dtype=torch.int32, device=DEV)
    d = mok.GroupedDesc(M, N, K, E, act=mok.DTYPES[act], flags=mok.FLAG_WGRAD_F32)
    ws = torch.empty(max(mok.grouped_workspace_query(d)["bwd_ws"], 16), dtype=torch.uint8, device=DEV)
    y, dw, db = torch.empty(M, N, dtype=t, device=DEV), torch.empty(E, N, K, device=DEV), torch.empty(E, N, device=DEV)
    mok.grouped_forward(d, x, w, off, y)
    for e, sl in ((0, slice(0, 300)), (1, slice(M // 2, M // 2 + 300)), (2, slice(M - 300, M))):
        near(y[sl], (x[sl].double() @ w[e].double().t()).cpu(), 24 * 2.0**-24 * (x[sl].double().abs() @ w[e].double().abs().t()).cpu(), "y")
    x[:] = 0            # the weight gradient of a few rows at both ends
    x[5], x[-3] = 1.0, 2.0
    y[:] = 0
    y[5, 1], y[-3, 2] = 3.0, 4.0
    mok.grouped_backward(d, y, x, w, off, dw=dw, db=db, ws=ws)
    want = torch.zeros(E, N, K, device=DEV)
    want[0, 1], want[2, 2] = 3.0, 8.0
    assert torch.equal(dw, want)
    assert db[0, 1] == 3 and db[2, 2] == 4 and float(db.abs().sum()) == 7
    mok.grouped_backward(d, y, x, w, off, dx=x, ws=ws)   # x itself is not read for dx
    assert torch.equal(x[-3].double(), (4 * w[2, 2].double()).to(t).double()) and (x[:5] == 0).all() and (x[-2:] == 0).all()
    del x, y
    E, N, K = 5, 4096, 1 << 17     # w of 2^31.3 elements
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[4, -1], w[3, 0] = 1.0, 2.0
    x = torch.ones(4, K, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(4, N, dtype=torch.bfloat16, device=DEV)
    d = mok.GroupedDesc(4, N, K, E)
    off = torch.tensor([0, 0, 0, 0, 2, 4], dtype=torch.int32, device=DEV)
    mok.grouped_forward(d, x, w, off, y)
    assert (y[:2, 0] == 2.0 * K).all() and (y[2:, -1] == K).all() and float(y.float().sum()) == 6.0 * K


# ---- refusals (no GPU needed) ----

@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 3), (dict(M=1 << 30), 3), (dict(N=0), 3), (dict(N=12), 3), (dict(K=4), 3), (dict(K=(1 << 20) + 8), 3),
    (dict(N=(1 << 20) + 8), 3), (dict(M=1 << 29, N=1 << 12), 3), (dict(N=1 << 20, K=1 << 20), 3), (dict(E=0), 3),
    (dict(E=1025), 3), (dict(E=1024, N=1 << 17, K=1024), 3), (dict(E=1024, N=1 << 20, epi=3), 3), (dict(act=2), 4),
    (dict(epi=4), 4), (dict(epi=-1), 4), (dict(flags=4), 3),
])
def test_descriptor_refusals(kw, status):
    mok = _mok()
    with pytest.raises(mok.MokError) as ei:
        mok.grouped_workspace_query(mok.GroupedDesc(**{**dict(M=4, N=16, K=8, E=2), **kw}))
    assert ei.value.status == status


def test_pointer_refusals():
    mok = _mok()
    lib, ok, odd = mok._lib, ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    d = mok.GroupedDesc(300, 16, 4096, 3, epi=mok.EPI_SILU)
    sz = mok.grouped_workspace_query(d)
    args = [ok] * 8
    for i in (0, 1, 3, 5):
        assert lib.mok_grouped_forward(d.c(), *args[:i], None, *args[i + 1:], sz["fwd_ws"], None) == 1, i
    for i in range(7):
        assert lib.mok_grouped_forward(d.c(), *args[:i], odd, *args[i + 1:], sz["fwd_ws"], None) == 2, i
    args = [ok] * 11
    assert lib.mok_grouped_backward(d.c(), *args, sz["bwd_ws"] - 1, None) == 6
    for i in (0, 1, 2, 3, 4, 10):
        assert lib.mok_grouped_backward(d.c(), *args[:i], None, *args[i + 1:], sz["bwd_ws"], None) == 1, i
    for i in (5, 6, 7, 8, 9):
        assert lib.mok_grouped_backward(d.c(), *args[:i], odd, *args[i + 1:], sz["bwd_ws"], None) == 2, i
    assert lib.mok_grouped_workspace_query(d.c(), None) == 1
    assert lib.mok_grouped_workspace_query(None, ctypes.byref(mok._LinearSizes())) == 1


def test_binding_refusals():
    mok = _mok()
    d = mok.GroupedDesc(4, 16, 8, 2)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    good = dict(x=z(4, 8), w=z(2, 16, 8), off=off, y=z(4, 16))
    for bad in (dict(w=z(16, 8)), dict(x=z(4, 8).float()), dict(y=z(4, 8)), dict(x=None), dict(off=None), dict(off=off.long()),
                dict(off=off[:2]), dict(bias=z(2, 16)), dict(res=z(16, 4)), dict(w=z(2, 8, 16).transpose(1, 2)), dict()):
        with pytest.raises(ValueError):
            mok.grouped_forward(d, **{**good, **bad})
    with pytest.raises(ValueError):
        mok.grouped_backward(d, z(4, 16), z(4, 8), z(2, 16, 8), off, dw=z(2, 16, 8), dx_add=z(4, 8))
