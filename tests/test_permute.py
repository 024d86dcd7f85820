"""Rows to the experts' order and back (mok_dispatch_*, mok_combine_*) against the formula in fp64, and their refusals.

Tolerances: a sum of k products in fp32, one fused step each from the residual on, is within (k + 1) 2^-24 of the sum of
magnitudes; dgate is an fp32 sum of H exact or once rounded products in some order (sum_tol of test_linear.py, plus
one rounding of each fp32 product); the output's rounding adds half a step. Copies and zeros are exact."""
import ctypes

import pytest
import torch

from test_linear import DEV, _mok, near, sum_tol

KEEP = 77.0


class Case:
    def __init__(self, T, k, H, act, drop=0.0, pad=0, seed=0):
        mok = self.mok = _mok()
        self.t = t = mok.TORCH_DTYPE[mok.DTYPES[act]]
        g = torch.Generator().manual_seed(seed + 31 * T + 7 * k + H)
        S, R = T * k, T * k + pad
        self.perm = torch.full((R,), -1, dtype=torch.int32)
        self.inv = torch.full((S,), -1, dtype=torch.int32)
        rows = torch.randperm(R, generator=g)[:S]
        live = torch.rand(S, generator=g) >= drop
        self.inv[live] = rows[live].int()
        self.perm[rows[live]] = torch.arange(S)[live].int()
        self.inv = self.inv.view(T, k)
        n = lambda *s: torch.randn(*s, generator=g)
        self.x, self.o, self.res = n(T, H).to(t), n(R, H).to(t), n(T, H).to(t)
        self.gate = torch.rand(T, k, generator=g) - 0.2
        self.o[self.perm < 0] = float("nan")    # rows of no slot are not read
        self.d = mok.PermuteDesc(T, H, k, R, act=mok.DTYPES[act])
        self.T, self.k, self.H, self.R = T, k, H, R

    def new(self, *s, dtype=None):
        return torch.full(s, KEEP, dtype=dtype or self.t, device=DEV)

    def terms(self, gate):
        """[T, k, H] of gate * o[inv], 0 for dropped slots."""
        o = torch.nan_to_num(self.o.double())[self.inv.clamp(min=0).long()] if self.R else torch.zeros(self.T, self.k, self.H).double()
        return o * ((self.inv >= 0) * gate.double())[:, :, None]

    def check(self):
        mok, d, dev = self.mok, self.d, lambda v: v.to(DEV)
        perm, inv, gate = dev(self.perm), dev(self.inv), dev(self.gate)
        xs = self.new(self.R, self.H)
        mok.dispatch_forward(d, dev(self.x), perm, xs)
        want = torch.zeros(self.R, self.H, dtype=self.t)
        on = self.perm >= 0
        want[on] = self.x[(self.perm[on] // self.k).long()]
        assert torch.equal(xs.cpu(), want)
        for res in (True, False):
            for g in (True, False):
                y, dx = self.new(self.T, self.H), self.new(self.T, self.H)
                mok.combine_forward(d, dev(self.o), inv, y, gate=gate if g else None, res=dev(self.res) if res else None)
                t = self.terms(self.gate if g else torch.ones_like(self.gate))
                add = self.res.double() if res else torch.zeros(())
                size = t.abs().sum(1) + add.abs()
                near(y, t.sum(1) + add, (self.k + 1) * 2.0**-24 * size, "y")
                if not g:
                    mok.dispatch_backward(d, dev(self.o), inv, dx, add=dev(self.res) if res else None)
                    assert torch.equal(dx, y)
        for g in (True, False):
            for pads in (True, False):
                do, dg = self.new(self.R, self.H), self.new(self.T, self.k, dtype=torch.float32)
                mok.combine_backward(d, dev(self.x), dev(self.o), inv, do, gate=gate if g else None, dgate=dg,
                                     perm=perm if pads else None)
                do, dg = do.cpu(), dg.cpu()
                s = self.perm[on].long()
                gs = self.gate.view(-1)[s].double() if g else torch.ones(len(s)).double()
                near(do[on], gs[:, None] * self.x[s // self.k].double(), 0.0, "do")
                assert (do[~on] == (0.0 if pads else KEEP)).all()
                t = self.terms(torch.ones_like(self.gate)) * self.x.double()[:, None, :]
                near(dg, t.sum(-1), (sum_tol(self.H) + 2.0**-24) * t.abs().sum(-1), "dgate")
                assert (dg[self.inv < 0] == 0).all()
                only = self.new(self.R, self.H)
                mok.combine_backward(d, dev(self.x), None, inv, only, gate=gate if g else None, perm=perm if pads else None)
                assert torch.equal(only.cpu(), do)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", [(1, 1, 8), (1, 16, 64), (3, 2, 24), (5, 8, 7168), (64, 3, 1000), (257, 9, 136), (1000, 4, 520),
                                   (33, 7, 4104), (2, 5, 32768)])
def test_small(T, k, H, act):
    for drop, pad in ((0.0, 0), (0.3, 5), (1.0, 3)):
        print("case permute", T, k, H, act, drop, pad, flush=True)
        Case(T, k, H, act, drop, pad).check()


@pytest.mark.gpu
def test_batch():
    for act in ("bf16", "f32"):
        Case(4096, 8, 512, act, 0.05, 100).check()


@pytest.mark.gpu
@pytest.mark.parametrize("act,T", [("bf16", 1000), ("bf16", 2300), ("f32", 500), ("f32", 1150)])
def test_rows_that_the_last_cache_holds_and_more(act, T):
    """Less and more than 256 MB of rows in a call, which are stored in two ways. Small integers and gates that are powers of
    two: every output is exact, in bf16 (8 bits) too."""
    mok = _mok()
    k, H, t = 8, 7168, mok.TORCH_DTYPE[mok.DTYPES[act]]
    print("case permute caches", act, T, flush=True)
    g = torch.Generator(device=DEV).manual_seed(T)
    R = T * k + 5
    rows = torch.randperm(R, generator=g, device=DEV)[:T * k]
    live = torch.rand(T * k, generator=g, device=DEV) >= 0.1
    perm = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    perm[rows[live]] = torch.arange(T * k, device=DEV)[live].int()
    inv = torch.where(live, rows, torch.full_like(rows, -1)).int().view(T, k)
    x = torch.randint(-4, 5, (T, H), generator=g, device=DEV).to(t)
    o = torch.randint(-4, 5, (R, H), generator=g, device=DEV).to(t)
    gate = torch.exp2(torch.randint(-1, 2, (T, k), generator=g, device=DEV).float())
    new = lambda *s, dtype=t: torch.full(s, KEEP, dtype=dtype, device=DEV)
    d = mok.PermuteDesc(T, H, k, R, act=mok.DTYPES[act])
    xs, y, dx, do, dg = new(R, H), new(T, H), new(T, H), new(R, H), new(T, k, dtype=torch.float32)
    mok.dispatch_forward(d, x, perm, xs)
    slot = perm.clamp(min=0).long()
    on = (perm >= 0)[:, None]
    assert torch.equal(xs, torch.where(on, x[slot // k], torch.zeros((), dtype=t, device=DEV)))
    mok.combine_forward(d, o, inv, y, gate=gate)
    mok.dispatch_backward(d, o, inv, dx, add=x)
    wy, wdx, wdg = torch.zeros(T, H, device=DEV), x.float().clone(), torch.zeros(T, k, device=DEV)
    for j in range(k):
        v = o[inv[:, j].clamp(min=0).long()].float() * (inv[:, j] >= 0)[:, None]
        wy += gate[:, j:j + 1] * v
        wdx += v
        wdg[:, j] = (v * x.float()).sum(1)
    assert torch.equal(y, wy.to(t)) and torch.equal(dx, wdx.to(t))
    mok.combine_backward(d, x, o, inv, do, gate=gate, dgate=dg, perm=perm)
    assert torch.equal(do, torch.where(on, (gate.view(-1)[slot][:, None] * x[slot // k].float()).to(t), torch.zeros((), dtype=t, device=DEV)))
    assert torch.equal(dg, wdg)


@pytest.mark.gpu
def test_without_rows_or_tokens():
    mok = _mok()
    for T, R in ((0, 0), (0, 5), (5, 0)):
        d = mok.PermuteDesc(T, 64, 2, R)
        z = lambda *s, dtype=torch.bfloat16: torch.full(s, KEEP, dtype=dtype, device=DEV)
        perm = torch.full((R,), -1, dtype=torch.int32, device=DEV)
        inv = torch.full((T, 2), -1, dtype=torch.int32, device=DEV)
        xs, y, do, dg = z(R, 64), z(T, 64), z(R, 64), z(T, 2, dtype=torch.float32)
        mok.dispatch_forward(d, z(T, 64), perm, xs)
        mok.combine_forward(d, z(R, 64), inv, y)
        mok.combine_backward(d, z(T, 64), z(R, 64), inv, do, dgate=dg, perm=perm)
        assert (xs == 0).all() and (y == 0).all() and (do == 0).all() and (dg == 0).all()


@pytest.mark.gpu
def test_indices_out_of_range_are_none():
    mok = _mok()
    d = mok.PermuteDesc(4, 64, 2, 8)
    x = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    o = torch.ones(8, 64, dtype=torch.bfloat16, device=DEV)
    perm = torch.tensor([0, 8, -1, -(1 << 31), (1 << 31) - 1, 7, 9, 100], dtype=torch.int32, device=DEV)
    inv = torch.tensor([[0, 8], [-1, 100], [-(1 << 31), (1 << 31) - 1], [-7, 5]], dtype=torch.int32, device=DEV)
    xs, y, do = (torch.full((n, 64), KEEP, dtype=torch.bfloat16, device=DEV) for n in (8, 4, 8))
    dg = torch.full((4, 2), KEEP, device=DEV)
    mok.dispatch_forward(d, x, perm, xs)
    assert xs[:, 0].tolist() == [1, 0, 0, 0, 0, 1, 0, 0]
    mok.combine_forward(d, o, inv, y)
    assert y[:, 0].tolist() == [1, 0, 0, 1]
    mok.combine_backward(d, x, o, inv, do, dgate=dg, perm=perm)
    assert do[:, 0].tolist() == [1, 0, 0, 0, 0, 1, 0, 0] and dg.tolist() == [[64, 0], [0, 0], [0, 0], [0, 64]]


@pytest.mark.gpu
def test_values_that_are_not_finite_stay_in_their_rows():
    c = Case(40, 4, 136, "bf16", 0.2, 3)
    dev = lambda v: v.to(DEV)
    c.o[c.inv[3][c.inv[3] >= 0].long()] = float("inf")
    c.gate[5] = float("nan")
    y = c.new(40, 136)
    c.mok.combine_forward(c.d, dev(c.o), dev(c.inv), y, gate=dev(c.gate))
    ok = torch.isfinite(y.cpu()).all(1)
    some = (c.inv >= 0).any(1)
    for t in range(40):
        assert bool(ok[t]) == (t not in (3, 5) or not bool(some[t])), t


@pytest.mark.gpu
def test_in_place_captured_and_on_another_stream():
    c = Case(300, 6, 264, "bf16", 0.1, 10)
    dev = lambda v: v.to(DEV)
    o, inv, perm, gate, x = dev(torch.nan_to_num(c.o)), dev(c.inv), dev(c.perm), dev(c.gate), dev(c.x)
    want, same = c.new(300, 264), dev(c.res)
    c.mok.combine_forward(c.d, o, inv, want, gate=gate, res=dev(c.res))
    c.mok.combine_forward(c.d, o, inv, same, gate=gate, res=same)
    assert torch.equal(want, same)
    xs, y, do, dg = c.new(c.R, 264), c.new(300, 264), c.new(c.R, 264), c.new(300, 6, dtype=torch.float32)

    def step():
        c.mok.dispatch_forward(c.d, x, perm, xs)
        c.mok.combine_forward(c.d, xs, inv, y, gate=gate)
        c.mok.combine_backward(c.d, y, xs, inv, do, gate=gate, dgate=dg, perm=perm)
        c.mok.dispatch_backward(c.d, do, inv, y, add=x)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.mul_(0.75)
        perm.copy_(perm.roll(i))                       # another order of the same slots
        inv.view(-1)[perm[perm >= 0].long()] = torch.arange(c.R, device=DEV)[perm >= 0].int()
        step()
        want = [v.clone() for v in (xs, y, do, dg)]
        for v in (xs, y, do, dg):
            v.fill_(KEEP)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (xs, y, do, dg)))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows past 2^31 elements; powers of two, so every output is exact."""
    mok = _mok()
    T, k, H = 150000, 2, 8192      # 2^31.2 elements of xs
    print("case permute large", T, k, H, flush=True)
    d = mok.PermuteDesc(T, H, k)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    x.copy_(torch.exp2((torch.arange(T, device=DEV) % 7).float())[:, None].expand(T, H))
    perm = torch.arange(T * k, device=DEV).flip(0).to(torch.int32)
    inv = torch.arange(T * k, device=DEV).flip(0).to(torch.int32).view(T, k)
    xs, y = torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    mok.dispatch_forward(d, x, perm, xs)
    for r in (0, 1, T, 2 * T - 3, 2 * T - 1):
        assert torch.equal(xs[r], x[(2 * T - 1 - r) // 2])
    mok.dispatch_backward(d, xs, inv, y)
    assert torch.equal(y, 2 * x)
    dg = torch.empty(T, k, device=DEV)
    mok.combine_backward(d, x, xs.clone(), inv, xs, gate=torch.full((T, k), 4.0, device=DEV), dgate=dg)
    for r in (0, 1, T, 2 * T - 3, 2 * T - 1):
        assert torch.equal(xs[r], 4 * x[(2 * T - 1 - r) // 2])
    assert torch.equal(dg[:, 0], x[:, 0].float().square() * H) and torch.equal(dg[:, 0], dg[:, 1])


# ---- refusals (no GPU needed) ----

@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 3), (dict(T=1 << 31, R=0), 3), (dict(T=1 << 28, k=8), 3), (dict(k=0), 3), (dict(k=17), 3), (dict(H=4), 3),
    (dict(H=12), 3), (dict(H=(1 << 20) + 8), 3), (dict(R=-1), 3), (dict(R=1 << 31), 3), (dict(R=1 << 20, H=1 << 17), 3), (dict(act=2), 4),
])
def test_descriptor_refusals(kw, status):
    mok = _mok()
    d = mok.PermuteDesc(**{**dict(T=4, H=16, k=2, R=8), **kw})
    ok = ctypes.c_void_p(4096)
    lib = mok._lib
    assert lib.mok_dispatch_forward(d.c(), ok, ok, ok, None) == status
    assert lib.mok_dispatch_backward(d.c(), ok, ok, ok, ok, None) == status
    assert lib.mok_combine_forward(d.c(), ok, ok, ok, ok, ok, None) == status
    assert lib.mok_combine_backward(d.c(), ok, ok, ok, ok, ok, ok, ok, None) == status


def test_pointer_refusals():
    mok = _mok()
    lib, ok, odd = mok._lib, ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    d = mok.PermuteDesc(4, 16, 2).c()
    for fn, n, must in ((lib.mok_dispatch_forward, 3, (0, 1, 2)), (lib.mok_dispatch_backward, 4, (0, 1, 3)),
                        (lib.mok_combine_forward, 5, (0, 2, 4)), (lib.mok_combine_backward, 7, (0, 1, 3, 5))):
        args = [ok] * n
        for i in must:
            assert fn(d, *args[:i], None, *args[i + 1:], None) == 1, (n, i)
        for i in range(n):
            assert fn(d, *args[:i], odd, *args[i + 1:], None) == 2, (n, i)
        assert fn(None, *args, None) == 1


def test_binding_refusals():
    mok = _mok()
    d = mok.PermuteDesc(4, 16, 2)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for bad in (dict(x=None), dict(x=z(4, 8)), dict(perm=i(4, 2)), dict(perm=i(8).long()), dict(xs=z(4, 16)), dict(xs=z(16, 8).t()), {}):
        with pytest.raises(ValueError):
            mok.dispatch_forward(d, **{**dict(x=z(4, 16), perm=i(8), xs=z(8, 16)), **bad})
    for bad in (dict(o=None), dict(inv=i(8)), dict(gate=z(4, 2)), dict(res=z(8, 16)), {}):
        with pytest.raises(ValueError):
            mok.combine_forward(d, **{**dict(o=z(8, 16), inv=i(4, 2), y=z(4, 16)), **bad})
    for bad in (dict(dy=None), dict(o=None), dict(do=z(4, 16)), {}):
        with pytest.raises(ValueError):
            mok.combine_backward(d, **{**dict(dy=z(4, 16), o=z(8, 16), inv=i(4, 2), do=z(8, 16), dgate=torch.zeros(4, 2)), **bad})
