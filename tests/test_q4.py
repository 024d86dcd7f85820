"""Products with 4-bit weights and group scales (mok_q4_forward), dense and grouped by expert, against the formula in
fp64, the quantiser (mok_q4_quantize) bit for bit, and their refusals.

Tolerances: the formula is a sum over groups of s times fp32 sums of exact products. In bf16 the codes enter as 16 + q
and z + 16 times the sum of x is taken off again, so what fp32 errors are relative to is
s * sum |x| (32 + q + z) (fp32: s * sum |x| |q - z|); sum_tol(K) of test_linear.py of that covers sums of K terms in any
order. w itself is not rounded. A bf16 output adds half a step, 2^-8 of the value."""
import ctypes

import pytest
import torch

from test_linear import DEV, _mok, act64, near, sum_tol

KEEP = 77.0


class Case:
    """counts: rows of the groups, or a number of rows for a dense product."""

    def __init__(self, counts, N, K, group, act, epi, zeros, lead=0, tail=0, seed=0):
        mok = self.mok = _mok()
        self.t = t = mok.TORCH_DTYPE[mok.DTYPES[act]]
        self.dense = isinstance(counts, int)
        cl = [counts] if self.dense else counts
        E, M = len(cl), lead + sum(cl) + tail
        self.d = d = mok.Q4Desc(M, N, K, E, group, act=mok.DTYPES[act], epi=mok.EPILOGUES[epi])
        self.epi = epi
        self.off = [lead]
        for n in cl:
            self.off.append(self.off[-1] + n)
        g = torch.Generator().manual_seed(seed + M * 31 + N * 7 + K + E + group)
        n = lambda *s: torch.randn(*s, generator=g)
        P = d.P
        self.x, self.bias, self.res = n(M, K).to(t), n(E, P), n(M, N).to(t)
        self.code = torch.randint(0, 16, (E, P, K), generator=g, dtype=torch.uint8)
        self.q = self.code[..., 0::2] | self.code[..., 1::2] << 4
        self.s = (torch.exp(n(E, P, K // group) * 0.5) * 0.2 * K**-0.5 * torch.sign(n(E, P, K // group))).to(t)
        self.z = torch.randint(0, 16, (E, P, K // group), generator=g, dtype=torch.uint8) if zeros else None
        self.out = torch.ones(M, dtype=torch.bool)
        self.out[self.off[0]:self.off[-1]] = False
        for v in (self.x, self.res):
            v[self.out] = float("nan")
        self.goff = None if self.dense else torch.tensor(self.off, dtype=torch.int32, device=DEV)

    def forward(self, bias=True, res=True):
        d, dev = self.d, lambda v: v.to(DEV)
        y = torch.full((d.M, d.N), KEEP, dtype=self.t, device=DEV)
        ws = torch.full((max(self.mok.q4_workspace_query(d)["fwd_ws"], 16),), 255, dtype=torch.uint8, device=DEV)
        self.mok.q4_forward(d, dev(self.x), dev(self.q), dev(self.s), y, z=None if self.z is None else dev(self.z),
                            off=self.goff, bias=dev(self.bias) if bias else None, res=dev(self.res) if res else None, ws=ws)
        return y

    def check(self, bias=True, res=True):
        y, d, N = self.forward(bias, res).cpu(), self.d, self.d.N
        assert (y[self.out] == KEEP).all()
        for e in range(d.E):
            r = slice(self.off[e], self.off[e + 1])
            if r.start == r.stop:
                continue
            x = self.x[r].double()
            s = self.s[e].double().repeat_interleave(d.group, 1)
            z = self.z[e].double().repeat_interleave(d.group, 1) if self.z is not None else 8.0
            q = self.code[e].double()
            b = self.bias[e].double() if bias else torch.zeros(())
            p = x @ (s * (q - z)).t() + b
            big = s.abs() * (32 + q + z if self.t is torch.bfloat16 else (q - z).abs())
            err = sum_tol(d.K) * (x.abs() @ big.t() + b.abs())
            f = act64(self.epi, p)
            ef = 1.13 * err[:, :N] * p[:, N:].abs() + p[:, :N].abs() * err[:, N:] if self.epi == "swiglu" else 1.13 * err
            add = self.res[r].double() if res else torch.zeros(())
            near(y[r], f + add, ef + 2.0**-20 * (f.abs() + add.abs()), ("y", e))


# rows, N, K, group
DENSE = [(1, 8, 32, 32), (1, 24, 64, 64), (1, 40, 128, 128), (2, 136, 160, 32), (3, 1000, 192, 64), (1, 264, 4096, 128),
         (7, 72, 1152, 128), (16, 200, 96, 32), (17, 72, 320, 64), (31, 136, 2048, 128), (32, 520, 608, 32), (33, 24, 1024, 64),
         (64, 256, 256, 128), (65, 264, 384, 64), (130, 520, 160, 32), (300, 136, 1280, 128), (1, 8, 16384, 128), (257, 1032, 64, 32),
         (129, 128, 7168, 128), (512, 384, 352, 32)]
GROUPS = [([1], 24, 64, 32, 0, 2), ([0, 0, 2, 0], 40, 128, 128, 1, 0), ([3, 1, 0, 2], 136, 192, 64, 2, 3), ([17] * 5, 72, 160, 32, 0, 0),
          ([1, 0, 0, 1, 1] * 30, 64, 384, 128, 1, 1), ([64, 65, 0, 63, 1], 264, 320, 64, 5, 5), ([0] * 90 + [9] + [0] * 81, 16, 256, 128, 3, 3),
          ([300, 5, 0, 130], 72, 640, 128, 0, 7), ([200, 3, 257], 264, 288, 32, 1, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("epi", ["none", "silu", "gelu", "swiglu"])
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_dense(act, epi):
    for i, (M, N, K, G) in enumerate(DENSE):
        print("case q4", M, N, K, G, act, epi, flush=True)
        c = Case(M, N, K, G, act, epi, zeros=i % 2 == 0)
        c.check()
        c.check(bias=False, res=False)


@pytest.mark.gpu
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("act,epi", [("bf16", "none"), ("bf16", "swiglu"), ("f32", "gelu"), ("f32", "swiglu"), ("bf16", "silu")])
def test_grouped(act, epi, zeros):
    for counts, N, K, G, lead, tail in GROUPS:
        print("case q4 grouped", len(counts), sum(counts), N, K, G, act, epi, zeros, flush=True)
        c = Case(counts, N, K, G, act, epi, zeros, lead, tail)
        c.check()
        c.check(bias=False, res=False)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,G", [(1000, 512, 1024, 128), (2048, 264, 544, 32), (700, 2048, 256, 64), (4096, 136, 128, 128)])
def test_many_rows(M, N, K, G):
    for act, epi in (("bf16", "none"), ("bf16", "swiglu"), ("f32", "none")):
        print("case q4 many rows", M, N, K, G, act, epi, flush=True)
        Case(M, N, K, G, act, epi, zeros=epi == "none").check()


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K,G", [([1, 3, 0, 16] * 40, 520, 256, 128),    # a tile of w a wave
                                          ([2, 1, 0, 5] * 12, 520, 288, 32),       # two waves a tile
                                          ([16, 9, 1] * 8, 776, 4352, 64),         # two waves, x in stages
                                          ([16, 12] * 34, 968, 4352, 128),         # one wave, x in stages
                                          ([20, 40, 3, 0, 17], 136, 1088, 64)])    # groups of more than 16 rows
def test_few_rows_of_many_groups(counts, N, K, G):
    for act, epi in (("bf16", "swiglu"), ("f32", "none")) if K < 2000 else (("bf16", "none"),):
        print("case q4 many groups", len(counts), sum(counts), N, K, G, act, epi, flush=True)
        Case(counts, N, K, G, act, epi, zeros=True, tail=2).check(bias=False)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 320])
def test_tiles_of_groups_of_32_that_end_in_half_a_k_tile(K):
    for counts in ([20001], [9000, 0, 11001]):
        print("case q4 half K-tile", K, len(counts), flush=True)
        Case(counts, 264, K, 32, "bf16", "none", zeros=True).check()


@pytest.mark.gpu
@pytest.mark.parametrize("G", [32, 64, 128])
def test_tiles_of_ragged_groups(G):
    for epi in ("none", "swiglu"):
        print("case q4 tiles", G, epi, flush=True)
        Case([700, 3, 0, 900, 129], 1032, 1920 if G == 128 else 2016 // G * G, G, "bf16", epi, zeros=epi == "none", lead=3, tail=5).check()


@pytest.mark.gpu
def test_infinite_weights_and_rows():
    """An infinite scale reaches its group of rows of w only, a row of x that is not finite its row of y only."""
    for M in (5, 600):
        c = Case(M, 72, 256, 64, "bf16", "none", True)
        clean = c.forward(bias=False, res=False).cpu()
        c.s[0, 7, 1] = float("inf")
        c.x[3, 100] = float("inf")
        c.x[4, 0] = float("nan")
        got = c.forward(bias=False, res=False).cpu()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[3:5] = False
        keep[:, 7] = False
        assert torch.equal(got[keep], clean[keep])
        assert not torch.isfinite(got[:, 7]).any() and torch.isnan(got[4]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,N,K,group", [
    (5, 72, 256, 64), (5, 24, 128, 128), (3, 40, 96, 32), (16, 136, 1088, 64), (3, 72, 1152, 128), (2, 24, 32, 32),  # few rows
    ([4] * 40, 520, 288, 32), ([3, 0, 16] * 12, 520, 320, 64),                  # one and two waves on a tile of w
    ([16, 3], 264, 2112, 64), ([16] * 12, 776, 2080, 32), ([16, 3, 16, 16] * 10, 1032, 2176, 128),  # x in stages
    (700, 2056, 96, 32), (700, 520, 2112, 64), ([700, 3, 900], 1032, 640, 128)])  # tiles, also in slices of K
def test_infinities_in_fp32_rows_are_the_formulas(rows, N, K, group):
    """An infinity in x gives sum_k x w as fp32 arithmetic has it: an infinity of w's sign there, NaN where w is 0, wherever
    in K it lies, the last piece of 128 of it included. It stays in its row."""
    c = Case(rows, N, K, group, "f32", "none", True)
    print("case q4 infinities", c.d.M, N, K, group, flush=True)
    clean, want = c.forward(bias=False, res=False).cpu(), {}
    for e in range(c.d.E):
        at = [0, K // 2, K - 1, max(K - 128, 0), (K - 1) // 128 * 128]
        for i, (r, k) in enumerate(zip(range(c.off[e], c.off[e + 1]), at)):
            inf = float("inf") if (i + e) % 2 else -float("inf")
            c.x[r, k] = inf
            w = c.s[e, :, k // group] * (c.code[e, :, k].float() - c.z[e, :, k // group].float())
            want[r] = w * inf
    got = c.forward(bias=False, res=False).cpu()
    keep = torch.ones(c.d.M, dtype=torch.bool)
    for r, v in want.items():
        keep[r] = False
        assert torch.equal(torch.isnan(got[r]), torch.isnan(v)), r
        assert torch.equal(torch.nan_to_num(got[r], nan=0.0), torch.nan_to_num(v, nan=0.0)), r
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_code_and_zero_point_alone(group):
    """x = one unit vector: y is s (code - z) exactly (bf16: |code - z| s has at most 12 bits, rounded once)."""
    mok = _mok()
    K, N, M = 2 * group, 256, 24
    code = (torch.arange(N)[:, None] + torch.arange(K)[None, :]) % 16
    z = ((torch.arange(N) // 16)[:, None] + torch.zeros(1, 2)).to(torch.uint8)
    s = torch.exp2((torch.arange(N) % 5 - 2).float())[:, None].repeat(1, 2) * torch.tensor([[1.0, -1.5]])
    q = (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8)
    for act in (mok.BF16, mok.F32):
        t = mok.TORCH_DTYPE[act]
        x = torch.zeros(M, K)
        at = torch.arange(M) * 7 % K
        x[torch.arange(M), at] = 1.0
        y = torch.empty(M, N, dtype=t, device=DEV)
        d = mok.Q4Desc(M, N, K, 1, group, act=act)
        dev = lambda v: v.to(DEV)
        mok.q4_forward(d, dev(x.to(t)), dev(q[None]), dev(s.to(t)[None]), y, z=dev(z[None]))
        want = (s.repeat_interleave(group, 1) * (code - z.repeat_interleave(group, 1).float()))[:, at].t()
        assert torch.equal(y.cpu(), want.to(t))


def quantize64(w, group, zeros, t):
    v = w.float().view(*w.shape[:-1], -1, group)
    lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
    s = ((hi - lo) / 15 if zeros else torch.maximum(-lo, hi) / 7).to(t)
    sf = s.float()
    on = sf > 0
    safe = torch.where(on, sf, torch.ones(()))
    z = torch.where(on, torch.round(-lo / safe).clamp(0, 15), torch.full((), 8.0)) if zeros else torch.full_like(sf, 8.0)
    c = (torch.round(v / safe[..., None]) + z[..., None]).clamp(0, 15)
    c = torch.where(on[..., None], c, z[..., None]).view(w.shape).to(torch.uint8)
    return c[..., 0::2] | c[..., 1::2] << 4, s, z.to(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(group, act):
    """The codes, scales and zero points of the definition, bit for bit (fp32 divisions and roundings are exact steps
    of it); what they stand for is within half a scale of w, and half a step of the scale's rounding times the code."""
    mok = _mok()
    t = mok.TORCH_DTYPE[mok.DTYPES[act]]
    for E, N, K, epi in ((1, 8, group, "none"), (3, 40, 5 * group, "swiglu"), (2, 264, 2 * group, "none")):
        d = mok.Q4Desc(0, N, K, E, group, act=mok.DTYPES[act], epi=mok.EPILOGUES[epi])
        P = d.P
        g = torch.Generator().manual_seed(K + N)
        w = torch.randn(E, P, K, generator=g)
        w[0, 0, :group] = 0.0                                  # a group of zeros
        w[0, 1] = w[0, 1].abs()                                # of one sign
        w[0, 2] = -w[0, 2].abs()
        w[0, 3, :group] = torch.arange(group) % 15 - 7.0       # codes at their ends, ties
        w[0, 4, :group] = torch.arange(group) * 0.5
        w[-1, -1] *= 1e-30
        w = w.to(t)
        for zeros in (False, True):
            print("case q4 quantize", E, P, K, group, act, zeros, flush=True)
            q = torch.full((E, P, K // 2), 255, dtype=torch.uint8, device=DEV)
            s = torch.full((E, P, K // group), KEEP, dtype=t, device=DEV)
            z = torch.full((E, P, K // group), 255, dtype=torch.uint8, device=DEV) if zeros else None
            mok.q4_quantize(d, w.to(DEV), q, s, z)
            wq, wsc, wz = quantize64(w, group, zeros, t)
            assert torch.equal(s.cpu(), wsc) and torch.equal(q.cpu(), wq)
            if zeros:
                assert torch.equal(z.cpu(), wz)
            code = torch.stack([wq & 15, wq >> 4], -1).flatten(-2).double()
            sg = wsc.double().repeat_interleave(group, -1)
            back = sg * (code - wz.double().repeat_interleave(group, -1))
            # zero points move a group's ends by half a step each, as does the scale's rounding of 15 steps
            slack = (1.0 if zeros else 0.5) + 15 * {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}[t]
            assert ((back - w.double()).abs() <= slack * sg * 1.01 + 1e-37).all()


@pytest.mark.gpu
def test_quantised_weights_run():
    """q4_quantize's arrays in q4_forward: a product with the weights that they stand for."""
    mok = _mok()
    for act in ("bf16", "f32"):
        t = mok.TORCH_DTYPE[mok.DTYPES[act]]
        d = mok.Q4Desc(5, 64, 256, 2, 64, act=mok.DTYPES[act])
        w = torch.randn(2, 64, 256, device=DEV).to(t)
        q, s, z = torch.empty(2, 64, 128, dtype=torch.uint8, device=DEV), torch.empty(2, 64, 4, dtype=t, device=DEV), torch.empty(2, 64, 4, dtype=torch.uint8, device=DEV)
        mok.q4_quantize(d, w, q, s, z)
        x, y = torch.randn(5, 256, device=DEV).to(t), torch.empty(5, 64, dtype=t, device=DEV)
        mok.q4_forward(d, x, q, s, y, z=z, off=torch.tensor([0, 3, 5], dtype=torch.int32, device=DEV))
        want = torch.cat([x[:3].double() @ w[0].double().t(), x[3:].double() @ w[1].double().t()])
        # half a step of about |w|max 2 / 15 in each of 256 products of random signs, five times its root sum of squares
        assert ((y.double() - want).abs() < 5 * 0.5 * (2 * 3.5 / 15) * 16).all()


@pytest.mark.gpu
def test_rows_and_groups_do_not_touch_each_other():
    c = Case([5, 40, 3, 100], 72, 128, 32, "bf16", "none", True, lead=1, tail=1)
    clean = c.forward(bias=False, res=False).cpu()
    lo, hi = c.off[1], c.off[2]
    c.x[lo:hi] = float("nan")
    c.s[1] = float("inf")
    c.x[c.off[3] + 7] = float("inf")
    got = c.forward(bias=False, res=False).cpu()
    keep = torch.ones(c.d.M, dtype=torch.bool)
    keep[lo:hi] = False
    keep[c.off[3] + 7] = False
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.gpu
def test_offsets_that_descend_or_pass_the_rows_stay_inside():
    mok = _mok()
    for M in (60, 400):
        N, K, E = 40, 128, 6
        for off in ([-5, 70, 10, 200, -1, 3, 1 << 30], [60, 50, 40, 30, 20, 10, 0], [(1 << 31) - 1] * 7):
            print("case q4 bad offsets", M, off, flush=True)
            d = mok.Q4Desc(M, N, K, E, 32)
            y = torch.ones(M + 2, N, dtype=torch.bfloat16, device=DEV)
            mok.q4_forward(d, torch.zeros(M, K, dtype=torch.bfloat16, device=DEV), torch.zeros(E, N, K // 2, dtype=torch.uint8, device=DEV),
                           torch.zeros(E, N, 4, dtype=torch.bfloat16, device=DEV), y[1:-1], off=torch.tensor(off, dtype=torch.int32, device=DEV))
            assert (y[0] == 1).all() and (y[-1] == 1).all()


@pytest.mark.gpu
def test_in_place_captured_and_on_another_stream():
    for counts, dense in (([5, 0, 30, 1], False), (1, True), (600, True)):
        c = Case(counts, 264, 512, 128, "bf16", "swiglu", True)
        dev = lambda v: v.to(DEV)
        want, same = c.forward(), dev(c.res).clone()
        x, q, s, z, b, r = (dev(v) for v in (c.x, c.q, c.s, c.z, c.bias, c.res))
        ws = torch.empty(max(c.mok.q4_workspace_query(c.d)["fwd_ws"], 16), dtype=torch.uint8, device=DEV)
        c.mok.q4_forward(c.d, x, q, s, same, z=z, off=c.goff, bias=b, res=same, ws=ws)
        assert torch.equal(want, same)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            other = c.forward()
        st.synchronize()
        assert torch.equal(want, other)
        y = torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.mok.q4_forward(c.d, x, q, s, y, z=z, off=c.goff, bias=b, res=r, ws=ws)
        for _ in range(3):
            x.mul_(0.75)
            eager = torch.empty_like(y)
            c.mok.q4_forward(c.d, x, q, s, eager, z=z, off=c.goff, bias=b, res=r, ws=ws)
            y.fill_(KEEP)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(eager, y)


@pytest.mark.gpu
def test_codes_past_32_bits():
    """Codes of more than 2^32 bytes: the last expert's rows and columns."""
    mok = _mok()
    E, N, K = 9, 4096, 1 << 18
    print("case q4 large", E, N, K, flush=True)
    q = torch.full((E, N, K // 2), 0x88, dtype=torch.uint8, device=DEV)
    q[E - 1, N - 1] = 0x99
    s = torch.ones(E, N, K // 128, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(2, K, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(2, N, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0] * E + [2], dtype=torch.int32, device=DEV)
    mok.q4_forward(mok.Q4Desc(2, N, K, E, 128), x, q, s, y, off=off)
    assert (y[:, -1] == K).all() and float(y.float().sum()) == 2.0 * K


# ---- refusals (no GPU needed) ----

@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 3), (dict(M=1 << 30), 3), (dict(N=0), 3), (dict(N=12), 3), (dict(K=96), 3), (dict(K=0), 3), (dict(group=16), 3),
    (dict(group=0), 3), (dict(group=256, K=256), 3), (dict(E=0), 3), (dict(E=1025), 3), (dict(N=1 << 20, K=1 << 20), 3),
    (dict(act=2), 4), (dict(epi=4), 4), (dict(flags=1), 3),
])
def test_descriptor_refusals(kw, status):
    mok = _mok()
    with pytest.raises(mok.MokError) as ei:
        mok.q4_workspace_query(mok.Q4Desc(**{**dict(M=4, N=16, K=128), **kw}))
    assert ei.value.status == status


def test_pointer_refusals():
    mok = _mok()
    lib, ok, odd = mok._lib, ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    d = mok.Q4Desc(300, 16, 4096, 3).c()
    args = [ok] * 9
    big = 1 << 40
    for i in (0, 1, 2, 5, 7):
        assert lib.mok_q4_forward(d, *args[:i], None, *args[i + 1:], big, None) == 1, i
    for i in range(8):
        assert lib.mok_q4_forward(d, *args[:i], odd, *args[i + 1:], big, None) == 2, i
    args = [ok] * 4
    for i in (0, 1, 2):
        assert lib.mok_q4_quantize(d, *args[:i], None, *args[i + 1:], None) == 1, i
    for i in range(4):
        assert lib.mok_q4_quantize(d, *args[:i], odd, *args[i + 1:], None) == 2, i
    assert lib.mok_q4_workspace_query(d, None) == 1


def test_binding_refusals():
    mok = _mok()
    d = mok.Q4Desc(4, 16, 64, 2, 32)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    u = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    off = torch.zeros(3, dtype=torch.int32)
    good = dict(x=z(4, 64), q=u(2, 16, 32), s=z(2, 16, 2), y=z(4, 16), off=off)
    for bad in (dict(x=None), dict(q=u(2, 16, 64)), dict(s=z(2, 16, 2).float()), dict(z=u(2, 16, 1)), dict(off=None), dict(y=z(4, 8)), dict()):
        with pytest.raises(ValueError):
            mok.q4_forward(d, **{**good, **bad})
    with pytest.raises(ValueError):
        mok.q4_quantize(d, z(2, 16, 64), u(2, 16, 64), z(2, 16, 2))
