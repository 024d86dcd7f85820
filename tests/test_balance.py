"""Balance loss of the router with its counts and gradient (mok_balance_forward / _backward)
against the formula in fp64, and its refusals.

Tolerances: exp, the division and the sums of a row's scores (at most 1024, in lane order and
a tree of six) leave a score within some 2^-20 of its value (one of e^-16 and less: |z - m| 2^-24,
the spread here is below 30); a segment's mean adds fp32 sums
of at most ceil(T/512) rows per lane, then fp64. The gradient's bracket c - sum p c is relative
to c + sum p c. A bf16 gradient adds half a step, 2^-8."""
import ctypes

import pytest
import torch

DEV = "cuda"


def _mok():
    from mixture_experts_layer_stable_amd import mok
    return mok


class Run:
    """The operator's outputs, in arrays filled with values that must go."""

    def __init__(self, T, E, k, S, score, grad, coef=0.7, zcoef=0.0):
        mok = self.mok = _mok()
        self.d = mok.BalanceDesc(T, E, k, S=S, score=mok.SCORES[score], grad=mok.DTYPES[grad], coef=coef, zcoef=zcoef)
        n, i32 = max(S, 1), torch.int32
        f = lambda *s: torch.full(s, float("nan"), device=DEV)
        self.loss, self.prob, self.stat = f(2), f(n, E), f(T)
        self.counts = torch.full((n, E), -7, dtype=i32, device=DEV)
        self.tokens = torch.full((n + 2,), -7, dtype=i32, device=DEV)
        self.dz = f(T, E).to(mok.TORCH_DTYPE[mok.DTYPES[grad]])
        self.ws = torch.full((mok.balance_workspace_query(self.d)["fwd_ws"],), 255, dtype=torch.uint8, device=DEV)

    def __call__(self, z, idx, dloss, seg=None, mask=None):
        self.mok.balance_forward(self.d, z, idx, self.loss, self.counts, self.tokens, self.prob, self.stat, self.ws,
                                 seg=seg, mask=mask)
        self.mok.balance_backward(self.d, z, self.counts, self.tokens, self.stat, dloss, self.dz, seg=seg, mask=mask)
        return self.loss, self.counts, self.tokens, self.prob, self.dz


def reference(d, z, idx, dloss, seg=None, mask=None, softmax=True):
    """The definition, segment by segment, in fp64 on the CPU; also the size of each gradient's bracket."""
    z, idx, dloss = z.double().cpu(), idx.cpu().long(), dloss.double().cpu()
    T, E, k = d.T, d.E, d.k
    b = [0, T] if seg is None else seg.cpu().tolist()
    on = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu() != 0
    S = len(b) - 1
    cnt, prob, dz, size = torch.zeros(S, E), torch.zeros(S, E).double(), torch.zeros(T, E).double(), torch.zeros(T, E).double()
    live = [int(on[b[s]:b[s + 1]].sum()) for s in range(S)]
    full, N = sum(n > 0 for n in live), sum(live)
    l0 = l1 = 0.0
    for s in range(S):
        rows = [t for t in range(b[s], b[s + 1]) if on[t]]
        n = len(rows)
        if n == 0:
            continue
        zs = z[rows]
        e = idx[rows].reshape(-1)
        c = torch.bincount(e[(e >= 0) & (e < E)], minlength=E).double()
        if softmax:
            dead = (zs == -float("inf")).all(1)
            p = torch.where(dead[:, None], 0.0, torch.softmax(torch.where(dead[:, None], 0.0, zs), 1))
            lz = torch.where(dead, 0.0, torch.logsumexp(zs, 1))
            slope = torch.ones_like(p)
        else:
            dead = (zs == -float("inf")).all(1)[:, None]   # log sig: no underflow far below 0
            p = torch.where(dead, 0.0, torch.softmax(torch.nn.functional.logsigmoid(torch.where(dead, 0.0, zs)), 1))
            slope, lz = torch.sigmoid(-zs), torch.zeros(n).double()
        cnt[s], prob[s] = c, p.mean(0)
        l0 += E * float((c / (k * n) * p.mean(0)).sum())
        l1 += float((lz * lz).sum())
        dot = (p * c).sum(1, keepdim=True)
        G = dloss[0] * d.coef * E / (full * k * n * n)
        hz = dloss[1] * d.zcoef * 2 / N * lz[:, None] if d.zcoef else torch.zeros(n, 1).double()
        dz[rows] = p * slope * (G * (c - dot) + hz)
        size[rows] = p * slope * (G.abs() * (c + dot) + hz.abs())
    return (d.coef * l0 / max(full, 1), d.zcoef * l1 / max(N, 1)), cnt.int(), live + [full, N], prob, dz, size


def check(run, z, idx, dloss, seg=None, mask=None, softmax=True, bf16=False):
    loss, counts, tokens, prob, dz = run(z, idx, dloss, seg, mask)
    (l0, l1), cnt, tok, p, want, size = reference(run.d, z, idx, dloss, seg, mask, softmax)
    assert torch.equal(counts.cpu(), cnt) and tokens.cpu().tolist() == tok
    assert abs(float(loss[0]) - l0) <= 2e-6 * abs(l0) and abs(float(loss[1]) - l1) <= 2e-6 * abs(l1)
    # a lane adds at most ceil(T/512) rows' p: each fp32 addition is within 2^-24 of the sum
    assert ((prob.double().cpu() - p).abs() <= (2.0**-20 + 2.0**-24 * (run.d.T / 512 + 1)) * p + 1e-30).all()
    tol = 2.0**-18 * size + (1.01 * 2.0**-8 * want.abs() if bf16 else 0) + 1e-37
    off = (dz.double().cpu() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())


def inputs(T, E, k, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * std
    idx = torch.topk(z, k, 1).indices.int() if T else torch.zeros(0, k, dtype=torch.int32)
    return z.to(DEV), idx.to(DEV), torch.tensor([1.25, -0.5], device=DEV), g


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 2, 1), (64, 8, 2), (17, 3, 3), (100, 7, 2), (33, 31, 4),
                                   (1000, 32, 2), (257, 100, 16), (63, 128, 8), (40, 257, 8), (2048, 384, 8), (70, 511, 5),
                                   (19, 1000, 16), (12, 1023, 2), (30, 1024, 8), (9000, 12, 4)])
def test_one_segment(T, E, k):
    print("case balance", T, E, k, flush=True)
    z, idx, dl, _ = inputs(T, E, k, T + E)
    check(Run(T, E, k, 0, "softmax", "f32", zcoef=0.01), z, idx, dl)
    check(Run(T, E, k, 0, "sigmoid", "bf16"), z, idx, dl, softmax=False, bf16=True)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,cuts", [
    (50, 16, 2, [0, 50]), (50, 16, 2, [3, 3, 3, 20, 21, 21, 44]), (1, 9, 3, [0, 0, 1, 1]), (700, 40, 4, [700] * 5),
    (3000, 60, 4, [7, 100, 1000, 1001, 1002, 1002, 1500, 2900]), (513, 384, 8, list(range(0, 513, 8))),
    (40, 5, 1, list(range(41))), (9, 24, 2, [0] * 300 + [9]),
])
def test_ragged_segments_and_masks(T, E, k, cuts, score):
    print("case balance segments", T, E, len(cuts) - 1, score, flush=True)
    z, idx, dl, g = inputs(T, E, k, T * 3 + E)
    S, soft = len(cuts) - 1, score == "softmax"
    seg = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    run = Run(T, E, k, S, score, "f32", zcoef=0.1 if soft else 0.0)
    check(run, z, idx, dl, seg, None, soft)
    for share in (0.7, 0.0):
        mask = (torch.rand(T, generator=g) < share).to(DEV)
        zm, im = z.clone(), idx.clone()
        zm[~mask] = float("nan")     # what does not count is not used
        im[~mask] = 1 << 30
        run = Run(T, E, k, S, score, "bf16", zcoef=0.1 if soft else 0.0)
        check(run, zm, im, dl, seg, mask, soft, bf16=True)
        assert (run.dz[~mask] == 0).all()


@pytest.mark.gpu
def test_far_values_and_dropped_slots():
    """Logits of the type's lowest value, infinities, rows without a finite logit; slots with no expert."""
    T, E, k = 24, 20, 3
    z, idx, dl, _ = inputs(T, E, k, 4)
    z[0, 5:] = -float("inf")
    z[1] = -float("inf")
    z[2] = -3e38
    z[3, 0] = 1000.0
    z[4] = -90.0
    idx[6, 1], idx[7, 2], idx[8, 0] = -1, E, 1 << 30
    for score in ("softmax", "sigmoid"):
        run = Run(T, E, k, 0, score, "f32", zcoef=0.0)
        check(run, z, idx, dl, softmax=score == "softmax")
        assert (run.dz[1] == 0).all()
        check(run, z, idx, torch.tensor([0.5, float("inf")], device=DEV), softmax=score == "softmax")  # no z term
    z[2] = 0.0
    check(Run(T, E, k, 0, "softmax", "f32", zcoef=0.3), z, idx, dl)
    z[9, 3] = float("nan")   # a counted token's NaN reaches its gradient and no other token's
    loss, counts, tokens, prob, dz = Run(T, E, k, 0, "softmax", "f32")(z, idx, dl)
    assert torch.isnan(loss[0]) and torch.isnan(dz[9]).all()
    assert torch.isfinite(dz[:9]).all() and torch.isfinite(dz[10:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_against_autograd_and_differences(score):
    T, E, k = 12, 9, 2
    z, idx, dl, _ = inputs(T, E, k, 9)
    run = Run(T, E, k, 0, score, "f32", coef=1.0, zcoef=0.2 if score == "softmax" else 0.0)
    dz = run(z, idx, dl)[4].double().cpu()
    d, dl64 = run.d, dl.double().cpu()
    f = torch.bincount(idx.cpu().reshape(-1).long(), minlength=E).double() / (T * k)

    def loss(v):
        p = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v) / torch.sigmoid(v).sum(1, keepdim=True)
        return dl64[0] * d.coef * E * (f * p.mean(0)).sum() + dl64[1] * d.zcoef * torch.logsumexp(v, 1).square().mean()

    v = z.double().cpu().requires_grad_()
    want = torch.autograd.grad(loss(v), v)[0]
    assert (dz - want).abs().max() < 2e-6 * want.abs().max()
    v = v.detach()
    for s in range(3):
        u = torch.randn(T, E, generator=torch.Generator().manual_seed(s)).double()
        num = float(loss(v + 1e-5 * u) - loss(v - 1e-5 * u)) / 2e-5
        assert abs(num - float((dz * u).sum())) < 1e-5 * float((dz * u).abs().sum())


@pytest.mark.gpu
def test_follows_the_router_and_repeats():
    """On mok_route's own logits and idx the counts are the schedule's; the same bits twice and
    from a captured graph, replayed between eager calls."""
    mok = _mok()
    T, H, E, k = 500, 256, 24, 3
    g = torch.Generator().manual_seed(0)
    x, wr = torch.randn(T, H, generator=g).bfloat16().to(DEV), torch.randn(E, H, generator=g).bfloat16().to(DEV) / 16
    ld = mok.Desc(T, H, E, k, 128)
    buf = mok.Buffers(ld, backward=False)
    z = torch.empty(T, E, device=DEV)
    mok.route(ld, x, wr, None, buf.idx, buf.gate, z)
    mok.schedule_build(ld, buf.idx, buf.sched)
    dl = torch.tensor([1.0, 2.0], device=DEV)
    run = Run(T, E, k, 0, "softmax", "f32", zcoef=0.1)
    check(run, z, buf.idx, dl)
    assert torch.equal(run.counts[0], buf.schedule_views()["counts"])
    first = [t.clone() for t in run(z, buf.idx, dl)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(z, buf.idx, dl)
    for _ in range(3):
        outs = [run.loss, run.counts, run.tokens, run.prob, run.dz]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))
        again = Run(T, E, k, 0, "softmax", "f32", zcoef=0.1)(z, buf.idx, dl)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.gpu
def test_no_tokens():
    z, idx, dl, _ = inputs(0, 6, 2, 0)
    for S, seg in ((0, None), (3, torch.zeros(4, dtype=torch.int32, device=DEV))):
        run = Run(0, 6, 2, S, "softmax", "f32", zcoef=0.1)
        loss, counts, tokens, prob, dz = run(z, idx, dl, seg)
        assert loss.tolist() == [0, 0] and (counts == 0).all() and (tokens == 0).all() and (prob == 0).all()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    T, E, k = (1 << 22) + 5, 516, 2
    z = torch.zeros(T, E, device=DEV)
    z[:, 3], z[-1, 7], z[T // 2, 9] = 1.0, 4.0, 5.0
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    idx[:, 1] = 3
    idx[-1, 0] = 515
    dl = torch.tensor([1e9, 0.0], device=DEV)   # a gradient of T tokens, in fp32's range
    mok = _mok()
    d = mok.BalanceDesc(T, E, k)
    f, i32 = (lambda *s: torch.empty(*s, device=DEV)), torch.int32
    loss, counts, tokens, prob, stat, dz = f(2), f(1, E).to(i32), f(3).to(i32), f(1, E), f(T), f(T, E)
    ws = torch.empty(mok.balance_workspace_query(d)["fwd_ws"], dtype=torch.uint8, device=DEV)
    mok.balance_forward(d, z, idx, loss, counts, tokens, prob, stat, ws)
    mok.balance_backward(d, z, counts, tokens, stat, dl, dz)
    c = torch.zeros(E, dtype=torch.float64, device=DEV)
    c[0], c[3], c[515] = T - 1, T, 1
    assert torch.equal(counts[0].double(), c) and tokens.tolist() == [T, 1, T]
    rows = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    p = torch.softmax(z[rows].double(), 1)
    want = 1e9 * E / (k * float(T) ** 2) * p * (c - (p * c).sum(1, keepdim=True))
    size = 1e9 * E / (k * float(T) ** 2) * p * (c + (p * c).sum(1, keepdim=True))
    assert ((dz[rows].double() - want).abs() <= 2.0**-18 * size).all()
    base = torch.softmax(z[0].double(), 0)
    # every lane adds T/1024/16 rows' equal p in fp32
    assert ((prob[0].double() - base).abs() <= (2.0**-20 + T / 16384 * 2.0**-24) * base + 2.0 / T).all()


# ---- refusals (no GPU needed) ----

@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 3), (dict(T=1 << 31), 3), (dict(E=0), 3), (dict(E=1025), 3), (dict(k=0), 3), (dict(k=9), 3),
    (dict(E=64, k=17), 3), (dict(T=1 << 28, k=8), 3), (dict(S=-1), 3), (dict(S=65536), 3), (dict(score=2), 4), (dict(grad=2), 4),
    (dict(coef=float("nan")), 3), (dict(zcoef=float("inf")), 3), (dict(score=1, zcoef=0.1), 3),
])
def test_descriptor_refusals(kw, status):
    mok = _mok()
    with pytest.raises(mok.MokError) as ei:
        mok.balance_workspace_query(mok.BalanceDesc(**{**dict(T=4, E=8, k=2), **kw}))
    assert ei.value.status == status


def test_pointer_refusals():
    mok = _mok()
    lib, ok, odd = mok._lib, ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    d = mok.BalanceDesc(4, 8, 2, S=1)
    n = mok.balance_workspace_query(d)["fwd_ws"]
    args = [ok] * 10
    assert lib.mok_balance_forward(d.c(), *args, n - 1, None) == 6
    for i, st in ((0, 1), (1, 1), (2, 1), (4, 1), (5, 1), (6, 1), (7, 1), (8, 1), (9, 1)):
        assert lib.mok_balance_forward(d.c(), *args[:i], None, *args[i + 1:], n, None) == st, i
        assert lib.mok_balance_forward(d.c(), *args[:i], odd, *args[i + 1:], n, None) == 2, i
    assert lib.mok_balance_forward(d.c(), *args[:3], odd, *args[4:], n, None) == 2
    args = [ok] * 8
    for i in (0, 1, 3, 4, 5, 6, 7):
        assert lib.mok_balance_backward(d.c(), *args[:i], None, *args[i + 1:], None) == 1, i


def test_binding_refusals():
    mok = _mok()
    d = mok.BalanceDesc(4, 8, 2, S=2)
    f, i = torch.zeros, torch.int32
    good = dict(logits=f(4, 8), idx=f(4, 2, dtype=i), loss=f(2), counts=f(2, 8, dtype=i), tokens=f(4, dtype=i),
                prob=f(2, 8), stat=f(4), ws=f(1 << 16, dtype=torch.uint8), seg=f(3, dtype=i))
    for bad in (dict(idx=f(4, 2, dtype=torch.int64)), dict(seg=None), dict(seg=f(4, dtype=i)), dict(mask=f(4)),
                dict(counts=f(8, dtype=i)), dict(logits=f(8, 4).t()), dict(logits=None), dict()):
        with pytest.raises(ValueError):
            mok.balance_forward(d, **{**good, **bad})
