"""RMS norm with the residual's addition (mok_rmsnorm_forward / _backward) against the
formula in fp64, its MX rows against the layer's own quantiser, and its refusals.

Tolerances: a bf16 output is one rounding (2^-8 relative, half a step) of an fp32 result whose
own error is some 1e-6; fp32 sums over at most 32768 elements in tree order stay within
2^-24 * (8 + 15) of the sum of magnitudes."""
import ctypes
import os

import numpy as np
import pytest
import torch

DEV = "cuda"
HALF = {torch.bfloat16: 2.0**-8, torch.float32: 2.0**-24}


def _mok():
    from mixture_experts_layer_stable_amd import mok
    return mok


def _close(got, ref, scale=None, extra=0.0):
    """Every element within half a step of its own type plus fp32 arithmetic noise, which is
    relative to `scale` (the magnitudes that were added; default the value itself)."""
    ref = ref.double().cpu()
    got64 = got.double().cpu()
    scale = ref.abs() if scale is None else scale.double().cpu()
    tol = HALF[got.dtype] * ref.abs() * 1.01 + (2.0**-18 + extra) * scale + 1e-30
    bad = (got64 - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got64 - ref).abs() / tol).max()))


def _reference(x, res, w, eps):
    v = x.double() + (0 if res is None else res.double())
    rstd = 1 / torch.sqrt(v.square().mean(-1) + eps)
    return v, rstd, v * rstd[:, None] * w.double()


def _inputs(T, H, t, seed, res=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)
    gain = torch.exp(n(H))
    x, w = (n(T, H) * gain).to(t), (1 + 0.2 * n(H)).to(t)
    return x.to(DEV), ((3 * n(T, H) * gain).to(t).to(DEV) if res else None), w.to(DEV), n(T, H).to(t).to(DEV), \
        n(T, H).to(t).to(DEV)


SHAPES = [(1, 8), (3, 24), (5, 128), (64, 136), (33, 512), (7, 1000), (300, 1024), (9, 2048), (2, 2056), (130, 7168),
          (3, 16392), (2, 32768), (1031, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward_and_backward(T, H, act):
    mok = _mok()
    print("case norm", T, H, act, flush=True)
    t = mok.TORCH_DTYPE[mok.DTYPES[act]]
    for with_res in (True, False):
        x, res, w, dy, dr = _inputs(T, H, t, T * 7 + H, with_res)
        d = mok.NormDesc(T, H, act=mok.DTYPES[act], eps=1e-5)
        r, y, dx = (torch.full((T, H), float("nan"), dtype=t, device=DEV) for _ in range(3))
        rstd = torch.full((T,), float("nan"), device=DEV)
        dw = torch.full((H,), float("nan"), dtype=t, device=DEV)
        ws = torch.full((max(mok.norm_workspace_query(d)["bwd_ws"], 16),), 255, dtype=torch.uint8, device=DEV)
        mok.rmsnorm_forward(d, x, w, y=y, res=res, r=r, rstd=rstd)
        v, rs, want = _reference(x, res, w, 1e-5)
        _close(r, v)
        _close(rstd, rs)
        _close(y, want)
        # backward from the forward's own r and rstd
        xh = r.double() * rstd.double()[:, None]
        g = dy.double() * w.double()
        c = (g * xh).mean(-1, keepdim=True)
        for drv in (dr, None):
            mok.rmsnorm_backward(d, dy, r, w, rstd, dx, dw=dw, dr=drv, ws=ws)
            d64 = 0 if drv is None else drv.double()
            size = rs[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True)) + \
                (0 if drv is None else d64.abs())
            _close(dx, d64 + rstd.double()[:, None] * (g - xh * c), size)
            _close(dw, (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0))


@pytest.mark.gpu
def test_backward_is_the_gradient():
    """dx and dw against fp64 autograd of the forward and against differences of its loss."""
    mok = _mok()
    T, H = 6, 40
    x, res, w, dy, dr = _inputs(T, H, torch.float32, 3)
    d = mok.NormDesc(T, H, act=mok.F32, eps=1e-4)
    r, y, dx, rstd, dw = x.clone(), x.clone(), x.clone(), x[:, 0].clone().contiguous(), w.clone()
    ws = torch.empty(mok.norm_workspace_query(d)["bwd_ws"], dtype=torch.uint8, device=DEV)
    mok.rmsnorm_forward(d, x, w, y=y, res=res, r=r, rstd=rstd)
    mok.rmsnorm_backward(d, dy, r, w, rstd, dx, dw=dw, dr=dr, ws=ws)
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()

    def loss(xv, wv):
        v, _, yv = _reference(xv, res, wv, 1e-4)
        return (yv * dy.double()).sum() + (v * dr.double()).sum()

    gx, gw = torch.autograd.grad(loss(x64, w64), (x64, w64))
    assert (dx.double() - gx).abs().max() < 1e-5 * gx.abs().max()
    assert (dw.double() - gw).abs().max() < 1e-5 * gw.abs().max()
    for k in range(4):
        u = torch.randn(T, H, generator=torch.Generator().manual_seed(k)).double().to(DEV)
        num = (loss(x64 + 1e-5 * u, w64) - loss(x64 - 1e-5 * u, w64)) / 2e-5
        assert abs(float(num - (dx.double() * u).sum())) < 1e-4 * float((dx.double().abs() * u.abs()).sum())


@pytest.mark.gpu
def test_in_place_rows_and_repeats():
    """r over x, y over res, dx over dy; the same bits as with separate arrays, twice."""
    mok = _mok()
    T, H = 77, 1024
    x, res, w, dy, dr = _inputs(T, H, torch.bfloat16, 5)
    d = mok.NormDesc(T, H)
    ws = torch.empty(mok.norm_workspace_query(d)["bwd_ws"], dtype=torch.uint8, device=DEV)
    r, y, dx = (torch.empty_like(x) for _ in range(3))
    rstd, dw, dw2 = torch.empty(T, device=DEV), torch.empty_like(w), torch.empty_like(w)
    mok.rmsnorm_forward(d, x, w, y=y, res=res, r=r, rstd=rstd)
    mok.rmsnorm_backward(d, dy, r, w, rstd, dx, dw=dw, dr=dr, ws=ws)
    x2, res2, dy2, rstd2 = x.clone(), res.clone(), dy.clone(), torch.empty(T, device=DEV)
    mok.rmsnorm_forward(d, x2, w, y=res2, res=res2, r=x2, rstd=rstd2)
    mok.rmsnorm_backward(d, dy2, x2, w, rstd2, dy2, dw=dw2, dr=dr, ws=ws)
    for a, b in ((r, x2), (y, res2), (rstd, rstd2), (dx, dy2), (dw, dw2)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_zero_and_extreme_rows():
    """A zero row is 0 with rstd = 1/sqrt(eps); a NaN or infinite row leaves the others alone."""
    mok = _mok()
    T, H = 5, 256
    x = torch.ones(T, H, device=DEV)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 4] = float("inf")
    x[4] = 1e-30
    d = mok.NormDesc(T, H, act=mok.F32, eps=1e-6)
    y, rstd = torch.empty_like(x), torch.empty(T, device=DEV)
    mok.rmsnorm_forward(d, x, torch.ones(H, device=DEV), y=y, rstd=rstd)
    assert (y[1] == 0).all() and abs(float(rstd[1]) - 1e3) < 1e-2
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 4]) and (y[3, :4] == 0).all()
    _close(y[0], torch.full((H,), 1 / (1 + 1e-6) ** 0.5, dtype=torch.float64))
    assert (y[4] > 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("T,H", [(1, 256), (37, 1024), (130, 7168), (5, 16640)])
def test_mx_rows_are_the_layers_own(T, H, fmt):
    """q and s are the oracle quantiser's blocks of the stored bf16 y, bit for bit, with and
    without y itself being written."""
    import oracle as orc
    mok = _mok()
    x, res, w, _, _ = _inputs(T, H, torch.bfloat16, T + H)
    x[0, :32] = 0
    if res is not None:
        res[0, :32] = 0
    hq = H // 2 if fmt == "mxfp4" else H
    d = mok.NormDesc(T, H, quant=mok.DTYPES[fmt])
    y = torch.empty_like(x)
    outs = []
    for yy in (y, None):
        q = torch.full((T, hq), 99, dtype=torch.uint8, device=DEV)
        s = torch.full((H // 128, T, 4), 99, dtype=torch.uint8, device=DEV)
        mok.rmsnorm_forward(d, x, w, y=yy, res=res, q=q, s=s)
        outs.append((q.cpu(), s.cpu()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    el, sc = orc.mx.mx_quantize(y.double().cpu().numpy(), -1, fmt="e4m3" if fmt == "mxfp8" else "e2m1")
    got_s = outs[0][1].numpy().astype(np.int64).transpose(1, 0, 2).reshape(sc.shape) - 127
    np.testing.assert_array_equal(got_s, sc)
    if fmt == "mxfp8":
        got = outs[0][0].view(torch.float8_e4m3fn).double().numpy()
    else:
        b = outs[0][0].numpy()
        code = np.stack([b & 15, b >> 4], -1).reshape(T, H)
        got = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[code & 7] * np.where(code & 8, -1.0, 1.0)
    np.testing.assert_array_equal(np.abs(got), np.abs(el))
    np.testing.assert_array_equal(got, el + 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_norm_feeds_the_mx_layer(fmt):
    """The MX forward on rows that the norm has quantised into its workspace (FLAG_X_QUANT)
    gives the bits of the forward that quantises y itself, for each slot of the ring."""
    mok = _mok()
    T, H, E, k, I = 96, 512, 8, 2, 256
    x, res, w, _, _ = _inputs(T, H, torch.bfloat16, 11)
    g = torch.Generator().manual_seed(2)
    w1 = (torch.randn(E, 2 * I, H, generator=g) * H**-0.5).bfloat16().to(DEV)
    w2 = (torch.randn(E, H, I, generator=g) * I**-0.5).bfloat16().to(DEV)
    wr = (torch.randn(E, H, generator=g) * H**-0.5).bfloat16().to(DEV)
    for mb in (0, 1):
        d = mok.Desc(T, H, E, k, I, gemm=mok.DTYPES[fmt], mb_count=2, mb_index=mb, ring=2)
        mxw = mok.MxWeights(d)
        mok.weights_quantize(d, w1, w2, mxw)
        buf = mok.Buffers(d, backward=False)
        y, out = torch.empty_like(x), torch.empty_like(x)
        nd = mok.NormDesc(T, H, quant=mok.DTYPES[fmt])
        q, s = mok.x_quant_views(d, buf.fwd_ws)
        mok.rmsnorm_forward(nd, x, w, y=y, res=res, q=q, s=s)
        mok.route(d, y, wr, None, buf.idx, buf.gate)
        mok.schedule_build(d, buf.idx, buf.sched)
        dq = mok.Desc(**{**d.__dict__, "flags": mok.FLAG_X_QUANT})
        mok.moe_forward(dq, buf.sched, None, buf.gate, None, None, out, buf.saved, buf.fwd_ws, mxw=mxw)
        mok.moe_forward(d, buf.sched, y, buf.gate, None, None, buf.y, buf.saved, buf.fwd_ws, mxw=mxw)
        mok.check_schedule(d, buf.sched)
        assert torch.equal(out, buf.y)


@pytest.mark.gpu
def test_captured_and_replayed():
    """Forward and backward captured into a graph give the eager bits on every replay."""
    mok = _mok()
    T, H = 200, 1024
    x, res, w, dy, dr = _inputs(T, H, torch.bfloat16, 8)
    d = mok.NormDesc(T, H)
    r, y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    rstd = torch.empty(T, device=DEV)
    ws = torch.empty(mok.norm_workspace_query(d)["bwd_ws"], dtype=torch.uint8, device=DEV)

    def step():
        mok.rmsnorm_forward(d, x, w, y=y, res=res, r=r, rstd=rstd)
        mok.rmsnorm_backward(d, dy, r, w, rstd, dx, dw=dw, dr=dr, ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.mul_(1.5)
        step()
        want = [t.clone() for t in (y, r, rstd, dx, dw)]
        for t in (y, r, rstd, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, r, rstd, dx, dw)))


@pytest.mark.gpu
def test_empty_batch_and_flags():
    mok = _mok()
    d = mok.NormDesc(0, 512, flags=mok.FLAG_WGRAD_F32)
    e = torch.empty(0, 512, dtype=torch.bfloat16, device=DEV)
    w, f0 = torch.ones(512, dtype=torch.bfloat16, device=DEV), torch.empty(0, device=DEV)
    dw = torch.full((512,), 7.0, device=DEV)
    mok.rmsnorm_forward(d, e, w, y=e)
    mok.rmsnorm_backward(d, e, e, w, f0, e, dw=dw, ws=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert (dw == 0).all()
    # fp32 dw of bf16 rows, and no dw at all
    T = 40
    x, res, w, dy, dr = _inputs(T, 512, torch.bfloat16, 1)
    d = mok.NormDesc(T, 512, flags=mok.FLAG_WGRAD_F32)
    y, rstd, dx, dx2 = torch.empty_like(x), torch.empty(T, device=DEV), torch.empty_like(x), torch.empty_like(x)
    mok.rmsnorm_forward(d, x, w, y=y, rstd=rstd)
    ws = torch.empty(mok.norm_workspace_query(d)["bwd_ws"], dtype=torch.uint8, device=DEV)
    mok.rmsnorm_backward(d, dy, x, w, rstd, dx, dw=dw, ws=ws)
    prod = dy.double() * x.double() * rstd.double()[:, None]
    _close(dw, prod.sum(0), prod.abs().sum(0))
    mok.rmsnorm_backward(d, dy, x, w, rstd, dx2)
    assert torch.equal(dx, dx2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [((1 << 25) + 37, 8), ((1 << 18) + 3, 8200)])
def test_more_rows_than_workgroups_and_offsets_past_32_bits(T, H):
    mok = _mok()
    print("case norm large", T, H, flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty(T, H, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w = (1 + 0.1 * torch.randn(H, device=DEV, generator=g)).bfloat16()
    d = mok.NormDesc(T, H, eps=1e-5)
    y, rstd = torch.empty_like(x), torch.empty(T, device=DEV)
    mok.rmsnorm_forward(d, x, w, y=y, rstd=rstd)
    for sl in (slice(0, 100), slice(T // 2, T // 2 + 100), slice(T - 100, T)):
        _close(y[sl], _reference(x[sl], None, w, 1e-5)[2])
        _close(rstd[sl], _reference(x[sl], None, w, 1e-5)[1])
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(mok.norm_workspace_query(d)["bwd_ws"], dtype=torch.uint8, device=DEV)
    mok.rmsnorm_backward(d, y, x, w, rstd, dx, dw=dw, ws=ws)
    for sl in (slice(0, 100), slice(T - 100, T)):
        xh, gv = x[sl].double() * rstd[sl].double()[:, None], y[sl].double() * w.double()
        size = rstd[sl].double()[:, None] * (gv.abs() + xh.abs() * (gv * xh).abs().mean(-1, keepdim=True))
        _close(dx[sl], rstd[sl].double()[:, None] * (gv - xh * (gv * xh).mean(-1, keepdim=True)), size)
    want = torch.zeros(H, dtype=torch.float64, device=DEV)
    for b in range(0, T, 1 << 22):
        want += (y[b: b + (1 << 22)].double() * (x[b: b + (1 << 22)].double() * rstd[b: b + (1 << 22)].double()[:, None])).sum(0)
    # 512 workgroups add T/512 rows each in fp32, one after the other: T/512 * 2^-24 of a positive sum at most
    _close(dw, want, want, extra=T / 512 * 2.0**-24)


# ---- refusals (no GPU needed) ----

@pytest.mark.parametrize("kw,status", [
    (dict(H=0), 3), (dict(H=12), 3), (dict(H=32776), 3), (dict(T=-1), 3), (dict(T=1 << 31), 3), (dict(act=2), 4),
    (dict(act=0, quant=2), 4), (dict(quant=0), 4), (dict(quant=2, H=136), 3), (dict(quant=3, H=384), 3),
    (dict(eps=-1.0), 3), (dict(eps=float("nan")), 3), (dict(eps=float("inf")), 3), (dict(flags=2), 3),
])
def test_descriptor_refusals(kw, status):
    mok = _mok()
    d = mok.NormDesc(**{**dict(T=4, H=128), **kw})
    with pytest.raises(mok.MokError) as ei:
        mok.norm_workspace_query(d)
    assert ei.value.status == status


def test_pointer_refusals():
    mok = _mok()
    lib, P = mok._lib, ctypes.c_void_p
    d = mok.NormDesc(4, 128)
    c = d.c()
    ok = P(4096)
    assert lib.mok_rmsnorm_forward(c, None, None, ok, None, ok, None, None, None, None) == 1
    assert lib.mok_rmsnorm_forward(c, ok, None, ok, None, None, None, None, None, None) == 1
    assert lib.mok_rmsnorm_forward(c, ok, P(4100), ok, None, ok, None, None, None, None) == 2
    assert lib.mok_rmsnorm_forward(c, ok, None, ok, None, ok, None, None, P(4104), None) == 2
    q = mok.NormDesc(4, 128, quant=mok.MXFP8).c()
    assert lib.mok_rmsnorm_forward(q, ok, None, ok, None, ok, None, ok, None, None) == 1
    n = mok.norm_workspace_query(d)["bwd_ws"]
    assert lib.mok_rmsnorm_backward(c, ok, None, ok, ok, ok, ok, ok, ok, n - 1, None) == 6
    assert lib.mok_rmsnorm_backward(c, ok, None, ok, ok, ok, None, ok, ok, n, None) == 1
    assert lib.mok_rmsnorm_backward(c, ok, None, ok, ok, None, ok, None, None, 0, None) == 1
    big = mok.Desc(64, 128, 8, 2, 256, flags=mok.FLAG_X_QUANT)
    with pytest.raises(mok.MokError) as ei:
        mok.workspace_query(big)
    assert ei.value.status == 4


def test_binding_refusals():
    mok = _mok()
    d = mok.NormDesc(4, 128)
    t = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.ones(128, dtype=torch.bfloat16)
    for bad in (dict(x=t.float()), dict(x=t[:3]), dict(w=w[:64]), dict(y=torch.zeros(128, 4, dtype=torch.bfloat16).t()),
                dict(res=t.half()), dict(q=torch.zeros(4, 128, dtype=torch.uint8)), dict(y=None), dict(x=None), dict()):
        a = {**dict(x=t, w=w, y=t.clone()), **bad}
        with pytest.raises(ValueError):   # the last one: tensors that are not on the GPU
            mok.rmsnorm_forward(d, a.pop("x"), a.pop("w"), **a)
