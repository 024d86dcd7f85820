"""An expert layer from its parts, as a program would run it: route -> schedule -> dispatch -> grouped products ->
combine, and back; against mok_moe_forward / _backward where they compute the same, and against fp64 autograd for experts
that the layer itself does not have. Relative Frobenius errors within the layer's own bounds (bf16 5e-3, fp32 1e-5)."""
import pytest
import torch

from test_linear import DEV, _mok, act64

BOUND = {torch.bfloat16: 5e-3, torch.float32: 1e-5}


def rel(a, b):
    return float((a.double().cpu() - b.double().cpu()).norm() / b.double().cpu().norm())


class Layer:
    def __init__(self, T, H, E, k, I, act, epi, bias, seed=0):
        mok = self.mok = _mok()
        self.t = t = mok.TORCH_DTYPE[mok.DTYPES[act]]
        g = torch.Generator(device=DEV).manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(*s, generator=g, device=DEV) * std
        self.T, self.H, self.E, self.k, self.I, self.epi = T, H, E, k, I, epi
        self.desc = mok.Desc(T, H, E, k, 128 if I % 128 else I, act=mok.DTYPES[act])
        R, a = T * k, mok.DTYPES[act]
        self.up = mok.GroupedDesc(R, I, H, E, act=a, epi=mok.EPILOGUES[epi])
        self.down = mok.GroupedDesc(R, H, I, E, act=a)
        self.rows = mok.PermuteDesc(T, H, k, act=a)
        P = self.up.P
        self.x, self.dy = n(T, H).to(t), n(T, H).to(t)
        self.wr = n(E, H, std=H**-0.5).to(t)
        self.w1, self.w2 = n(E, P, H, std=H**-0.5).to(t), n(E, H, I, std=I**-0.5).to(t)
        self.b1, self.b2 = (n(E, P, std=0.5), n(E, H, std=0.5)) if bias else (None, None)
        new = lambda *s, dtype=t: torch.empty(*s, dtype=dtype, device=DEV)
        self.xs, self.pre, self.h, self.o, self.y = new(R, H), new(R, P), new(R, I), new(R, H), new(T, H)
        self.do, self.dh, self.dxs, self.dx = new(R, H), new(R, I), new(R, H), new(T, H)
        self.dgate, self.dw1, self.dw2 = new(T, k, dtype=torch.float32), new(E, P, H), new(E, H, I)
        self.db1, self.db2 = (new(E, P, dtype=torch.float32), new(E, H, dtype=torch.float32)) if bias else (None, None)
        size = max(mok.grouped_workspace_query(self.up)["bwd_ws"], mok.grouped_workspace_query(self.down)["bwd_ws"], 16)
        self.ws = new(size, dtype=torch.uint8)
        self.sched = new(mok.workspace_query(self.desc)["sched"], dtype=torch.uint8)
        self.idx, self.gate = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        v = mok.schedule_views(self.desc, self.sched)
        self.off, self.perm, self.inv = v["offsets"], v["perm"], v["inv"].view(T, k)

    def route(self):
        self.mok.route(self.desc, self.x, self.wr, None, self.idx, self.gate)
        self.mok.schedule_build(self.desc, self.idx, self.sched)

    def forward(self):
        m = self.mok
        m.dispatch_forward(self.rows, self.x, self.perm, self.xs)
        m.grouped_forward(self.up, self.xs, self.w1, self.off, self.h, bias=self.b1, pre=None if self.epi == "none" else self.pre)
        m.grouped_forward(self.down, self.h, self.w2, self.off, self.o, bias=self.b2)
        m.combine_forward(self.rows, self.o, self.inv, self.y, gate=self.gate)

    def backward(self):
        m = self.mok
        m.combine_backward(self.rows, self.dy, self.o, self.inv, self.do, gate=self.gate, dgate=self.dgate)
        m.grouped_backward(self.down, self.do, self.h, self.w2, self.off, dx=self.dh, dw=self.dw2, db=self.db2, ws=self.ws)
        m.grouped_backward(self.up, self.dh, self.xs, self.w1, self.off, dx=self.dxs, dw=self.dw1, db=self.db1,
                           pre=None if self.epi == "none" else self.pre, ws=self.ws)
        m.dispatch_backward(self.rows, self.dxs, self.inv, self.dx)

    def oracle(self):
        """y and the gradients in fp64 by autograd, on the CPU, for the routing that the GPU chose."""
        c = lambda v: v.detach().double().cpu().requires_grad_()
        x, w1, w2, gate = c(self.x), c(self.w1), c(self.w2), c(self.gate)
        b1, b2 = (c(self.b1), c(self.b2)) if self.b1 is not None else (None, None)
        idx = self.idx.cpu().long()
        y = torch.zeros(self.T, self.H, dtype=torch.float64)
        for e in range(self.E):
            t, j = (idx == e).nonzero(as_tuple=True)
            if len(t) == 0:
                continue
            p = x[t] @ w1[e].t() + (b1[e] if b1 is not None else 0)
            o = act64(self.epi, p) @ w2[e].t() + (b2[e] if b2 is not None else 0)
            y = y.index_add(0, t, gate[t, j][:, None] * o)
        leaves = [v for v in (x, w1, w2, gate, b1, b2) if v is not None]
        return y.detach(), torch.autograd.grad(y, leaves, self.dy.double().cpu(), allow_unused=True)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k,I,act,epi,bias", [
    (64, 128, 8, 2, 256, "f32", "swiglu", False), (300, 256, 32, 4, 136, "bf16", "gelu", True), (1, 256, 16, 8, 128, "bf16", "swiglu", True),
    (1000, 512, 12, 3, 264, "bf16", "silu", True), (777, 128, 100, 2, 72, "f32", "none", True), (2048, 1024, 32, 2, 512, "bf16", "swiglu", False)])
def test_layer(T, H, E, k, I, act, epi, bias):
    print("case parts", T, H, E, k, I, act, epi, bias, flush=True)
    L = Layer(T, H, E, k, I, act, epi, bias)
    L.route()
    L.forward()
    L.backward()
    y, grads = L.oracle()
    got = [L.dx, L.dw1, L.dw2, L.dgate] + ([L.db1, L.db2] if bias else [])
    errs = {"y": rel(L.y, y)}
    for name, a, b in zip(("dx", "dw1", "dw2", "dgate", "db1", "db2"), got, grads):
        errs[name] = rel(a, b)
    print(errs, flush=True)
    assert max(errs.values()) < BOUND[L.t], errs


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_same_as_the_layer(act):
    """SwiGLU experts without biases: y, the expert term of dx, dw1, dw2 and dgate are the layer's, to its own bound."""
    L = Layer(700, 256, 16, 4, 256, act, "swiglu", False, seed=1)
    mok = L.mok
    L.route()
    L.forward()
    L.backward()
    buf = mok.Buffers(L.desc, DEV)
    mok.moe_forward(L.desc, L.sched, L.x, L.gate, L.w1, L.w2, buf.y, buf.saved, buf.fwd_ws)
    mok.moe_backward(L.desc, L.sched, L.x, L.idx, L.gate, L.w1, L.w2, None, buf.saved, L.dy, buf.dx, buf.dw1, buf.dw2, buf.dgate,
                     None, buf.bwd_ws)
    torch.cuda.synchronize()
    for name in ("y", "dx", "dw1", "dw2", "dgate"):
        assert rel(getattr(L, name), getattr(buf, name)) < BOUND[L.t], name


@pytest.mark.gpu
def test_captured_step_beside_eager_ones():
    """The whole step captured, replayed with other tokens (and so other routes) between eager steps."""
    L = Layer(256, 256, 16, 4, 128, "bf16", "swiglu", True)

    def step():
        L.route()
        L.forward()
        L.backward()

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    names = ("y", "dx", "dw1", "dw2", "dgate", "db1", "db2")
    g = torch.Generator(device=DEV).manual_seed(9)
    for _ in range(3):
        L.x.copy_(torch.randn(256, 256, generator=g, device=DEV))
        step()
        want = [getattr(L, n).clone() for n in names]
        for n in names:
            getattr(L, n).fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, getattr(L, n)) for a, n in zip(want, names))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 200])
def test_serving_with_4_bit_weights(T):
    """Decoded tokens (and a short prompt) through experts whose weights q4_quantize made, against fp64 with the weights
    that the codes stand for."""
    L = Layer(T, 256, 16, 4, 128, "bf16", "swiglu", True, seed=2)
    mok, E = L.mok, L.E
    q = {}
    for name, w, N, K, epi in (("up", L.w1, L.I, L.H, mok.EPI_SWIGLU), ("down", L.w2, L.H, L.I, mok.EPI_NONE)):
        d = mok.Q4Desc(T * L.k, N, K, E, 64, epi=epi)
        a = dict(q=torch.empty(E, d.P, K // 2, dtype=torch.uint8, device=DEV), s=torch.empty(E, d.P, K // 64, dtype=L.t, device=DEV),
                 z=torch.empty(E, d.P, K // 64, dtype=torch.uint8, device=DEV))
        mok.q4_quantize(d, w, a["q"], a["s"], a["z"])
        q[name] = (d, a)
        code = torch.stack([a["q"] & 15, a["q"] >> 4], -1).flatten(-2).double()
        w64 = a["s"].double().repeat_interleave(64, -1) * (code - a["z"].double().repeat_interleave(64, -1))
        q[name + "64"] = w64.cpu()
    L.route()
    mok.dispatch_forward(L.rows, L.x, L.perm, L.xs)
    for name, x, y, b in (("up", L.xs, L.h, L.b1), ("down", L.h, L.o, L.b2)):
        d, a = q[name]
        mok.q4_forward(d, x, a["q"], a["s"], y, z=a["z"], off=L.off, bias=b)
    mok.combine_forward(L.rows, L.o, L.inv, L.y, gate=L.gate, res=L.x)
    want = L.x.double().cpu()
    idx, gate, x = L.idx.cpu().long(), L.gate.double().cpu(), L.x.double().cpu()
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            p = x[t] @ q["up64"][e].t() + L.b1[e].double().cpu()
            o = act64("swiglu", p) @ q["down64"][e].t() + L.b2[e].double().cpu()
            want = want.index_add(0, t, gate[t, j][:, None] * o)
    assert rel(L.y, want) < BOUND[L.t]
