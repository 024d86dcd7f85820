"""The operators around the layer together with it, as a transformer block's training step runs
them: norm with the residual -> router with its balance loss -> routed experts + a shared expert,
and back, against fp64 autograd of the same formulas on the same inputs.

Tolerance: a bf16 tensor on the way is off by at most 2^-8 of each value, in the root mean square
2^-8 / sqrt(3) = 2.3e-3; a result behind up to sixteen such roundings in a row is within
4 * 2.3e-3 < 1e-2 of its norm when they are independent, 2e-2 with the routed experts' own bound
of 5e-3 in the same chain. The loss has only y in bf16 behind it: 1e-3 of the
loss (the logits of y, whose rounding moves each p by up to 2^-8, average out over the tokens)."""
import pytest
import torch

DEV = "cuda"


class Block:
    def __init__(self, T, H, E, k, I, S, seed=0):
        from mixture_experts_layer_stable_amd import mok
        self.mok, self.T, self.H, self.E, self.k, self.I = mok, T, H, E, k, I
        g = torch.Generator().manual_seed(seed)
        n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16().to(DEV)
        self.x, self.res, self.dr = n(T, H), n(T, H, std=2.0), n(T, H)
        self.w = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16().to(DEV)
        self.wr, self.w1, self.w2 = n(E, H, std=H**-0.5), n(E, 2 * I, H, std=H**-0.5), n(E, H, I, std=I**-0.5)
        self.s1, self.s2 = n(2 * I, H, std=H**-0.5), n(H, I, std=I**-0.5)
        cut = torch.randint(0, T + 1, (S - 1,), generator=g).sort().values
        self.seg = torch.cat([torch.tensor([0]), cut, torch.tensor([T])]).int().to(DEV)
        self.mask = (torch.rand(T, generator=g) < 0.85).to(DEV)
        self.dloss = torch.tensor([300.0, 40.0], device=DEV)   # large enough to be seen in dx and dwr
        d = self.d = mok.Desc(T, H, E, k, I)
        self.buf = mok.Buffers(d)
        self.nd = mok.NormDesc(T, H)
        self.bd = mok.BalanceDesc(T, E, k, S=S, grad=mok.BF16, coef=1.0, zcoef=1.0)
        self.up, self.down = mok.LinearDesc(T, I, H, epi=mok.EPI_SWIGLU), mok.LinearDesc(T, H, I)
        self.rt = mok.LinearDesc(T, E, H)
        b, f = (lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=DEV)), (lambda *s: torch.empty(*s, device=DEV))
        self.r, self.y, self.rstd, self.logits = b(T, H), b(T, H), f(T), f(T, E)
        self.loss, self.prob, self.stat = f(2), f(S, E), f(T)
        self.counts, self.tokens = f(S, E).int(), f(S + 2).int()
        self.h, self.pre, self.out = b(T, I), b(T, 2 * I), b(T, H)
        self.dlogits, self.dh, self.dx = b(T, E), b(T, I), b(T, H)
        self.dw, self.ds1, self.ds2, self.dwr = b(H), b(2 * I, H), b(H, I), b(E, H)
        need = [mok.norm_workspace_query(self.nd)["bwd_ws"], mok.balance_workspace_query(self.bd)["fwd_ws"]]
        for v in (self.up, self.down, self.rt):
            need += list(mok.linear_workspace_query(v).values())
        self.ws = torch.empty(max(need), dtype=torch.uint8, device=DEV)   # one workspace, calls in order

    def forward(self):
        m, b, ws = self.mok, self.buf, self.ws
        m.rmsnorm_forward(self.nd, self.x, self.w, y=self.y, res=self.res, r=self.r, rstd=self.rstd)
        m.route(self.d, self.y, self.wr, None, b.idx, b.gate, self.logits)
        m.balance_forward(self.bd, self.logits, b.idx, self.loss, self.counts, self.tokens, self.prob, self.stat, ws,
                          seg=self.seg, mask=self.mask)
        m.schedule_build(self.d, b.idx, b.sched)
        m.moe_forward(self.d, b.sched, self.y, b.gate, self.w1, self.w2, b.y, b.saved, b.fwd_ws)
        m.linear_forward(self.up, self.y, self.s1, self.h, pre=self.pre, ws=ws)
        m.linear_forward(self.down, self.h, self.s2, self.out, res=b.y, ws=ws)

    def backward(self):
        """self.dr is the gradient of r and of the block's output (the next residual is their sum)."""
        m, b, ws = self.mok, self.buf, self.ws
        m.linear_backward(self.down, self.dr, self.h, self.s2, dx=self.dh, dw=self.ds2, ws=ws)
        m.moe_backward(self.d, b.sched, self.y, b.idx, b.gate, self.w1, self.w2, self.wr, b.saved, self.dr, b.dx, b.dw1,
                       b.dw2, b.dgate, b.dwr, b.bwd_ws)
        m.linear_backward(self.up, self.dh, self.y, self.s1, dx=b.dx, dw=self.ds1, pre=self.pre, dx_add=b.dx, ws=ws)
        m.balance_backward(self.bd, self.logits, self.counts, self.tokens, self.stat, self.dloss, self.dlogits,
                           seg=self.seg, mask=self.mask)
        m.linear_backward(self.rt, self.dlogits, self.y, self.wr, dx=b.dx, dw=self.dwr, dx_add=b.dx, dw_add=b.dwr, ws=ws)
        m.rmsnorm_backward(self.nd, b.dx, self.r, self.w, self.rstd, self.dx, dw=self.dw, dr=self.dr, ws=ws)

    def reference(self):
        """fp64 autograd on the CPU, with the selection that the router made."""
        p = {n: getattr(self, n).double().cpu().requires_grad_() for n in ("x", "w", "wr", "w1", "w2", "s1", "s2")}
        idx, T, k, E = self.buf.idx.long().cpu(), self.T, self.k, self.E
        r = p["x"] + self.res.double().cpu()
        y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + self.nd.eps) * p["w"]
        z = y @ p["wr"].t()
        gate = torch.softmax(torch.gather(z, 1, idx), 1)
        swiglu = lambda v: torch.nn.functional.silu(v[..., : self.I]) * v[..., self.I:]
        out = swiglu(y @ p["s1"].t()) @ p["s2"].t()
        routed = []
        for e in range(E):
            o = swiglu(y @ p["w1"][e].t()) @ p["w2"][e].t()
            routed.append(o * (gate * (idx == e)).sum(1, keepdim=True))
        out = out + sum(routed)
        on, seg = self.mask.cpu(), self.seg.cpu().tolist()
        pick = [[t for t in range(a, b) if on[t]] for a, b in zip(seg, seg[1:])]
        live = [s for s in pick if s]
        l0 = sum(E * ((torch.bincount(idx[s].reshape(-1), minlength=E).double() / (k * len(s))) * torch.softmax(z[s], 1).mean(0)
                      ).sum() for s in live) / len(live)
        l1 = torch.logsumexp(z[on], 1).square().mean()
        d, dl = self.dr.double().cpu(), self.dloss.double().cpu()
        grads = torch.autograd.grad((d * (out + r)).sum() + dl[0] * l0 + dl[1] * l1, list(p.values()))
        return out.detach(), (float(l0), float(l1)), dict(zip(p, grads))


def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k,I,S", [(192, 256, 16, 2, 128, 5), (77, 384, 8, 3, 256, 1)])
def test_block_step(T, H, E, k, I, S):
    print("case block", T, H, E, k, I, S, flush=True)
    b = Block(T, H, E, k, I, S)
    b.forward()
    b.backward()
    b.mok.check_schedule(b.d, b.buf.sched)
    out, (l0, l1), g = b.reference()
    errs = dict(out=rel(b.out, out), x=rel(b.dx, g["x"]), w=rel(b.dw, g["w"]), wr=rel(b.dwr, g["wr"]),
                w1=rel(b.buf.dw1, g["w1"]), w2=rel(b.buf.dw2, g["w2"]), s1=rel(b.ds1, g["s1"]), s2=rel(b.ds2, g["s2"]))
    print(errs, flush=True)
    assert max(errs.values()) < 2e-2, errs
    assert abs(float(b.loss[0]) - l0) < 1e-3 * l0 and abs(float(b.loss[1]) - l1) < 1e-3 * l1
    assert int(b.counts.sum()) == int(b.mask.sum()) * k


@pytest.mark.gpu
def test_block_step_in_a_graph_and_on_another_stream():
    """The whole step, captured and replayed between eager steps and run on a stream of its own: the same bits."""
    b = Block(160, 256, 8, 2, 128, 3, seed=4)
    outs = lambda: [t.clone() for t in (b.out, b.loss, b.counts, b.dx, b.dw, b.dwr, b.ds1, b.ds2, b.buf.dw1, b.buf.dw2)]

    def step():
        b.forward()
        b.backward()

    step()
    torch.cuda.synchronize()
    want = outs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, outs()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        b.x.mul_(1.25)
        step()
        torch.cuda.synchronize()
        want = outs()
        for t in (b.out, b.loss, b.dx, b.dw, b.dwr, b.ds1, b.ds2):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, outs())), i
