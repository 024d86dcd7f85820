"""Cases of the operators around the MoE layer step: the RMS norm with the residual's addition (and MX output), the
router's balance loss with its counts and gradient, and the matrix product with bias, activation and residual in its
epilogue. Each case runs in a plain form of elementary torch operations, or (own = True) through mok's entry points."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a single decoded token enters an MXFP8 layer: latency
        dict(name="norm-fwd-1x7168-mxfp8", op="norm", dir="fwd", T=1, H=7168, type="bf16", res=True, quant=True),
        # one micro-batch of the streamed MXFP8 step: y for the router, quantised rows for the experts
        dict(name="norm-fwd-2048x7168-mxfp8", op="norm", dir="fwd", T=2048, H=7168, type="bf16", res=True, quant=True),
        # a whole training batch in bf16
        dict(name="norm-fwd-16384x7168", op="norm", dir="fwd", T=16384, H=7168, type="bf16", res=True, quant=False),
        dict(name="norm-bwd-16384x7168", op="norm", dir="bwd", T=16384, H=7168, type="bf16", res=True, quant=False),
        # fp32 rows of an odd count and width, forward and backward, no residual
        dict(name="norm-step-777x1000-f32", op="norm", dir="step", T=777, H=1000, type="f32", res=False, quant=False),
        # the smallest router: loss and gradient of one small batch
        dict(name="balance-64x8", op="balance", T=64, E=8, k=2, S=0, score="softmax", z=True, mask=False, grad="f32"),
        # packed sequences of uneven lengths with padding tokens among them
        dict(name="balance-16384x384-ragged", op="balance", T=16384, E=384, k=8, S=37, score="softmax", z=True,
             mask=True, grad="bf16"),
        # normalised sigmoid scores over a long accumulated batch
        dict(name="balance-131072x256-sigmoid", op="balance", T=131072, E=256, k=8, S=0, score="sigmoid", z=False,
             mask=False, grad="f32"),
        # the shared expert's gate and up projections for a few decoded tokens: the weights are read once
        dict(name="linear-fwd-5x2048x7168-swiglu", op="linear", dir="fwd", M=5, N=2048, K=7168, type="bf16",
             epi="swiglu", bias=False, add=False),
        # the same for a training batch
        dict(name="linear-fwd-16384x2048x7168-swiglu", op="linear", dir="fwd", M=16384, N=2048, K=7168, type="bf16",
             epi="swiglu", bias=False, add=False),
        # fp32 product with every part of the epilogue, odd sizes
        dict(name="linear-fwd-2500x1000x520-f32", op="linear", dir="fwd", M=2500, N=1000, K=520, type="f32",
             epi="gelu", bias=True, add=True),
        # the shared expert's backward: gradients of its input (added to the routed experts') and weights
        dict(name="linear-bwd-8192x2048x7168-swiglu", op="linear", dir="bwd", M=8192, N=2048, K=7168, type="bf16",
             epi="swiglu", bias=False, add=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "balance", "linear"])
    if op == "norm":
        quant = rng.random() < 0.4
        H = _log(rng, 128, 8192, 128 if quant else 8)
        T = _log(rng, 1, min(131072, 16384 * 7168 // H))
        if quant:
            return dict(op="norm", dir="fwd", T=T, H=H, type="bf16", res=rng.random() < 0.7, quant=True)
        f32 = rng.random() < 0.3 and 2 * T * H <= 16384 * 7168
        return dict(op="norm", dir=rng.choice(["fwd", "bwd", "step"] if 2 * T * H <= 16384 * 7168 else ["fwd", "bwd"]),
                    T=T, H=H, type="f32" if f32 else "bf16", res=rng.random() < 0.7, quant=False)
    if op == "balance":
        E = _log(rng, 4, 1024)
        T = _log(rng, 1, 131072 * 256 // max(E, 256))
        score = rng.choice(["softmax", "softmax", "sigmoid"])
        return dict(op="balance", T=T, E=E, k=rng.randint(1, min(E, 16, 9)), S=rng.choice([0, 1, 5, 64, 300]),
                    score=score, z=score == "softmax" and rng.random() < 0.6, mask=rng.random() < 0.5,
                    grad=rng.choice(["f32", "bf16"]))
    f32 = rng.random() < 0.2
    dir_ = rng.choice(["fwd", "fwd", "bwd"])
    epi = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu"])
    while True:
        N, K = _log(rng, 64, 8192, 8), _log(rng, 64, 8192, 8)
        M = _log(rng, 1, 16384)
        cost = 2.0 * M * N * K * (2 if epi == "swiglu" else 1) * (2 if dir_ == "bwd" else 1) * (8 if f32 else 1)
        if cost <= 0.9e12:
            break
    return dict(op="linear", dir=dir_, M=M, N=N, K=K, type="f32" if f32 else "bf16", epi=epi, bias=rng.random() < 0.4,
                add=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "norm":
        es, n = (4 if c["type"] == "f32" else 2), c["T"] * c["H"]
        fwd = es * n * (2 + 2 * c["res"]) + 4 * c["T"] + es * c["H"] + (n * 33 // 32 if c["quant"] else 0)
        bwd = es * n * (3 + c["res"]) + 4 * c["T"] + 2 * es * c["H"]
        return {"bytes": fwd * (c["dir"] != "bwd") + bwd * (c["dir"] != "fwd"),
                "flops": n * (6.0 * (c["dir"] != "bwd") + 10.0 * (c["dir"] != "fwd"))}
    if c["op"] == "balance":
        n = c["T"] * c["E"]
        return {"bytes": 4 * n + 4 * c["T"] * c["k"] + 4 * n + n * (4 if c["grad"] == "f32" else 2), "flops": 16.0 * n}
    es, M, N, K = (4 if c["type"] == "f32" else 2), c["M"], c["N"], c["K"]
    Np = 2 * N if c["epi"] == "swiglu" else N
    if c["dir"] == "fwd":
        return {"bytes": es * (M * K + Np * K + M * N * (1 + c["add"]) + M * Np * (c["epi"] != "none")),
                "flops": 2.0 * M * Np * K}
    return {"bytes": es * (M * N + M * Np * (c["epi"] != "none") + (M * K + Np * K) * (2 + c["add"])),
            "flops": 4.0 * M * Np * K}


# ------------------------------------------------------------------------------------------------ inputs

def _inputs(case, seed):
    """The tensors of a case, from the seed alone (also the inputs of exact())."""
    c, g = case, torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).mul_(std).to(dtype)

    if c["op"] == "norm":
        t, T, H = TYPES[c["type"]], c["T"], c["H"]
        i = dict(w=(1 + normal(H, std=0.1)).to(t))
        gain = torch.exp(normal(H, std=0.5))  # a residual stream's channels differ in size
        if c["dir"] != "bwd":
            i["x"] = normal(T, H).mul_(gain).to(t)
            if c["res"]:
                i["res"] = normal(T, H, std=3.0).mul_(gain).to(t)
        if c["dir"] != "fwd":
            i["dy"] = normal(T, H, dtype=t)
            if c["res"]:
                i["dr"] = normal(T, H, dtype=t)
        if c["dir"] == "bwd":  # what the forward left
            i["r"] = normal(T, H, std=2.0).mul_(gain).to(t)
            i["rstd"] = torch.rsqrt(i["r"].float().square().mean(-1) + EPS)
        return i
    if c["op"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        logits = normal(T, E, std=1.5).add_(normal(E))  # some experts are liked better
        idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        i = dict(logits=logits, idx=idx, dloss=normal(2).abs_().add_(0.5))
        if c["S"]:  # offsets of S sequences; a few tokens behind the last are in none
            cut = torch.rand(c["S"] - 1, generator=g, device=DEV).mul_(T + 1).floor_().clamp_(max=T)
            ends = torch.tensor([0.0, float(T - T // 50)], device=DEV)
            i["seg"] = torch.cat([ends, cut.clamp_(max=T - T // 50)]).sort().values.to(torch.int32)
        if c["mask"]:
            i["mask"] = (torch.rand(T, generator=g, device=DEV) < 0.9).to(torch.uint8)
        return i
    t, M, N, K = TYPES[c["type"]], c["M"], c["N"], c["K"]
    Np = 2 * N if c["epi"] == "swiglu" else N
    i = dict(x=normal(M, K, dtype=t), w=normal(Np, K, std=K ** -0.5, dtype=t))
    if c["dir"] == "fwd":
        if c["bias"]:
            i["bias"] = normal(Np, std=0.5)
        if c["add"]:
            i["res"] = normal(M, N, dtype=t)
    else:
        i["dy"] = normal(M, N, dtype=t)
        if c["epi"] != "none":
            i["pre"] = normal(M, Np, dtype=t)
        if c["add"]:
            i["dx_add"] = normal(M, K, dtype=t)
            i["dw_add"] = normal(Np, K, dtype=t)
    return i


def prepare(case, seed):
    state = dict(case=case, i=_inputs(case, seed))
    if own:
        state["plan"] = _plan(case)
    return state


def _coef(case):
    return 0.01, (0.001 if case["z"] else 0.0)


def _plan(case):
    """What a program keeps between its calls of mok: the descriptor, workspace and output tensors."""
    from mixture_experts_layer_stable_amd import mok
    c = case

    def new(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    def ws(n):
        return new(max(n, 256), dtype=torch.uint8)

    if c["op"] == "norm":
        t, T, H = TYPES[c["type"]], c["T"], c["H"]
        d = mok.NormDesc(T, H, act=mok.DTYPES[c["type"]], quant=mok.MXFP8 if c["quant"] else None, eps=EPS)
        p = dict(mok=mok, d=d)
        if c["dir"] != "bwd":
            p.update(y=new(T, H, dtype=t), rstd=new(T), r=new(T, H, dtype=t) if c["res"] else None)
            if c["quant"]:
                p.update(q=new(T, H, dtype=torch.uint8), s=new(H // 128, T, 4, dtype=torch.uint8))
        if c["dir"] != "fwd":
            p.update(dx=new(T, H, dtype=t), dw=new(H, dtype=t), ws=ws(mok.norm_workspace_query(d)["bwd_ws"]))
        return p
    if c["op"] == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], max(c["S"], 1)
        coef, zcoef = _coef(c)
        d = mok.BalanceDesc(T, E, k, S=c["S"], score=mok.SCORES[c["score"]], grad=mok.DTYPES[c["grad"]], coef=coef,
                            zcoef=zcoef)
        return dict(mok=mok, d=d, loss=new(2), counts=new(S, E, dtype=torch.int32), tokens=new(S + 2, dtype=torch.int32),
                    prob=new(S, E), stat=new(T), dlogits=new(T, E, dtype=TYPES[c["grad"]]),
                    ws=ws(mok.balance_workspace_query(d)["fwd_ws"]))
    t, M, N, K = TYPES[c["type"]], c["M"], c["N"], c["K"]
    Np = 2 * N if c["epi"] == "swiglu" else N
    d = mok.LinearDesc(M, N, K, act=mok.DTYPES[c["type"]], epi=mok.EPILOGUES[c["epi"]])
    sz = mok.linear_workspace_query(d)
    if c["dir"] == "fwd":
        return dict(mok=mok, d=d, y=new(M, N, dtype=t), pre=new(M, Np, dtype=t) if c["epi"] != "none" else None,
                    ws=ws(sz["fwd_ws"]))
    return dict(mok=mok, d=d, dx=new(M, K, dtype=t), dw=new(Np, K, dtype=t), db=new(Np) if c["bias"] else None,
                ws=ws(sz["bwd_ws"]))


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    c, i = state["case"], state["i"]
    if own:
        return _own(c, i, state["plan"])
    if c["op"] == "norm":
        return _plain_norm(c, i)
    if c["op"] == "balance":
        return _plain_balance(c, i)
    return _plain_linear(c, i)


def _own(c, i, p):
    mok, d = p["mok"], p["d"]
    out = {}
    if c["op"] == "norm":
        if c["dir"] != "bwd":
            mok.rmsnorm_forward(d, i["x"], i["w"], y=p["y"], res=i.get("res"), r=p["r"], q=p.get("q"), s=p.get("s"),
                                rstd=p["rstd"])
            out.update(y=p["y"], rstd=p["rstd"])
            if c["res"]:
                out["r"] = p["r"]
            if c["quant"]:  # the E4M3 elements and E8M0 scales, as the values that they stand for
                out.update(q=p["q"].view(torch.float8_e4m3fn), s=p["s"].view(torch.float8_e8m0fnu))
        if c["dir"] != "fwd":
            r = i["r"] if c["dir"] == "bwd" else (p["r"] if c["res"] else i["x"])
            rstd = i["rstd"] if c["dir"] == "bwd" else p["rstd"]
            mok.rmsnorm_backward(d, i["dy"], r, i["w"], rstd, p["dx"], dw=p["dw"], dr=i.get("dr"), ws=p["ws"])
            out.update(dx=p["dx"], dw=p["dw"])
        return out
    if c["op"] == "balance":
        mok.balance_forward(d, i["logits"], i["idx"], p["loss"], p["counts"], p["tokens"], p["prob"], p["stat"], p["ws"],
                            seg=i.get("seg"), mask=i.get("mask"))
        mok.balance_backward(d, i["logits"], p["counts"], p["tokens"], p["stat"], i["dloss"], p["dlogits"],
                             seg=i.get("seg"), mask=i.get("mask"))
        return dict(loss=p["loss"], counts=p["counts"], prob=p["prob"], dlogits=p["dlogits"])
    if c["dir"] == "fwd":
        mok.linear_forward(d, i["x"], i["w"], p["y"], bias=i.get("bias"), res=i.get("res"), pre=p["pre"], ws=p["ws"])
        return dict(y=p["y"], pre=p["pre"]) if p["pre"] is not None else dict(y=p["y"])
    mok.linear_backward(d, i["dy"], i["x"], i["w"], dx=p["dx"], dw=p["dw"], db=p["db"], pre=i.get("pre"),
                        dx_add=i.get("dx_add"), dw_add=i.get("dw_add"), ws=p["ws"])
    return dict(dx=p["dx"], dw=p["dw"], db=p["db"]) if p["db"] is not None else dict(dx=p["dx"], dw=p["dw"])


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_norm(c, i):
    t, out, w = TYPES[c["type"]], {}, i["w"].float()
    if c["dir"] != "bwd":
        v = i["x"].float()
        if c["res"]:
            v = v + i["res"].float()
        rstd = torch.rsqrt((v * v).mean(-1) + EPS)
        y = (v * rstd[:, None] * w).to(t)
        out.update(y=y, rstd=rstd)
        if c["res"]:
            out["r"] = v.to(t)
        if c["quant"]:
            out["q"], out["s"] = _plain_mx(y)
    if c["dir"] != "fwd":
        if c["dir"] == "bwd":
            r, rstd = i["r"].float(), i["rstd"]
        else:
            r = v.to(t).float()
        xh, dy = r * rstd[:, None], i["dy"].float()
        g = dy * w
        dx = rstd[:, None] * (g - xh * (g * xh).mean(-1, keepdim=True))
        if c["res"]:
            dx = dx + i["dr"].float()
        out.update(dx=dx.to(t), dw=(dy * xh).sum(0).to(t))
    return out


def _plain_mx(y):
    """MXFP8 of bf16 rows: E4M3 elements, and the E8M0 scales of 32 along a row as [H/128][T][4]."""
    T, H = y.shape
    b = y.float().view(T, H // 32, 32)
    amax = b.abs().amax(-1)
    s = (torch.frexp(amax).exponent - 9).clamp(-127, 127)  # floor(log2 amax) - 8
    s = torch.where(amax == 0, torch.full_like(s, -127), s)
    q = torch.ldexp(b, -s[..., None]).clamp(-448, 448).view(T, H).to(torch.float8_e4m3fn)
    s = (s + 127).to(torch.uint8).view(T, H // 128, 4).transpose(0, 1).contiguous()
    return q, s.view(torch.float8_e8m0fnu)


def _rows(c, i):
    """Segment of each row, and whether the row counts."""
    T, S = c["T"], max(c["S"], 1)
    t = torch.arange(T, device=DEV)
    if c["S"]:
        seg = i["seg"].long()
        s = torch.searchsorted(seg, t, right=True) - 1
        on = (t >= seg[0]) & (t < seg[-1])
        s = s.clamp(0, S - 1)
    else:
        s, on = torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool)
    if "mask" in i:
        on = on & (i["mask"] != 0)
    return s, on, S


def _sums(s, rows, S):
    """Sums of the rows of each segment, in 64 bits."""
    if S == 1:
        return rows.sum(0, keepdim=True, dtype=torch.float64)
    return (torch.arange(S, device=DEV)[:, None] == s).double() @ rows.double()


def _plain_balance(c, i):
    z, idx, E, k = i["logits"], i["idx"].long(), c["E"], c["k"]
    coef, zcoef = _coef(c)
    s, on, S = _rows(c, i)
    onf = on.float()
    n = torch.stack([on.sum()]) if S == 1 else _sums(s, on.double()[:, None], S).squeeze(1).long()
    hot = torch.zeros_like(z).scatter_add_(1, idx, onf[:, None].expand(-1, k))
    counts = _sums(s, hot, S).long()
    if c["score"] == "softmax":
        m = z.amax(-1, keepdim=True)
        e = torch.exp(z - m)
        den = e.sum(-1, keepdim=True)
        p, lse = e / den, (m + torch.log(den)).squeeze(1)
    else:
        sg = 1 / (1 + torch.exp(-z))
        den = sg.sum(-1, keepdim=True)
        p = sg / den
    p = p * onf[:, None]
    Q = _sums(s, p, S)
    nd, cd = n.double(), counts.double()
    full = (n > 0).sum().clamp(min=1).double()
    scale = torch.where(n > 0, coef * E / (k * full * nd.clamp(min=1) ** 2), torch.zeros_like(nd))
    N = on.sum().clamp(min=1).double()
    loss = (scale * (cd * Q).sum(1)).sum()
    lossz = zcoef * (lse.double().square() * onf).sum() / N if zcoef else torch.zeros_like(loss)
    g = (i["dloss"][0] * scale).float()[s][:, None]
    cs = counts.float()[s]
    d = cs - (p * cs).sum(-1, keepdim=True)
    if c["score"] == "softmax":
        dz = g * p * d
        if zcoef:
            dz = dz + (i["dloss"][1] * (2 * zcoef) / N).float() * lse[:, None] * p
    else:
        dz = g * p * (1 - sg) * d
    return dict(loss=torch.stack([loss, lossz]).float(), counts=counts.to(torch.int32),
                prob=(Q / nd.clamp(min=1)[:, None]).float(), dlogits=dz.to(TYPES[c["grad"]]))


def _plain_linear(c, i):
    t, x, w, N = TYPES[c["type"]], i["x"].float(), i["w"].float(), c["N"]
    if c["dir"] == "fwd":
        pre = x @ w.t()
        if c["bias"]:
            pre = pre + i["bias"]
        if c["epi"] == "none":
            y = pre
        elif c["epi"] == "gelu":
            y = pre * 0.5 * (1 + torch.erf(pre * math.sqrt(0.5)))
        else:
            y = pre[:, :N] / (1 + torch.exp(-pre[:, :N]))
            if c["epi"] == "swiglu":
                y = y * pre[:, N:]
        if c["add"]:
            y = y + i["res"].float()
        return dict(y=y.to(t), pre=pre.to(t)) if c["epi"] != "none" else dict(y=y.to(t))
    dy = i["dy"].float()
    if c["epi"] == "none":
        dpre = dy
    elif c["epi"] == "gelu":
        a = i["pre"].float()
        dpre = dy * (0.5 * (1 + torch.erf(a * math.sqrt(0.5))) + a * torch.exp(-0.5 * a * a) / math.sqrt(2 * math.pi))
    else:
        a = i["pre"][:, :N].float()
        sg = 1 / (1 + torch.exp(-a))
        ds = sg * (1 + a * (1 - sg))
        dpre = dy * ds if c["epi"] == "silu" else torch.cat([dy * i["pre"][:, N:].float() * ds, dy * a * sg], 1)
    dx, dw = dpre @ w, dpre.t() @ x
    if c["add"]:
        dx, dw = dx + i["dx_add"].float(), dw + i["dw_add"].float()
    out = dict(dx=dx.to(t), dw=dw.to(t))
    if c["bias"]:
        out["db"] = dpre.sum(0)
    return out


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    c, i = case, _inputs(case, seed)
    d = {n: v.double() if v.is_floating_point() else v for n, v in i.items()}
    return {"norm": _exact_norm, "balance": _exact_balance, "linear": _exact_linear}[c["op"]](c, d)


def _exact_norm(c, i):
    out, H = {}, c["H"]
    if c["dir"] != "bwd":
        v = i["x"] + (i["res"] if c["res"] else 0)
        rstd = 1 / torch.sqrt(v.square().sum(-1) / H + EPS)
        out.update(y=torch.einsum("th,t,h->th", v, rstd, i["w"]), rstd=rstd)
        if c["res"]:
            out["r"] = v
        if c["quant"]:
            b = out["y"].to(torch.bfloat16).double().view(c["T"], H // 128, 4, 32)  # the layer quantises stored bf16 rows
            top = b.abs().amax(-1)
            s = (torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 8).clamp(-127, 127)
            u = b * torch.exp2(-s)[..., None]
            step = torch.exp2(torch.floor(torch.log2(u.abs().clamp(min=2.0 ** -6))) - 3)  # E4M3: 3 bits of fraction
            out["q"] = (torch.round(u / step) * step).clamp(-448, 448).view(c["T"], H)
            out["s"] = torch.exp2(s).transpose(0, 1).contiguous()
    if c["dir"] != "fwd":
        if c["dir"] == "bwd":
            r, rstd = i["r"], i["rstd"]
        else:
            r = v
        g = i["dy"] * i["w"]
        dot = (g * r).sum(-1)
        dx = g * rstd[:, None] - r * (dot * rstd ** 3 / H)[:, None]
        out.update(dx=dx + i["dr"] if c["res"] else dx, dw=torch.einsum("th,th,t->h", i["dy"], r, rstd))
    return out


def _exact_balance(c, i):
    """Differentiates the loss segment by segment (no formula for the gradient)."""
    z = i["logits"].clone().requires_grad_(True)
    coef, zcoef = _coef(c)
    bounds = i["seg"].tolist() if c["S"] else [0, c["T"]]
    on = i["mask"] != 0 if "mask" in i else torch.ones(c["T"], dtype=torch.bool, device=DEV)
    S, E = len(bounds) - 1, c["E"]
    live = [int(on[a:b].sum()) for a, b in zip(bounds, bounds[1:])]
    loss, lossz, prob = z.new_zeros(()), z.new_zeros(()), []
    for s in range(S):
        if live[s] == 0:
            prob.append(z.new_zeros(E))
            continue
        rows = slice(bounds[s], bounds[s + 1])
        pick = on[rows].nonzero().squeeze(1) + bounds[s]
        zs = z[pick]
        p = torch.softmax(zs, 1) if c["score"] == "softmax" else torch.sigmoid(zs) / torch.sigmoid(zs).sum(1, keepdim=True)
        share = torch.bincount(i["idx"][pick].reshape(-1).long(), minlength=E).double() / (live[s] * c["k"])
        loss = loss + coef * E * (share * p.mean(0)).sum() / sum(n > 0 for n in live)
        if zcoef:
            lossz = lossz + zcoef * torch.logsumexp(zs, 1).square().sum() / sum(live)
        prob.append(p.detach().mean(0))
    total = i["dloss"][0] * loss + i["dloss"][1] * lossz
    dz = torch.autograd.grad(total, z)[0] if total.requires_grad else torch.zeros_like(z)
    return dict(loss=torch.stack([loss, lossz]).detach(), counts=None, prob=torch.stack(prob), dlogits=dz)


def _exact_linear(c, i):
    N = c["N"]

    def act(a):
        if c["epi"] == "none":
            return a
        if c["epi"] == "gelu":
            return torch.special.ndtr(a) * a
        h = torch.sigmoid(a[:, :N]) * a[:, :N]
        return h * a[:, N:] if c["epi"] == "swiglu" else h

    if c["dir"] == "fwd":
        pre = torch.mm(i["x"], i["w"].t().contiguous())
        if c["bias"]:
            pre = pre + i["bias"]
        y = act(pre) + (i["res"] if c["add"] else 0)
        return dict(y=y, pre=pre) if c["epi"] != "none" else dict(y=y)
    dpre = i["dy"]
    if c["epi"] != "none":
        pre = i["pre"].clone().requires_grad_(True)
        dpre = torch.autograd.grad(act(pre), pre, i["dy"])[0]
    out = dict(dx=torch.mm(dpre, i["w"]), dw=torch.mm(dpre.t().contiguous(), i["x"]))
    if c["add"]:
        out.update(dx=out["dx"] + i["dx_add"], dw=out["dw"] + i["dw_add"])
    if c["bias"]:
        out["db"] = dpre.sum(0)
    return out
