"""Matrix products at shapes that the plan sends to each of its tiles, with and without slices of K, ragged in every
direction and from two 128-byte pieces of K on; and a check that no tile is left out. References in fp64 on the GPU;
tolerances of test_linear.py."""
import ctypes

import pytest
import torch

import test_linear
from test_linear import DEV, SMALL, Case

BF16, F32 = "bf16", "f32"
# act, epi, M, N, K; the largest tile (0) unless said, KT: 128-byte pieces of K
FORWARD = [
    (BF16, "none", 6977, 1696, 72), (BF16, "gelu", 8229, 904, 136), (BF16, "silu", 917, 8240, 200),   # KT 2, 3, 4
    (BF16, "none", 1033, 7208, 1032), (BF16, "none", 129, 4352, 18896),                              # KT 17; in slices
    (BF16, "swiglu", 645, 8912, 72), (BF16, "swiglu", 8307, 464, 136), (BF16, "swiglu", 395, 8296, 1032),
    (F32, "none", 1795, 8480, 8), (F32, "gelu", 1867, 8200, 72), (F32, "silu", 8213, 1864, 136),      # KT 1, 3, 5
    (F32, "none", 69, 3808, 34304), (F32, "swiglu", 781, 8, 14920),                                  # in slices
    (F32, "swiglu", 3845, 3976, 8), (F32, "swiglu", 8205, 848, 72), (F32, "swiglu", 4099, 328, 1032),
]
BACKWARD = [
    (BF16, "none", 7595, 72, 1552), (BF16, "none", 8281, 136, 920), (BF16, "none", 1031, 1032, 7208),  # dx
    (BF16, "none", 129, 18896, 4352),                                                                # dx in slices
    (BF16, "none", 65, 8232, 1456), (BF16, "none", 131, 8296, 920), (BF16, "gelu", 1001, 912, 8224),   # dw
    (BF16, "none", 18896, 136, 4352),                                                                # dw in slices
    (BF16, "swiglu", 2049, 1032, 3976),                                                              # both
    (F32, "none", 1795, 8, 8480), (F32, "none", 1923, 72, 7912), (F32, "silu", 772, 1032, 8808),       # dx
    (F32, "none", 69, 34304, 3808),                                                                  # dx in slices
    (F32, "none", 1, 3472, 4424), (F32, "none", 7, 6816, 2248), (F32, "none", 65, 4000, 3856),         # dw
    (F32, "swiglu", 1001, 424, 8272),                                                                # both
    (F32, "none", 34304, 72, 3808),                                                                  # dw in slices
]
FORWARD += [(BF16, e, *c) for e, c in (   # tiles 1 and 2, in one piece and in slices
    ("gelu", (365, 440, 912)), ("silu", (585, 552, 2144)), ("none", (33, 24, 584)), ("gelu", (417, 400, 1080)),
    ("swiglu", (281, 312, 904)), ("swiglu", (493, 488, 1824)), ("swiglu", (35, 24, 592)), ("swiglu", (333, 344, 1160)))]
BACKWARD += [(BF16, "none", 3373, 808, 24), (BF16, "none", 3397, 2000, 8), (BF16, "none", 6200, 8, 7832)]


def plan(kind, act, epi, M, N, K):
    """(tile, slices of K) of a product: linear_plan (csrc/block.h) of the built library."""
    mok = test_linear._mok()
    f = mok._lib._ZN3mok11linear_planEiiilil
    f.restype, f.argtypes = ctypes.c_uint64, [ctypes.c_int] * 3 + [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    v = f(("fwd", "dx", "dw").index(kind), mok.DTYPES[act], mok.EPILOGUES[epi], M, N, K)
    return v & 0xffffffff, v >> 32


def plans(act, epi, M, N, K, kinds=("fwd", "dx", "dw")):
    P = 2 * N if epi == "swiglu" else N
    got = {}
    if "fwd" in kinds:
        got["swiglu" if epi == "swiglu" else "fwd"] = plan("fwd", act, epi, M, N, K)
    if "dx" in kinds:
        got["dx"], got["dw"] = plan("dx", act, "none", M, K, P), plan("dw", act, "none", P, K, M)
    return got


def test_every_tile_is_reached():
    """By the shapes here and the small ones of test_linear.py: each type, product, tile, in one piece and in slices.
    Up to 32 rows forward take the kernel for few rows (4)."""
    got = set()
    for cases, kinds in ((FORWARD, ("fwd",)), (BACKWARD, ("dx",))):
        for c in cases:
            got |= {(c[0], k, t, s > 1) for k, (t, s) in plans(*c, kinds=kinds).items()}
    big = [c for c in got if c[2] == 0]
    for act in (BF16, F32):
        for epi in ("none", "swiglu"):
            for m, n, k in SMALL:
                got |= {(act, q, t, s > 1) for q, (t, s) in plans(act, epi, m, n, k).items()}
    want = {(a, k, 0, s) for a in (BF16, F32) for k in ("fwd", "swiglu", "dx", "dw") for s in (False, True)}
    want -= {(BF16, "swiglu", 0, True)}
    assert want <= set(big), sorted(want - set(big))
    want |= {(BF16, k, t, s) for k in ("fwd", "swiglu", "dx", "dw") for t in (1, 2, 3) for s in (False, True)}
    want |= {(F32, k, 1, s) for k in ("fwd", "swiglu", "dx", "dw") for s in (False, True)}
    want |= {(a, k, 4, False) for a in (BF16, F32) for k in ("fwd", "swiglu")}
    assert want <= got, sorted(want - got)


def on_gpu(c, monkeypatch):
    """The case's tensors on the GPU, so that its references are formed there."""
    for n in ("x", "w", "bias", "res", "dy", "pre", "dx_add", "dw_add"):
        setattr(c, n, getattr(c, n).to(DEV))
    near = test_linear.near
    monkeypatch.setattr(test_linear, "near", lambda got, want, tol, name: near(got, want.cpu(), torch.as_tensor(tol).cpu(), name))
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("act,epi,M,N,K", FORWARD)
def test_forward_tiles(act, epi, M, N, K, monkeypatch):
    print("case linear tiles fwd", act, epi, M, N, K, flush=True)
    c = on_gpu(Case(M, N, K, act, epi), monkeypatch)
    c.check_forward()
    c.check_forward(bias=False, res=False)


@pytest.mark.gpu
@pytest.mark.parametrize("act,epi,M,N,K", BACKWARD)
def test_backward_tiles(act, epi, M, N, K, monkeypatch):
    print("case linear tiles bwd", act, epi, M, N, K, flush=True)
    for wgrad_f32 in ((True, False) if act == BF16 else (False,)):
        on_gpu(Case(M, N, K, act, epi, wgrad_f32=wgrad_f32), monkeypatch).check_backward(add=wgrad_f32 or act == F32)
        monkeypatch.undo()


@pytest.mark.gpu
@pytest.mark.parametrize("act,M,N,K", [(BF16, 1033, 7208, 264), (F32, 1795, 8480, 40)])
def test_large_tiles_keep_to_their_rows(act, M, N, K):
    """A NaN in a row of x and an infinity in one of w reach that row and column only; rows around y and dx stay."""
    assert plan("fwd", act, "none", M, N, K)[0] == 0
    c = Case(M, N, K, act, "none")
    x, w = c.x.to(DEV), c.w.to(DEV)
    y = c.new(M, N)
    c.mok.linear_forward(c.d, x, w, y, ws=c.fws)
    x[700, K - 3], w[511, 2] = float("nan"), float("inf")
    big = torch.full((M + 2, N), 3.0, dtype=c.t, device=DEV)
    c.mok.linear_forward(c.d, x, w, big[1:-1], ws=c.fws)
    keep = torch.ones(M, N, dtype=torch.bool, device=DEV)
    keep[700], keep[:, 511] = False, False
    assert torch.equal(big[1:-1][keep], y[keep])
    assert not torch.isfinite(big[1:-1][~keep]).any()
    assert (big[0] == 3).all() and (big[-1] == 3).all()


@pytest.mark.gpu
def test_large_tiles_captured_repeated_and_in_place():
    """One training step of a SwiGLU product on the largest tiles: the same bits eagerly, again, over its addends and from
    a graph replayed between eager steps."""
    M, N, K = 2959, 1440, 2856
    p = plans(BF16, "swiglu", M, N, K)
    assert p["swiglu"][0] == p["dx"][0] == p["dw"][0] == 0, p
    c = Case(M, N, K, BF16, "swiglu")
    x, w, dy, pre, ax, aw = (v.to(DEV) for v in (c.x, c.w, c.dy, c.pre, c.dx_add, c.dw_add))
    outs = y, q, dx, dw, db = c.new(M, N), c.new(M, 2 * N), c.new(M, K), c.new(2 * N, K), c.new(2 * N, dtype=torch.float32)

    def step():
        c.mok.linear_forward(c.d, x, w, y, pre=q, ws=c.fws)
        c.mok.linear_backward(c.d, dy, x, w, dx=dx, dw=dw, db=db, pre=q, dx_add=ax, dw_add=aw, ws=c.bws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.mul_(0.75)
        step()
        want = [v.clone() for v in outs]
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))
    c.mok.linear_backward(c.d, dy, x, w, dx=ax, dw=aw, db=db, pre=q, dx_add=ax, dw_add=aw, ws=c.bws)
    assert torch.equal(ax, dx) and torch.equal(aw, dw)
