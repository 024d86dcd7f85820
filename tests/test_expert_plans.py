"""Grouped products and products with 4-bit weights at shapes that their plans send to each kernel, tile and number of
slices, ragged in every direction; and checks that none is left out. References in fp64 and tolerances of test_grouped.py
and test_q4.py."""
import ctypes

import pytest
import torch

import test_grouped
import test_linear
import test_q4
from test_linear import DEV

BF16, F32 = "bf16", "f32"
Grouped, Q4 = test_grouped.Case, test_q4.Case


def grouped_plan(kind, act, epi, M, N, K, E):
    """(tile, slices of the rows) of a grouped product: grouped_plan (csrc/grouped.h) of the built library."""
    mok = test_linear._mok()
    f = mok._lib._ZN3mok12grouped_planEiiilili
    f.restype = ctypes.c_uint64
    f.argtypes = [ctypes.c_int] * 3 + [ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_int]
    v = f(("fwd", "dx", "dw").index(kind), mok.DTYPES[act], mok.EPILOGUES[epi], M, N, K, E)
    return v & 0xffffffff, v >> 32


def grouped_plans(act, epi, M, N, K, E):
    P = 2 * N if epi == "swiglu" else N
    return {"swiglu" if epi == "swiglu" else "fwd": grouped_plan("fwd", act, epi, M, N, K, E),
            "dx": grouped_plan("dx", act, "none", M, K, P, E), "dw": grouped_plan("dw", act, "none", P, K, M, E)}


def q4_split(act, epi, M, N, K, E=1):
    """0: the kernel for few rows; else tiles, in so many slices of K (csrc/q4.h). Groups, one among them: E > 1."""
    mok = test_linear._mok()
    f = mok._lib._ZN3mok8q4_splitEiiliii
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_int] * 2 + [ctypes.c_int64] + [ctypes.c_int] * 3
    return f(mok.DTYPES[act], mok.EPILOGUES[epi], M, N, K, E)


# ---- grouped products ----

# act, epi, rows of the groups, N, K; four rows in front of the groups and three behind them
GROUPED = [
    (F32, "none", [9000, 0, 12500, 1, 10700], 216, 64), (F32, "gelu", [9000, 0, 12500, 1, 10700], 216, 72),   # 128 x 128 forward
    (F32, "swiglu", [18000, 12782], 72, 112), (F32, "none", [9000, 11500, 0, 12000], 80, 216),              # and dx
    (F32, "swiglu", [9000, 11500, 0, 12000], 80, 216), (F32, "silu", [9000, 0, 23493], 80, 232),
    (F32, "none", [30, 0, 1, 33, 5] * 4, 72, 4904), (F32, "swiglu", [30, 0, 1, 33, 5] * 4, 40, 4904),        # and dw
    (BF16, "none", [40, 0, 1, 34, 23] * 4, 72, 136), (BF16, "silu", [40, 0, 1, 34, 23] * 4, 72, 152),        # 32-row kernel
    (BF16, "none", [3000, 0, 64, 1, 129, 2000, 2500, 31, 6000, 1200, 3333, 2301], 2888, 136),              # 256 x 256 dw
    (BF16, "swiglu", [3000, 0, 64, 1, 129, 2000, 2500, 31, 6000, 1200, 3333, 2301], 1448, 136),
    (BF16, "none", [11000, 8360], 4240, 144), (BF16, "swiglu", [11000, 8360], 2120, 144),                   # in slices
    (BF16, "none", [33, 0, 1, 97, 0, 20, 64, 5] * 3, 1048, 264), (BF16, "gelu", [33, 0, 1, 97, 0, 20, 64, 5] * 3, 1048, 264),
    (BF16, "swiglu", [33, 0, 1, 97, 0, 20, 64, 5] * 3, 520, 392),                                           # 32-row K-tiles of dw
    (BF16, "none", [1001], 64, 72),                                                                  # small dw in slices
]


def test_every_grouped_kernel_is_reached():
    """By the shapes here and the small ones of test_grouped.py: each type, product and tile, dw also in slices. 4, 5: the
    kernels of 16 and 32 rows, 6: dw by K-tiles of 32 rows."""
    cases = [(a, e, 4 + sum(c) + 3, N, K, len(c)) for a, e, c, N, K in GROUPED]
    cases += [(a, e, lead + sum(c) + tail, N, K, len(c)) for c, N, K, lead, tail in test_grouped.SMALL for a in (BF16, F32)
              for e in ("none", "swiglu")]
    cases += [(a, e, 3 + sum(c), N, K, len(c)) for a, e in ((BF16, "none"), (BF16, "swiglu")) for c, N, K in  # test_larger
              (([1000, 24, 0, 1024], 1024, 512), ([4100], 264, 1032), ([2500, 3000], 776, 520))]
    cases += [(BF16, e, 6084, N, K, 24) for N, K, e in ((2048, 1024, "none"), (1032, 1032, "swiglu"))]        # heights
    got = {(c[0], k, t, s > 1) for c in cases for k, (t, s) in grouped_plans(*c).items()}
    want = {(BF16, k, t, False) for k in ("fwd", "swiglu", "dx", "dw") for t in range(4)} | {(BF16, "dw", 6, False)}
    want |= {(F32, k, t, False) for k in ("fwd", "swiglu", "dx", "dw") for t in range(2)}
    want |= {(BF16, "dw", t, True) for t in range(4)} | {(F32, "dw", 1, True)}
    want |= {(a, k, t, False) for a in (BF16, F32) for k in ("fwd", "swiglu") for t in (4, 5)}
    assert want <= got, sorted(want - got)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(GROUPED)))
def test_grouped_kernels(i):
    act, epi, counts, N, K = GROUPED[i]
    print("case grouped plans", i, act, epi, len(counts), sum(counts), N, K, flush=True)
    for wgrad_f32 in ((True, False) if act == BF16 else (False,)):
        c = Grouped(counts, N, K, act, epi, lead=4, tail=3, wgrad_f32=wgrad_f32)
        c.check_backward(add=wgrad_f32 or act == F32)
        first = c.backward(add=False)
        assert all(torch.equal(a, b) for a, b in zip(first, c.backward(add=False)))  # the same bits again
    c.check_forward(bias=i % 2 == 0, res=i % 2 == 1)


@pytest.mark.gpu
@pytest.mark.parametrize("act,epi,counts,N,K", [GROUPED[3], GROUPED[10], GROUPED[12], GROUPED[14]])
def test_grouped_kernels_keep_to_their_groups(act, epi, counts, N, K):
    """What is not finite in one group's rows and weights stays in that group's outputs, on the large tiles too."""
    c = Grouped(counts, N, K, act, epi, lead=4, tail=3)
    clean, grads = c.forward(bias=False, res=False)[0].cpu(), [v.cpu() for v in c.backward(add=False)]
    e = max(range(len(counts) - 1), key=lambda i: counts[i])
    lo, hi = c.off[e], c.off[e + 1]
    for v in (c.x, c.dy, c.pre):
        v[lo:hi] = float("nan")
    c.w[e] = float("inf")
    got, bad = c.forward(bias=False, res=False)[0].cpu(), [v.cpu() for v in c.backward(add=False)]
    keep = torch.ones(c.d.M, dtype=torch.bool)
    keep[lo:hi] = False
    others = [g for g in range(len(counts)) if g != e]
    assert torch.equal(got[keep], clean[keep]) and torch.equal(bad[0][keep], grads[0][keep])
    assert torch.equal(bad[1][others], grads[1][others]) and torch.equal(bad[2][others], grads[2][others])


# ---- products with 4-bit weights ----

# act, epi, rows, N, K, group: tiles in 1, 2, 4, 8, 16 and 32 slices of K, which divide its pieces of 128 or do not,
# with groups of 32 that end in half a K-tile
SLICED = [
    (BF16, "none", 203, 4104, 96, 32), (BF16, "swiglu", 390, 1032, 192, 64), (BF16, "gelu", 390, 2056, 128, 128),
    (BF16, "none", 260, 7176, 2080, 32), (BF16, "swiglu", 100, 7176, 2112, 64), (BF16, "silu", 260, 7176, 2176, 128),
    (BF16, "gelu", 391, 1544, 992, 32), (BF16, "none", 389, 2056, 960, 64), (BF16, "swiglu", 65, 4104, 1024, 128),
    (BF16, "swiglu", 701, 264, 2080, 32), (BF16, "silu", 700, 520, 2112, 64), (BF16, "none", 699, 520, 2048, 128),
    (BF16, "swiglu", 21, 2056, 7200, 32), (BF16, "none", 20, 4104, 7232, 64), (BF16, "gelu", 129, 4104, 7168, 128),
    (BF16, "none", 21, 2056, 14368, 32), (BF16, "swiglu", 130, 1032, 7168, 128), (BF16, "swiglu", 20, 1032, 14400, 64),
    (BF16, "silu", 390, 4104, 192, 64), (BF16, "swiglu", 203, 2056, 96, 32), (BF16, "swiglu", 390, 1032, 128, 128),
    (F32, "none", 700, 2056, 192, 64), (F32, "swiglu", 700, 1032, 96, 32), (F32, "swiglu", 701, 1032, 256, 128),
    (F32, "none", 700, 2056, 96, 32), (F32, "swiglu", 701, 1032, 192, 64), (F32, "gelu", 700, 2056, 128, 128),
    (F32, "silu", 130, 7176, 1056, 32), (F32, "swiglu", 100, 4104, 1088, 64), (F32, "none", 65, 7176, 1024, 128),
    (F32, "swiglu", 261, 1032, 992, 32), (F32, "none", 700, 520, 2112, 64), (F32, "swiglu", 700, 264, 2048, 128),
    (F32, "gelu", 700, 136, 7200, 32), (F32, "swiglu", 130, 520, 5184, 64), (F32, "none", 67, 776, 14336, 128),
]
# act, epi, rows of the groups, N, K, group: tiles of ragged groups
TILED = [(BF16, "none", [0, 300, 5, 0, 131], 2056, 288, 32), (BF16, "swiglu", [257, 0, 1, 128, 40], 1032, 320, 64),
         (BF16, "gelu", [700, 3, 129], 776, 640, 128), (F32, "none", [0, 600, 5, 0, 231], 2056, 288, 32),
         (F32, "swiglu", [557, 0, 1, 128, 240], 1032, 320, 64), (F32, "silu", [1400, 3, 229], 1032, 640, 128)]
# The kernel for few rows: one, two or eight waves on a tile of w, x in LDS as a whole or in stages
FEW = [(BF16, "none", [16, 0, 3, 1] * 16, 776, 4224, 128), (BF16, "swiglu", [12, 1, 0, 2] * 10, 776, 4128, 32),
       (BF16, "swiglu", [16] * 6, 776, 4160, 64), (BF16, "none", [16] * 12, 776, 4128, 32), (BF16, "gelu", [16, 3], 264, 4224, 128),
       (BF16, "swiglu", [16, 3], 136, 5152, 32), (F32, "none", [16] * 40, 1032, 2112, 64), (F32, "swiglu", [16] * 24, 776, 2080, 32),
       (F32, "swiglu", [16] * 6, 776, 2176, 128), (F32, "silu", [16] * 12, 776, 2080, 32), (F32, "none", [16, 3], 264, 2112, 64),
       (F32, "swiglu", [16, 3], 136, 2144, 32), (F32, "none", [1, 3, 0, 16] * 40, 520, 256, 128), (F32, "none", [2, 1, 0, 5] * 12, 520, 288, 32),
       (BF16, "none", [1, 3, 0, 16] * 40, 520, 320, 64), (BF16, "none", [2, 1, 0, 5] * 12, 520, 288, 32)]


def few_form(act, epi, counts, N, K):
    """(waves that share a tile of w, x comes in stages) of the kernel for few rows, by the rule of q4_few.hip for groups."""
    E, M = len(counts), sum(counts)
    tiles = (N // 8 if epi == "swiglu" else (N + 15) // 16) * (M // 16 + min(E, M))
    rows = 1
    while rows < min(16, max(counts)):
        rows *= 2
    staged = (K + 127) // 128 * rows * (256 if act == BF16 else 512) > 128 << 10
    return 1 if tiles >= 4096 else 2 if tiles >= 1024 else 8, staged


def test_every_4bit_kernel_is_reached():
    sw = lambda epi: epi == "swiglu"
    dense = [(c, q4_split(c[0], c[1], *c[2:5])) for c in SLICED]
    got = {(c[0], sw(c[1]), c[5], s > 1) for c, s in dense if s > 0}
    assert got == {(a, w, g, s) for a in (BF16, F32) for w in (False, True) for g in (32, 64, 128) for s in (False, True)}, got
    assert {(c[0], s) for c, s in dense} == {(a, s) for a in (BF16, F32) for s in (1, 2, 4, 8, 16, 32)}, dense
    assert any((c[4] + 127) // 128 % s for c, s in dense) and any(c[4] % 64 == 32 and s > 1 for c, s in dense)
    assert {q4_split(c[0], c[1], sum(c[2]), c[3], c[4], len(c[2])) for c in TILED} == {1}
    assert {q4_split(c[0], c[1], sum(c[2]), c[3], c[4], len(c[2])) for c in FEW} == {0}
    got = {(c[0], *few_form(*c[:5])) for c in FEW}
    assert got == {(a, ws, st) for a in (BF16, F32) for ws in (1, 2, 8) for st in (False, True)} - {(a, 8, False) for a in (BF16, F32)}
    # eight waves and x as a whole: the dense shapes of test_q4.py
    assert all(q4_split(a, e, *c[:3]) == 0 for c in test_q4.DENSE for a in (BF16, F32) for e in ("none", "swiglu"))


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(SLICED)))
def test_4bit_dense_tiles_and_slices(i):
    act, epi, M, N, K, G = SLICED[i]
    print("case q4 slices", i, act, epi, M, N, K, G, q4_split(act, epi, M, N, K), flush=True)
    c = Q4(M, N, K, G, act, epi, zeros=i % 2 == 0)
    assert (c.mok.q4_workspace_query(c.d)["fwd_ws"] > 0) == (q4_split(act, epi, M, N, K) > 1)
    c.check()
    c.check(bias=i % 2 == 1, res=i % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(TILED)))
def test_4bit_tiles_of_groups(i):
    act, epi, counts, N, K, G = TILED[i]
    print("case q4 tiles", i, act, epi, sum(counts), N, K, G, flush=True)
    c = Q4(counts, N, K, G, act, epi, zeros=i % 2 == 0, lead=3, tail=2)
    c.check()
    c.check(bias=i % 2 == 1, res=i % 2 == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(FEW)))
def test_4bit_few_rows(i):
    act, epi, counts, N, K, G = FEW[i]
    print("case q4 few", i, act, epi, len(counts), sum(counts), N, K, G, flush=True)
    c = Q4(counts, N, K, G, act, epi, zeros=i % 2 == 0)
    c.check(bias=i % 2 == 1, res=i % 2 == 0)
    first = c.forward()
    assert all(torch.equal(first, c.forward()) for _ in range(3))


@pytest.mark.gpu
@pytest.mark.parametrize("act,epi,rows,N,K,G", [SLICED[0], SLICED[3], SLICED[12], SLICED[29], SLICED[31], *TILED])
def test_4bit_tiles_keep_to_their_rows_and_groups(act, epi, rows, N, K, G):
    """A row of x or a scale that is not finite reaches its row and its column (of its group) only."""
    c = Q4(rows, N, K, G, act, epi, True)
    clean = c.forward(bias=False, res=False).cpu()
    e = len(c.off) - 2
    c.s[e, 7, -1] = float("inf")
    c.x[c.off[e] + 1, K - 1], c.x[c.off[e] + 2, 0] = float("inf"), float("nan")
    got = c.forward(bias=False, res=False).cpu()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[c.off[e] + 1:c.off[e] + 3] = False
    keep[c.off[e]:c.off[e + 1], 7] = False
    assert torch.equal(got[keep], clean[keep])
    assert torch.isnan(got[c.off[e] + 2]).all()
    if epi == "none":
        assert not torch.isfinite(got[c.off[e]:c.off[e + 1], 7]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,G,few", [(5, 72, 256, 64, True), (600, 72, 256, 64, True), (2048, 264, 544, 32, True),
                                         (4096, 136, 128, 128, True), (390, 2056, 128, 128, False), (700, 520, 2112, 64, False)])
def test_4bit_infinity_in_a_bf16_row(M, N, K, G, few):
    """The kernel for few rows, which small matrices take at any number of rows, gives NaN in that row, tiles an infinity of
    w's sign and NaN where w is 0."""
    assert (q4_split(BF16, "none", M, N, K) == 0) == few
    c = Q4(M, N, K, G, BF16, "none", True)
    clean = c.forward(bias=False, res=False).cpu()
    c.x[3, K - 1] = float("inf")
    got = c.forward(bias=False, res=False).cpu()
    w = c.s[0, :, -1].float() * (c.code[0, :, -1].float() - c.z[0, :, -1].float())
    want = torch.full((N,), float("nan")) if few else w * float("inf")
    assert torch.equal(torch.isnan(got[3]), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got[3].float(), nan=0.0, posinf=1.0, neginf=-1.0),
                       torch.nan_to_num(want, nan=0.0, posinf=1.0, neginf=-1.0))
    got[3] = clean[3]
    assert torch.equal(got, clean)


@pytest.mark.gpu
@pytest.mark.parametrize("act,epi,rows,N,K,G", [SLICED[2], SLICED[4], SLICED[12], SLICED[34], *TILED[1:3]])
def test_4bit_tiles_in_place_captured_and_on_another_stream(act, epi, rows, N, K, G):
    """The residual's array as the output's, a stream of its own, and two graphs that share the slices' workspace."""
    c = Q4(rows, N, K, G, act, epi, True)
    dev = lambda v: v.to(DEV)
    want, same = c.forward(), dev(c.res).clone()
    x, q, s, z, b, r = (dev(v) for v in (c.x, c.q, c.s, c.z, c.bias, c.res))
    ws = torch.empty(max(c.mok.q4_workspace_query(c.d)["fwd_ws"], 16), dtype=torch.uint8, device=DEV)
    go = lambda y, res: c.mok.q4_forward(c.d, x, q, s, y, z=z, off=c.goff, bias=b, res=res, ws=ws)
    go(same, same)
    assert torch.equal(want, same)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = c.forward()
    st.synchronize()
    assert torch.equal(want, other)
    ys, graphs = [torch.empty_like(want) for _ in range(2)], []
    for y in ys:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            go(y, r)
    for _ in range(3):
        x.mul_(0.75)
        eager = torch.empty_like(want)
        go(eager, r)
        for y, graph in zip(ys, graphs):
            y.fill_(test_q4.KEEP)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, ys[0]) and torch.equal(eager, ys[1])


@pytest.mark.gpu
@pytest.mark.parametrize("act,epi,M,N", [(BF16, "none", 1800, 1032), (BF16, "swiglu", 1800, 520), (F32, "none", 1800, 1032)])
def test_4bit_tiles_with_offsets_that_descend_or_pass_the_rows_stay_inside(act, epi, M, N):
    K, E, G = 128, 6, 32
    assert q4_split(act, epi, M, N, K, E) == 1
    mok = test_linear._mok()
    t = mok.TORCH_DTYPE[mok.DTYPES[act]]
    d = mok.Q4Desc(M, N, K, E, G, act=mok.DTYPES[act], epi=mok.EPILOGUES[epi])
    z = lambda *s, dtype=t: torch.zeros(*s, dtype=dtype, device=DEV)
    x, q, s = z(M, K), z(E, d.P, K // 2, dtype=torch.uint8), z(E, d.P, K // G)
    for off in ([-5, M + 70, 10, 200, -1, 3, 1 << 30], [M, 1500, 1200, 900, 600, 300, 0], [(1 << 31) - 1] * 7, [-(1 << 31)] * 7):
        print("case q4 tiles bad offsets", act, epi, off, flush=True)
        y = torch.ones(M + 2, N, dtype=t, device=DEV)
        mok.q4_forward(d, x, q, s, y[1:-1], off=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert (y[0] == 1).all() and (y[-1] == 1).all()
