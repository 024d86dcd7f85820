"""Calls at the ends of what the operators around the layer take."""
import pytest
import torch

DEV = "cuda"


def _mok():
    from mixture_experts_layer_stable_amd import mok
    return mok


@pytest.mark.gpu
def test_norm_of_rows_with_subnormal_squares():
    """Powers of two, whose squares and sums are exact also where they are subnormal: rstd is off by its own rounding,
    half a step of 2^-24, y by that, its product's and its own."""
    mok = _mok()
    H = 256
    x = torch.ones(6, H, device=DEV)
    for i, e in enumerate((-62, -63, -64, -66, -70)):   # mean squares 2^-124 (normal) .. 2^-140
        x[i] *= 2.0**e
        x[i, ::2] *= -1
        x[i, ::4] *= 2
    x[5] = 0
    for eps in (0.0, 1e-39):
        d = mok.NormDesc(6, H, act=mok.F32, eps=eps)
        y, rstd = torch.full_like(x, float("nan")), torch.full((6,), float("nan"), device=DEV)
        mok.rmsnorm_forward(d, x, torch.ones(H, device=DEV), y=y, rstd=rstd)
        e64 = float(torch.tensor(eps, dtype=torch.float32).double())
        # the mean plus eps is rounded to fp32: below 2^-126 to a multiple of 2^-149
        mean = (x.double().square().mean(-1) + e64).float().double()
        want = 1 / torch.sqrt(mean)
        live = mean > 0
        assert live.sum() == (6 if eps else 5)
        assert ((rstd.double() - want).abs() <= 2.0**-24 * 1.01 * want)[live].all(), (rstd, want)
        ref = x.double() * want[:, None]
        assert ((y.double() - ref).abs() <= 3.03 * 2.0**-24 * ref.abs())[live].all()
    assert (y[5] == 0).all()          # eps = 1e-39: a zero row stays one


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,cuts", [
    (4096, 8, 2, [0] + [1001] * 5000 + [4096]), (4096, 8, 2, [0, 256] + [300] * 4000 + [301] + [512] * 100 + [600] * 100 + [4096]),
    (700, 384, 4, [5] * 70 + [33] * 200 + [34] * 64 + [698]), (40, 16, 2, [7] * 65 + [8] * 130 + [39] * 3 + [40] * 70),
])
def test_balance_with_runs_of_empty_sequences(T, E, k, cuts, score):
    from test_balance import Run, check, inputs
    print("case balance empties", T, E, len(cuts) - 1, score, flush=True)
    z, idx, dl, g = inputs(T, E, k, T + E)
    seg = torch.tensor(cuts, dtype=torch.int32, device=DEV)
    mask = (torch.rand(T, generator=g) < 0.8).to(DEV)
    soft = score == "softmax"
    check(Run(T, E, k, len(cuts) - 1, score, "f32", zcoef=0.1 if soft else 0.0), z, idx, dl, seg, mask, soft)


@pytest.mark.gpu
def test_empty_sequences_cost_the_same_wherever_they_lie():
    """60000 empty sequences in the middle of the tokens take no longer than behind the last token (which is what the
    second launch takes for them); one after the other they would be 60000 dependent loads."""
    from test_balance import Run, inputs
    T, E, k, S = 4096, 8, 2, 60000
    z, idx, dl, _ = inputs(T, E, k, 1)
    us = {}
    for name, cuts in (("behind", [0, 1001] + [T] * (S - 1)), ("inside", [0] + [1001] * (S - 1) + [T])):
        seg = torch.tensor(cuts, dtype=torch.int32, device=DEV)
        run, times = Run(T, E, k, S, "softmax", "f32"), []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            run.mok.balance_forward(run.d, z, idx, run.loss, run.counts, run.tokens, run.prob, run.stat, run.ws, seg=seg)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 1e3)
        us[name] = sorted(times)[2]
    print("60000 empty sequences, us:", us, flush=True)
    assert us["inside"] < 3 * us["behind"], us


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(2048, 8), (256, 64)])
def test_small_batches_of_many_sequences_take_the_faster_path(T, E):
    """64 sequences in one workgroup would take two to four times as long as 65, which are too many for it."""
    from test_balance import Run, inputs
    us = {}
    for S in (64, 65):
        z, idx, _, _ = inputs(T, E, 2, 1)
        seg = torch.linspace(0, T, 65).int().tolist() + [T] * (S - 64)
        run, times = Run(T, E, 2, S, "softmax", "f32"), []
        seg = torch.tensor(seg, dtype=torch.int32, device=DEV)
        for _ in range(11):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                run.mok.balance_forward(run.d, z, idx, run.loss, run.counts, run.tokens, run.prob, run.stat, run.ws, seg=seg)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 100)
        us[S] = sorted(times)[5]
    print("sequences, us:", us, flush=True)
    assert us[64] < 1.4 * us[65], us


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 2, 3, 4])
def test_a_small_batch_adds_its_waves_in_64_bits(E):
    """T * E at the limit of one workgroup. The first of every 1024 tokens have p = 1 for expert 0 in the first wave and
    0.4 of a step of that wave's sum, in all, in each other wave: added one after the other in fp32 they would be lost."""
    from test_balance import Run
    k = 1
    T = (1 << 14) // E // 1024 * 1024
    groups = 1024                       # tokens that the workgroup takes at once (one lane each)
    own = T // groups * 64              # tokens of a wave
    z = torch.zeros(T, E, device=DEV)
    tok = torch.arange(T, device=DEV) % groups // 64
    p = 1.0
    if E > 1:
        step = 2.0 ** (own.bit_length() - 1 - 23)
        p = 0.4 * step / own
        z[:, 0] = torch.where(tok == 0, 0.0, torch.log(torch.tensor(p * (E - 1), dtype=torch.float64)).float())
        z[:, 1:] = torch.where(tok == 0, -float("inf"), 0.0)[:, None]
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    run = Run(T, E, k, 0, "softmax", "f32", coef=0.5)
    loss, counts, tokens, prob, _ = run(z, idx, torch.ones(2, device=DEV))
    want = torch.softmax(z.double(), 1).mean(0)
    # p to 2^-20 each (its share of the sum is 15 * 0.4 steps), a wave's sum of equal values within 2^-24 for each of its
    # T / 1024 + 6 additions (of ones: exact); the mean's own rounding
    small = own * 15 * p if E > 1 else 0.0
    tol = 2.0**-24 * want[0] + (2.0**-20 + (T // groups + 6) * 2.0**-24) * small / T
    print("small batch", E, T, float((prob[0, 0].double() - want[0]) / (2.0**-24 * want[0])), flush=True)
    assert (prob[0, 0].double() - want[0]).abs() <= tol * 1.01
    l0 = run.d.coef * E * want[0]       # every slot is expert 0's
    assert (loss[0].double() - l0).abs() <= (tol / want[0] + 2.0**-24) * l0
    assert int(counts[0, 0]) == T and tokens.tolist() == [T, 1, T]


def test_x_quant_views_of_a_ring_given_as_0():
    """mb_count and ring 0 stand for 1."""
    mok = _mok()
    d = mok.Desc(8, 512, 8, 2, 256, gemm=mok.MXFP8, mb_count=0, ring=0)
    ws = torch.zeros(mok.workspace_query(d)["fwd_ws"], dtype=torch.uint8)
    q, s = mok.x_quant_views(d, ws)
    one = mok.Desc(8, 512, 8, 2, 256, gemm=mok.MXFP8)
    q1, s1 = mok.x_quant_views(one, ws)
    assert q.data_ptr() == q1.data_ptr() and s.data_ptr() == s1.data_ptr()
    assert q.shape == (8, 512) and s.shape == (4, 8, 4)
