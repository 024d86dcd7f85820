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
