"""Calls at the ends of what the operators around the layer take."""
import pytest
import torch

DEV = "cuda"


def _mok():
    from mixture_experts_layer_stable_amd import mok
    return mok


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
