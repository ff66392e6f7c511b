"""Gradients whose sizes differ from row to row and from step to step: what f16 holds of them (needs a B200)."""
import numpy as np
import pytest
import torch

import oracle
import train_ref as R
from joint_attention_block_b200 import ops, synth
from test_gpu_train import FMTS, _clean_errors, gen, randn  # noqa: F401
from train_ref import run_backward, run_forward, within

pytestmark = pytest.mark.gpu


@FMTS
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_backward_of_rows_of_different_size(hd, fmt):
    """Two rows of dO 2^24 times the others.  Each row of dQ depends on its own row of dO alone, so the small rows'
    bounds are those of the same formula on these rows by themselves (the scale below which f16 rounds dS coarsely
    comes from their own largest norm)."""
    B, S, H = 2, 700, 2
    d, g = H * hd, gen(211)
    q, k, v = randn(g, B, S, d, std=0.125, fmt=fmt), randn(g, B, S, d, std=8.0, fmt=fmt), randn(g, B, S, d, fmt=fmt)
    do = randn(g, B, S, d, std=2.0 ** -10, fmt=fmt)
    big = [5, 300]
    do[:, big] = randn(g, B, 2, d).sign().to(do.dtype) * 2.0 ** 14
    small = [i for i in range(S) if i not in big]
    out, lse = run_forward(q, k, v, H, hd, fmt)
    grads = run_backward(q, k, v, out, do, lse, H, hd, fmt)
    hq, hk, hv, ho, hdo = (R.heads(t, H) for t in (q, k, v, out, do))
    got = [R.heads(grads[..., i * d:(i + 1) * d], H) for i in range(3)]
    ref, tol = R.attention_grad_bounds(hq, hk, hv, ho, hdo, lse.double(), fmt)
    for i, name in enumerate(("dq", "dk", "dv")):
        within(got[i], ref[i], tol[i], name)
    ref, tol = R.attention_grad_bounds(hq[:, :, small], hk, hv, ho[:, :, small], hdo[:, :, small],
                                       lse[..., small].double(), fmt)
    within(got[0][:, :, small], ref[0], tol[0], "dq of the small rows")


def weight(seed, rows, cols):
    """Frozen e4m3 codes [rows, cols], their row scales of several sizes, and the fp64 values."""
    w = synth.normal(13, seed, (rows, cols), std=0.04) * np.exp2(np.arange(rows) % 4)[:, None].astype(np.float32)
    codes, scale = synth.quantize_rows_e4m3(w)
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(),
            torch.from_numpy(oracle.dequant(codes, scale)).double().cuda())


@FMTS
@pytest.mark.parametrize("std", [1e-4, 1e-2, 1.0])
@pytest.mark.parametrize("N,K", [(768, 256), (256, 1024)])
def test_gradient_through_a_frozen_product(N, K, std, fmt):
    """dx = dy W of y = x W^T: the transposed codes, dy scale / max(scale) as the operand and max(scale) as every output
    channel's scale.  (dy scale itself lies below f16's normal range already at dy = 0.1.)"""
    M = 333
    w8, scale, w = weight(N + K, N, K)
    dy = randn(gen(223), M, N, std=std, fmt=fmt)
    top = scale.max()
    a = (dy.float() * (scale / top)).to(dy.dtype)
    dx = torch.full((M, K), float("nan"), dtype=torch.float32, device="cuda")
    ops.gemm_w8a16(a, w8.t().contiguous(), top.repeat(K), dx, a_fmt=fmt, y_fmt=2)
    ref = dy.double() @ w
    # the operand's rounding (relative, or half of the format's last step below its normal range), the fp32 quotient's
    # and product's, N additions in fp32
    size = dy.double().abs() @ w.abs()
    low = R.TINY[fmt] * (w.abs() * (top / scale).double()[:, None]).sum(0)
    within(dx, ref, (R.U[fmt] + (N + 8) * 2.0 ** -24) * size + low, "dx")
