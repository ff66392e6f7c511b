"""Gradients whose sizes differ from row to row and from step to step: what f16 holds of them (needs a B200)."""
import numpy as np
import pytest
import torch

import oracle
import train_ref as R
from joint_attention_block_b200 import ops, synth
from test_gpu_train import FMTS, _clean_errors, config, gen, randn  # noqa: F401
from train_ref import nan_like, run_backward, run_forward, within, ws

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


@FMTS
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_gradient_beyond_the_range_is_an_infinity(hd, fmt):
    """Every query attends to key 0, whose dv is the sum of 300 rows of 2^14 (f16: beyond 65504); in bf16 it is finite."""
    S = 300
    q, k = torch.full((1, S, hd), 2.0, device="cuda", dtype=R.DT[fmt]), torch.zeros(1, S, hd, device="cuda", dtype=R.DT[fmt])
    k[:, 0] = 2.0
    v = randn(gen(229), 1, S, hd, fmt=fmt)
    do = torch.full_like(q, 2.0 ** 14)
    out, lse = run_forward(q, k, v, 1, hd, fmt)
    g = run_backward(q, k, v, out, do, lse, 1, hd, fmt)
    dv = g[..., 2 * hd:]
    if fmt == 1:
        assert (dv[:, 0] == float("inf")).all()
    else:
        assert ((dv[:, 0].double() - S * 2.0 ** 14).abs() <= 3 * R.U[fmt] * S * 2.0 ** 14).all()
    assert torch.isfinite(dv[:, 1:]).all()


@FMTS
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_gradient_of_an_infinity_is_not_finite(hd, fmt):
    """An infinity in dout reaches every gradient it enters, and nothing of the other heads and elements."""
    B, S, H = 2, 333, 3
    d, g = H * hd, gen(233)
    q, k, v = (randn(g, B, S, d, fmt=fmt) for _ in range(3))
    do = randn(g, B, S, d, std=0.02, fmt=fmt)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    ref = run_backward(q, k, v, out, do, lse, H, hd, fmt).view(B, S, 3, H, hd)
    do[0, 7, hd + 3] = float("inf")
    got = run_backward(q, k, v, out, do, lse, H, hd, fmt).view(B, S, 3, H, hd)
    assert not torch.isfinite(got[0, 7, 0, 1]).any()       # its own row of dq
    assert not torch.isfinite(got[0, :, 1, 1]).any()       # every row of dk
    assert not torch.isfinite(got[0, :, 2, 1, 3]).any()    # its channel of dv
    assert torch.equal(got[1], ref[1]) and torch.equal(got[0, :, :, ::2], ref[0, :, :, ::2])


def test_elementwise_gradients_beyond_the_range_are_infinities():
    """Rows of zeros, whose gradient is dy / sqrt(eps) = 1000 dy: 1e5 in f16."""
    hd, H, fmt = 64, 4, 1
    d = H * hd
    cfg, one = config(H, hd), torch.ones(hd, device="cuda").bfloat16()
    qkv, dqk = torch.zeros(1, 9, 3 * d, device="cuda").half(), torch.full((1, 9, 2 * d), 100.0, device="cuda").half()
    dx, dg = nan_like(1, 9, 2 * d, fmt=fmt), [nan_like(hd, fmt=2) for _ in range(2)]
    ops.qknorm_mrope_backward(qkv, dqk, dx, cfg, 9, 0, 0, one, one, *dg, ws(ops.qknorm_mrope_backward_workspace_bytes(cfg, 1, 9)),
                              fmt=fmt)
    assert (dx[:, 0] == float("inf")).all()  # token 0, whose rotation is none
    for rows, cols in ((5, 256), (5, 2048)):
        x, dy = torch.zeros(rows, cols, device="cuda").bfloat16(), torch.full((rows, cols), -100.0, device="cuda").half()
        gain, dx, dg = torch.ones(cols, device="cuda").bfloat16(), nan_like(rows, cols, fmt=1), nan_like(cols, fmt=2)
        ops.rmsnorm_rows_backward(x, gain, dy, dx, dg, 1e-6, ws(ops.rmsnorm_rows_backward_workspace_bytes(rows, cols)), dy_fmt=1,
                                  dx_fmt=1)
        assert (dx == -float("inf")).all()
