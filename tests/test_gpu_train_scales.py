"""Gradients whose sizes differ from row to row and from step to step: what f16 holds of them (needs a B200)."""
import pytest
import torch

import train_ref as R
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
