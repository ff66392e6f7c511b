"""Calls of the training pass that the header allows and the other tests do not make (needs a B200)."""
import pytest
import torch

import train_ref as R
from joint_attention_block_b200 import ops
from test_gpu_train import FMTS, _clean_errors, gen, qk_backward_case, randn  # noqa: F401
from train_ref import nan_like, run_backward, run_forward, within, ws

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [264, 4096])
def test_rmsnorm_gradient_of_the_gain_into_a_slice(cols):
    """The gain's gradient into the middle of a buffer of all parameters' gradients, 4-byte aligned only."""
    g = gen(227)
    x, dy = randn(g, 50, cols, fmt=0), randn(g, 50, cols, std=0.02, fmt=0)
    gain = torch.ones(cols, device="cuda").bfloat16()
    w = ws(ops.rmsnorm_rows_backward_workspace_bytes(50, cols))
    dx, dg = nan_like(50, cols, fmt=0), nan_like(cols, fmt=2)
    ops.rmsnorm_rows_backward(x, gain, dy, dx, dg, 1e-6, w)
    for at in (1, 2, 3):
        flat, dx1 = torch.full((cols + 8,), 7.0, device="cuda"), nan_like(50, cols, fmt=0)
        ops.rmsnorm_rows_backward(x, gain, dy, dx1, flat[at:at + cols], 1e-6, w)
        assert torch.equal(flat[at:at + cols], dg) and torch.equal(dx1, dx)
        assert (flat[:at] == 7.0).all() and (flat[at + cols:] == 7.0).all()
    none = torch.empty(0, cols, device="cuda", dtype=torch.bfloat16)
    ops.rmsnorm_rows_backward(none, gain, none, none.clone(), flat[1:1 + cols], 1e-6, w)
    assert not flat[1:1 + cols].any() and flat[0] == 7.0


@FMTS
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_of_one_tensor_in_every_place(hd, fmt):
    """q, k and v the same tensor, dout the forward's own output: inputs may share memory."""
    B, S, H = 2, 190, 2
    d = H * hd
    x = randn(gen(239), B, S, d, std=0.5, fmt=fmt)
    out, lse = run_forward(x, x, x, H, hd, fmt)
    g = run_backward(x, x, x, out, out, lse, H, hd, fmt)
    hx, ho = R.heads(x, H), R.heads(out, H)
    ref, ref_lse, tol, tol_lse = R.attention_bounds(hx, hx, hx, fmt)
    within(ho, ref, tol, "out")
    within(lse, ref_lse, tol_lse, "lse")
    ref, tol = R.attention_grad_bounds(hx, hx, hx, ho, ho, lse.double(), fmt)
    for i, name in enumerate(("dq", "dk", "dv")):
        within(R.heads(g[..., i * d:(i + 1) * d], H), ref[i], tol[i], name)


@FMTS
def test_attention_of_single_rows(fmt):
    """Elements of one row, taken from buffers whose elements lie further apart: P = 1, so dq = dk = 0 up to what out's
    rounding leaves in delta, and dv = dout."""
    B, H, hd = 300, 3, 64
    d, g = H * hd, gen(241)
    q, k, v = randn(g, B, 1, 2 * d, fmt=fmt)[..., d:], randn(g, B, 1, 3 * d, fmt=fmt)[..., :d], randn(g, B, 1, d, fmt=fmt)
    do = randn(g, B, 1, d, std=0.02, fmt=fmt)
    lens = torch.tensor([b % 3 for b in range(B)], dtype=torch.int32, device="cuda")  # 2: clamped to 1
    for kl in (None, lens):
        live = torch.ones(B, dtype=torch.bool, device="cuda") if kl is None else kl > 0
        out, lse = run_forward(q, k, v, H, hd, fmt, kl)
        grads = run_backward(q, k, v, out, do, lse, H, hd, fmt, kl)
        assert torch.equal(out[live], v[live]) and torch.equal(grads[..., 2 * d:][live], do[live])
        ref, tol = R.attention_grad_bounds(*(R.heads(t, H) for t in (q, k, v, v, do)),
                                           (R.heads(q, H) * R.heads(k, H)).sum(-1) / 8, fmt)
        for i, name in enumerate(("dq", "dk")):
            within(R.heads(grads[..., i * d:(i + 1) * d], H)[live], ref[i][live], tol[i][live], name)
        assert not out[~live].any() and not lse[~live].any() and not grads[~live].any()


@FMTS
@pytest.mark.parametrize("lens", [False, True], ids=["full", "padded"])
def test_qk_gradient_of_elements_of_one_token(lens, fmt):
    """Fewer tokens an element than CTAs: a step of the walk skips hundreds of elements."""
    B = 1800
    qk_backward_case(B, 1, 0, 0, 4, 64, fmt, 251, lens=[b % 2 for b in range(B)] if lens else None)
