"""Calls of the training pass that the header allows and the other tests do not make (needs a B200)."""
import pytest
import torch

from joint_attention_block_b200 import ops
from test_gpu_train import _clean_errors, gen, nan_like, randn, ws  # noqa: F401

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
