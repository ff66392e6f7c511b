"""The gradient kernels' rings and item lists walked many times over: several tokens per CTA and several long
items per CTA pair, so that slots are reused, barrier phases wrap and sums run on (needs a B200)."""
import pytest
import torch

import train_ref as R
from joint_attention_block_b200 import ops
from test_gpu_train import FMTS, _clean_errors, qk_backward_case  # noqa: F401

pytestmark = pytest.mark.gpu


# At most 444 CTAs take the tokens of q (and as many those of k) at 16 threads a token, 222 at 128, 148 at 256
# and 74 above; a CTA's ring has at most eight slots.  So every CTA here reuses each slot, and with fewer rows
# per element than CTAs it steps over whole elements.
@FMTS
@pytest.mark.parametrize("padded", [False, True], ids=["full", "padded"])
@pytest.mark.parametrize("B,H,hd", [(64, 4, 64), (40, 16, 128), (24, 32, 128), (10, 36, 128), (10, 64, 128)])
def test_qk_backward_of_many_tokens_per_cta(B, H, hd, padded, fmt):
    n_text, gh, gw = 40, 5, 15
    lens = [(17 * b) % (n_text + 1) for b in range(B)] if padded else None
    qk_backward_case(B, n_text, gh, gw, H, hd, fmt, 107 + B, lens=lens)
