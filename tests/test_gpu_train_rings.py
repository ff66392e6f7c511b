"""The gradient kernels' rings and item lists walked many times over: several tokens per CTA and several long
items per CTA pair, so that slots are reused, barrier phases wrap and sums run on (needs a B200)."""
import pytest
import torch

import train_ref as R
from joint_attention_block_b200 import ops
from test_gpu_train import FMTS, _clean_errors, qk_backward_case, qkv_case  # noqa: F401
from train_ref import nan_like, run_backward, run_forward, within, ws

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


@FMTS
@pytest.mark.parametrize("S,H,hd", [(520, 4, 128), (520, 4, 64), (90, 3, 64)])
def test_attention_gradients_in_a_row_in_one_workspace(S, H, hd, fmt):
    """Inputs, lengths and workspace written and read by call after call without a pause: every call sees what its
    own inputs' kernels and its own preparation wrote, so it equals the same call by itself in a fresh workspace."""
    B, calls, d = 3, 10, H * hd
    w = ws(ops.joint_attention_backward_workspace_bytes(B, S, H, hd))
    cases, refs = [], []
    for i in range(calls):
        q, k, v, do = (t.contiguous() for t in qkv_case(B, S, H, hd, fmt, 400 + i, do_std=10.0 ** (i % 3 - 2)))
        lens = torch.tensor([(131 * (i + b) + 17 * b) % (S + 1) for b in range(B)], dtype=torch.int32, device="cuda")
        out, lse = run_forward(q, k, v, H, hd, fmt, lens)
        cases.append((q, k, v, out, do, lse, lens))
        refs.append(run_backward(q, k, v, out, do, lse, H, hd, fmt, lens))
    bufs = [torch.empty_like(t) for t in cases[0]]
    got = [nan_like(B, S, 3 * d, fmt=fmt) for _ in range(calls)]
    torch.cuda.synchronize()
    for case, g in zip(cases, got):
        for dst, src in zip(bufs, case):
            dst.copy_(src)
        q, k, v, out, do, lse, lens = bufs
        ops.joint_attention_backward(q, k, v, out, do, lse, g[..., :d], g[..., d:2 * d], g[..., 2 * d:], H, hd, w,
                                     key_lens=lens, fmt=fmt)
    torch.cuda.synchronize()
    for i, (g, ref) in enumerate(zip(got, refs)):
        assert torch.equal(g, ref), i


@FMTS
@pytest.mark.parametrize("padded", [False, True], ids=["full", "padded"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_gradient_of_many_long_items(hd, padded, fmt):
    """Nearly three items of two tiles and four to six blocks for each of the 74 CTA pairs and pass, so that rings and
    accumulators run on from item to item; heads and elements of very different size, so that one item's scale of
    dS (f16) is wrong for the next; in the padded batch the last items of a pair are only zeroed."""
    B, S, H = 26, 420, 4
    d = H * hd
    q, k, v, do = (R.heads(t, H).clone() for t in qkv_case(B, S, H, hd, fmt, 500 + hd))
    size = torch.arange(B * H, device="cuda").view(B, H, 1, 1)
    v = v * 2.0 ** ((size * 5) % 11 - 5)
    do = do * 2.0 ** ((size * 7) % 17 - 8)
    q, k, v, do = (R.flat(t).to(R.DT[fmt]) for t in (q, k, v, do))
    lens = [(0, 420, 257, 416, 400, 1, 385)[b % 7] for b in range(B)] if padded else [S] * B
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda") if padded else None
    out, lse = run_forward(q, k, v, H, hd, fmt, kl)
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt, kl)
    for b, n in enumerate(lens):
        assert not g[b, n:].any()
        if n == 0:
            continue
        q1, k1, v1, o1, do1 = (t[b:b + 1, :n] for t in (q, k, v, out, do))
        ref, ref_lse, tol, tol_lse = R.attention_bounds(*(R.heads(t, H) for t in (q1, k1, v1)), fmt)
        within(R.heads(o1, H), ref, tol, f"out of element {b}")
        within(lse[b:b + 1, :, :n], ref_lse, tol_lse, f"lse of element {b}")
        refs, tols = R.attention_grad_bounds(*(R.heads(t, H) for t in (q1, k1, v1, o1, do1)),
                                             lse[b:b + 1, :, :n].double(), fmt)
        for i, name in enumerate(("dq", "dk", "dv")):
            within(R.heads(g[b:b + 1, :n, i * d:(i + 1) * d], H), refs[i], tols[i], f"{name} of element {b}")
