"""One training step through the attention sublayer as a user would run it, against 64-bit autograd:
x1 = x + Attn(MRoPE(RMSNorm(q)), MRoPE(RMSNorm(k)), v) W_o^T with q, k, v = RMSNorm(x) W_qkv^T, frozen
e4m3 weights, gradients of x and of the three gains (needs a B200)."""
import pytest
import torch

import oracle
import train_ref as R
from joint_attention_block_b200 import ops, synth
from test_gpu_train import config, gains, gen, nan_like, randn, ws

pytestmark = pytest.mark.gpu

H, HD, SEC, THETA, EPS = 4, 64, (8, 12, 12), 10000.0, 1e-6
D = H * HD


def weights(seed, rows, cols):
    w = synth.normal(11, seed, (rows, cols), std=0.04)
    codes, scale = synth.quantize_rows_e4m3(w)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda(), torch.from_numpy(
        oracle.dequant(codes, scale)).double().cuda()


def exact(x, g1, gq, gk, wqkv, wo, lens, n_text, gh, gw, B, S):
    h = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * g1
    q, k, v = (h @ wqkv.T).view(B, S, 3, H, HD).unbind(2)
    out = []
    for b in range(B):
        n = lens[b] + gh * gw
        ang = R.angles(R.positions(lens[b], gh, gw, -1, S, "cuda")[None, :n], SEC, THETA, HD)
        rq, rk = R.qk_forward(q[b:b + 1, :n], gq, ang, EPS), R.qk_forward(k[b:b + 1, :n], gk, ang, EPS)
        o = R.attention(rq.transpose(1, 2), rk.transpose(1, 2), v[b:b + 1, :n].transpose(1, 2))[0]
        out.append(torch.cat([R.flat(o), torch.zeros(1, S - n, D, dtype=torch.float64, device="cuda")], 1))
    return x + torch.cat(out) @ wo.T


@pytest.mark.parametrize("padded", [False, True], ids=["full", "padded"])
def test_training_step_of_the_attention_sublayer(padded):
    B, n_text, gh, gw = 2, 40, 9, 13
    S = n_text + gh * gw
    lens = [40, 11] if padded else [40, 40]
    g = gen(131)
    x, dx1 = randn(g, B, S, D, fmt=0), randn(g, B, S, D, std=0.1)
    for b, n in enumerate(lens):
        dx1[b, n + gh * gw:] = 0  # the loss does not see padding
    (wq8, sq, wqkv), (wo8, so, wo) = weights(1, 3 * D, D), weights(2, D, D)
    cfg, (gq, gk) = config(H, HD), gains(7, HD)
    g1 = (1 + 0.05 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    tl = torch.tensor(lens, dtype=torch.int32, device="cuda") if padded else None
    kl = torch.empty(B, dtype=torch.int32, device="cuda") if padded else None

    # forward: what the step keeps is x, qkv, qk, o, lse
    M = B * S
    h, qkv, qk = nan_like(M, D, fmt=1), nan_like(B, S, 3 * D, fmt=1), nan_like(B, S, 2 * D, fmt=1)
    o, lse, x1 = nan_like(B, S, D, fmt=1), nan_like(B, H, S, fmt=2), nan_like(M, D, fmt=2)
    ops.rmsnorm_rows(x, g1, h, EPS, x_fmt=0, y_fmt=1)
    ops.gemm_w8a16(h, wq8, sq, qkv.view(M, 3 * D), a_fmt=1, y_fmt=1)
    ops.qknorm_mrope_out(qkv, qk, cfg, n_text, gh, gw, gq, gk, text_lens=tl, key_lens=kl, fmt=1)
    ops.joint_attention_lse(qk[..., :D], qk[..., D:], qkv[..., 2 * D:], o, lse, H, HD,
                            ws(ops.joint_attention_lse_workspace_bytes(B, S, H, HD)), key_lens=kl, fmt=1)
    ops.gemm_w8a16(o.view(M, D), wo8, so, x1, residual=x.view(M, D), a_fmt=1, y_fmt=2, res_fmt=0)

    # backward; the frozen products' gradients are the same GEMM on the transposed codes, the scales on the
    # incoming side
    one = torch.ones(D, device="cuda")
    do, dh = nan_like(M, D, fmt=1), nan_like(M, D, fmt=1)
    ops.gemm_w8a16((dx1.view(M, D) * so).half(), wo8.t().contiguous(), one, do, a_fmt=1, y_fmt=1)
    dqkv = nan_like(B, S, 3 * D, fmt=1)
    ops.joint_attention_backward(qk[..., :D], qk[..., D:], qkv[..., 2 * D:], o, do.view(B, S, D), lse, dqkv[..., :D],
                                 dqkv[..., D:2 * D], dqkv[..., 2 * D:], H, HD,
                                 ws(ops.joint_attention_backward_workspace_bytes(B, S, H, HD)), key_lens=kl, fmt=1)
    dgq, dgk, dg1 = nan_like(HD, fmt=2), nan_like(HD, fmt=2), nan_like(D, fmt=2)
    ops.qknorm_mrope_backward(qkv, dqkv[..., :2 * D], dqkv[..., :2 * D], cfg, n_text, gh, gw, gq, gk, dgq, dgk,
                              ws(ops.qknorm_mrope_backward_workspace_bytes(cfg, B, S)), text_lens=tl, fmt=1)
    ops.gemm_w8a16((dqkv.view(M, 3 * D) * sq).half(), wq8.t().contiguous(), one, dh, a_fmt=1, y_fmt=1)
    dx = nan_like(M, D, fmt=2)
    ops.rmsnorm_rows_backward(x.view(M, D), g1, dh, dx, dg1, EPS, ws(ops.rmsnorm_rows_backward_workspace_bytes(M, D)),
                              dres=dx1.view(M, D), x_fmt=0, dy_fmt=1, dx_fmt=2)

    leaves = [t.double().requires_grad_(True) for t in (x, g1, gq, gk)]
    y = exact(*leaves, wqkv, wo, lens, n_text, gh, gw, B, S)
    y.backward(dx1.double())
    # f16 roundings on the way: h, qkv, qk, P, o forward; dx1 s, do, P, dS, dq dk dv, their norm gradient, dqkv s,
    # dh backward: 13 of at most 2^-11 of what they round, each allowed to double on its way through
    tol = 26 * 2.0 ** -11
    live = torch.zeros(B, S, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        live[b, :n + gh * gw] = True
    rel = lambda a, r: ((a.double() - r).norm() / r.norm()).item()
    got = x1.view(B, S, D)[live]
    assert rel(got, y.detach()[live]) <= 10 * 2.0 ** -11
    sub = lambda t: t.view(B, S, D)[live] - dx1[live]  # without the residual's share
    assert rel(sub(dx), sub(leaves[0].grad)) <= tol
    for mine, leaf, name in ((dg1, leaves[1], "g1"), (dgq, leaves[2], "g_q"), (dgk, leaves[3], "g_k")):
        assert rel(mine, leaf.grad) <= tol, name
    if padded:
        assert not dqkv[~live].any() and not (dx.view(B, S, D)[~live]).any()
