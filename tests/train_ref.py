"""Plain 64-bit formulas of the attention sublayer's training pass, and how far a kernel that rounds to
16 bits at the documented places may be from them, element by element (first-order bounds).

u is half a step of the 16-bit format (bf16 2^-8, fp16 2^-11).  For each product the bound carries the
rounding of the 16-bit operand (P or dS), the relative error eta of a recomputed probability, the fp32
accumulation and the rounding of the result."""
import math

import torch

from joint_attention_block_b200 import ops

DT = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}
U = {0: 2.0 ** -8, 1: 2.0 ** -11, 2: 2.0 ** -24}
TINY = {0: 2.0 ** -134, 1: 2.0 ** -25, 2: 2.0 ** -150}  # half a subnormal step


def heads(t, H):
    """[B, S, H hd] -> [B, H, S, hd] in fp64."""
    B, S, d = t.shape
    return t.double().view(B, S, H, d // H).transpose(1, 2)


def flat(t):
    B, H, S, hd = t.shape
    return t.transpose(1, 2).reshape(B, S, H * hd)


def logit_error(q, k):
    """Absolute error of a scaled logit: an fp32 dot product of hd exact products, one fp32 multiply-add and
    exp2's own error (a few 2^-23 of the exponent and of the value)."""
    hd = q.shape[-1]
    big = (q.abs() @ k.abs().mT).amax().item() / math.sqrt(hd)
    return (hd + 16) * 2.0 ** -24 * big + 2.0 ** -20


def attention(q, k, v):
    x = (q @ k.mT) / math.sqrt(q.shape[-1])
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    return p @ v, lse, p


def attention_bounds(q, k, v, fmt):
    """Reference out, lse and their bounds (P is rounded, the row sum is not)."""
    out, lse, p = attention(q, k, v)
    eta, u = logit_error(q, k), U[fmt]
    acc = (q.shape[-2] / 8 + 16) * 2.0 ** -23
    floor = TINY[fmt] * 2 ** 8 if fmt == 1 else 0.0  # f16 P below its normal range, relative to the row maximum's 1
    tol = u * out.abs() + (u + 2 * eta + acc) * (p @ v.abs()) + floor * v.abs().sum(-2, keepdim=True) + TINY[fmt]
    return out, lse, tol, 2 * eta + 2.0 ** -20 * (1 + lse.abs())


def attention_grad_bounds(q, k, v, out, do, lse, fmt):
    """dq, dk, dv of the formula on the given out and lse, and their bounds."""
    hd, n, u = q.shape[-1], q.shape[-2], U[fmt]
    scale = 1 / math.sqrt(hd)
    p = torch.exp((q @ k.mT) * scale - lse[..., None])
    dp = do @ v.mT
    delta = (do * out).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    eta = logit_error(q, k) + 2.0 ** -22 * (1 + lse.abs().amax().item())
    acc = (n / 8 + 16) * 2.0 ** -23
    e_dp = (hd + 8) * 2.0 ** -24 * (do.abs() @ v.abs().mT + (do * out).abs().sum(-1, keepdim=True))
    e_ds = (u + 2 * eta + acc) * ds.abs() + p * e_dp
    e_p = (u + 2 * eta + acc) * p
    if fmt == 1:  # half a subnormal step of the scaled value: P by 2^15, dS so that 2 A B lies above 2^13
        ab = 2 * do.norm(dim=-1).amax((-1,), keepdim=True)[..., None] * v.norm(dim=-1).amax((-1,), keepdim=True)[..., None]
        e_p = e_p + 2.0 ** -40
        e_ds = e_ds + 2.0 ** -25 * ab * 2.0 ** -13
    # below 2^-126 fp32 and bf16 values may be flushed to zero: at most 2^-126 off in each P, which enters
    # dS times |dP - delta|, in each dS, and in each of the n products of a sum
    low = 2.0 ** -126
    e_p = e_p + low
    e_ds = e_ds + low * (1 + (dp - delta).abs())
    g = [ds @ k * scale, ds.mT @ q * scale, p.mT @ do]
    tol = [e_ds @ k.abs() * scale, e_ds.mT @ q.abs() * scale, e_p.mT @ do.abs()]
    return g, [t + u * x.abs() + TINY[fmt] + n * low for t, x in zip(tol, g)]


def angles(pos, sections, theta, hd):
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor(list(sections))).to(pos.device)
    f = (theta ** (-2.0 * torch.arange(hd // 2, dtype=torch.float64, device=pos.device) / hd)).float().double()
    return pos.double()[..., axis] * f  # [..., S, hd/2]


def positions(n_text, gh, gw, t_img, seq, device):
    """(t, h, w) of the first n_text + gh gw rows, zeros behind them."""
    p = torch.zeros(seq, 3, dtype=torch.int64)
    p[:n_text] = torch.arange(n_text)[:, None]
    c = torch.arange(gh * gw)
    p[n_text:n_text + gh * gw] = torch.stack([torch.full_like(c, n_text if t_img < 0 else t_img), c // max(gw, 1),
                                              c % max(gw, 1)], -1)
    return p.to(device)


def qk_forward(x, g, ang, eps):
    """x [B, S, H, hd] fp64, ang [B, S, hd/2]."""
    u = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * g
    a, b = u.chunk(2, -1)
    cs, sn = ang.cos()[:, :, None], ang.sin()[:, :, None]
    return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)


def qk_backward(x, g, ang, eps, dy):
    hd = x.shape[-1]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    cs, sn = ang.cos()[:, :, None], ang.sin()[:, :, None]
    a, b = dy.chunk(2, -1)
    dz = torch.cat([a * cs + b * sn, b * cs - a * sn], -1)
    az = torch.cat([(a * cs).abs() + (b * sn).abs(), (b * cs).abs() + (a * sn).abs()], -1)  # sizes entering dz
    xh, du = x * r, dz * g
    dx = r * (du - xh * (du * xh).mean(-1, keepdim=True))
    size = r * (az * g.abs() + xh.abs() * (az * g.abs() * xh.abs()).mean(-1, keepdim=True))
    return dx, (dz * xh), size, az * xh.abs()


def rms_backward(x, g, dy, eps):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    xh, du = x * r, dy * g
    dx = r * (du - xh * (du * xh).mean(-1, keepdim=True))
    size = r * (du.abs() + xh.abs() * (du * xh).abs().mean(-1, keepdim=True))
    return dx, dy * xh, size


def ws(nbytes):
    """Scratch full of NaN patterns."""
    return torch.full((max(int(nbytes), 256),), 0xFF, dtype=torch.uint8, device="cuda")


def nan_like(*shape, fmt):
    return torch.full(shape, float("nan"), dtype=DT[fmt], device="cuda")


def within(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    over = (got - ref).abs() - tol
    worst = ((got - ref).abs() / tol.clamp_min(1e-300)).amax().item() if got.numel() else 0.0
    assert (over <= 0).all(), f"{what}: {worst:.3g} times the bound, at {int((over > 0).sum())} of {over.numel()}"
    return worst


def run_forward(q, k, v, H, hd, fmt, key_lens=None):
    B, S = q.shape[:2]
    out = nan_like(B, S, H * hd, fmt=fmt)
    lse = nan_like(B, H, S, fmt=2)
    w = ws(ops.joint_attention_lse_workspace_bytes(B, S, H, hd)) if key_lens is not None else None
    ops.joint_attention_lse(q, k, v, out, lse, H, hd, w, key_lens=key_lens, fmt=fmt)
    return out, lse


def run_backward(q, k, v, out, do, lse, H, hd, fmt, key_lens=None, stream=None):
    B, S = q.shape[:2]
    d = H * hd
    g = nan_like(B, S, 3 * d, fmt=fmt)
    w = ws(ops.joint_attention_backward_workspace_bytes(B, S, H, hd))
    ops.joint_attention_backward(q, k, v, out, do, lse, g[..., :d], g[..., d:2 * d], g[..., 2 * d:], H, hd, w,
                                 key_lens=key_lens, fmt=fmt, stream=stream)
    return g
