"""The training pass of the attention sublayer against its 64-bit formulas (needs a B200)."""
import math

import pytest
import torch

import train_ref as R
from joint_attention_block_b200 import ops, synth
from train_ref import DT, U, nan_like, run_backward, run_forward, within, ws

pytestmark = pytest.mark.gpu
FMTS = pytest.mark.parametrize("fmt", [0, 1], ids=["bf16", "f16"])


@pytest.fixture(autouse=True)
def _clean_errors():
    yield
    st = ops.poll_error()
    assert st == 0, f"a kernel recorded a device-side error: status {st}, word {ops.last_device_error():#x}"


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, fmt=2):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DT[fmt])


def qkv_case(B, S, H, hd, fmt, seed, do_std=0.02):
    g = gen(seed)
    qk, qkv = randn(g, B, S, 2 * H * hd, fmt=fmt), randn(g, B, S, 3 * H * hd, fmt=fmt)
    d = H * hd
    return qk[..., :d], qk[..., d:], qkv[..., 2 * d:], randn(g, B, S, d, std=do_std, fmt=fmt)


# one token; one key block, short, exact and one over; ragged; more query tiles than one CTA pair's
SHAPES = [(1, 1, 1, 64), (2, 80, 4, 64), (1, 127, 2, 128), (1, 128, 2, 128), (2, 129, 1, 64), (1, 300, 2, 128),
          (1, 641, 3, 64), (1, 1100, 1, 128), (200, 48, 2, 128)]


@FMTS
@pytest.mark.parametrize("B,S,H,hd", SHAPES)
def test_attention_forward(B, S, H, hd, fmt):
    q, k, v, _ = qkv_case(B, S, H, hd, fmt, 100 + S)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    ref, ref_lse, tol, tol_lse = R.attention_bounds(R.heads(q, H), R.heads(k, H), R.heads(v, H), fmt)
    within(R.heads(out, H), ref, tol, "out")
    within(lse, ref_lse, tol_lse, "lse")


@FMTS
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_forward_equals_the_inference_call(hd, fmt):
    B, S, H = 2, 333, 3
    g = gen(5)
    qkv = randn(g, B, S, 3 * H * hd, fmt=fmt)
    d = H * hd
    ref = torch.empty(B, S, d, dtype=DT[fmt], device="cuda")
    ops.joint_attention(qkv, ref, H, hd, fmt=fmt)
    out, _ = run_forward(qkv[..., :d], qkv[..., d:2 * d], qkv[..., 2 * d:], H, hd, fmt)
    assert torch.equal(out, ref)


@FMTS
@pytest.mark.parametrize("B,S,H,hd", SHAPES)
def test_attention_backward(B, S, H, hd, fmt):
    q, k, v, do = qkv_case(B, S, H, hd, fmt, 200 + S)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt)
    ref, tol = R.attention_grad_bounds(*(R.heads(t, H) for t in (q, k, v, out, do)), lse.double(), fmt)
    for i, name in enumerate(("dq", "dk", "dv")):
        within(R.heads(g[..., i * H * hd:(i + 1) * H * hd], H), ref[i], tol[i], name)


@FMTS
@pytest.mark.parametrize("std", [1e-5, 1e-3, 30.0])
def test_attention_backward_of_small_and_large_gradients(std, fmt):
    """dO far below and above 1: f16's dS would vanish or overflow without its scale.  (dO of 1e-5 is
    subnormal in f16 itself; the reference takes the rounded values.)"""
    B, S, H, hd = 1, 700, 2, 128
    q, k, v, do = qkv_case(B, S, H, hd, fmt, 31, do_std=std)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt)
    ref, tol = R.attention_grad_bounds(*(R.heads(t, H) for t in (q, k, v, out, do)), lse.double(), fmt)
    for i, name in enumerate(("dq", "dk", "dv")):
        within(R.heads(g[..., i * H * hd:(i + 1) * H * hd], H), ref[i], tol[i], name)


@FMTS
def test_attention_of_zero_gradients_and_peaked_rows(fmt):
    """dO = 0 gives exact zeros; one dominating key per row (P = 1 there, 0 elsewhere) stays finite."""
    B, S, H, hd = 1, 260, 1, 64
    q, k, v, do = qkv_case(B, S, H, hd, fmt, 37)
    q, k = q * 12, k * 12
    out, lse = run_forward(q, k, v, H, hd, fmt)
    assert not run_backward(q, k, v, out, torch.zeros_like(do), lse, H, hd, fmt).any()
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt)
    ref, tol = R.attention_grad_bounds(*(R.heads(t, H) for t in (q, k, v, out, do)), lse.double(), fmt)
    for i, name in enumerate(("dq", "dk", "dv")):
        within(R.heads(g[..., i * hd:(i + 1) * hd], H), ref[i], tol[i], name)


LENS = [(300, [300, 0, 1, 127, 128, 129, 255, 256, 299]), (128, [128, 5, 0]), (1200, [1200, 513, 512, 1])]


@FMTS
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("S,lens", LENS, ids=["S300", "S128", "S1200"])
def test_attention_padded(S, lens, hd, fmt):
    """Rows behind an element's count hold NaN and infinities and change nothing; they come out as zeros,
    and every element equals itself run alone at its own length."""
    B, H = len(lens), 2
    d = H * hd
    q, k, v, do = (t.clone() for t in qkv_case(B, S, H, hd, fmt, 300 + S))
    for b, n in enumerate(lens):
        for i, t in enumerate((q, k, v, do)):
            t[b, n:] = (float("nan"), float("inf"), -float("inf"), float("nan"))[i]
            t[b, n + 1::2] = float("nan")
    kl = torch.tensor([n if n < S else n + 7 for n in lens], dtype=torch.int32, device="cuda")  # clamped to S
    out, lse = run_forward(q, k, v, H, hd, fmt, kl)
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt, kl)
    for b, n in enumerate(lens):
        assert not out[b, n:].any() and not lse[b, :, n:].any() and not g[b, n:].any()
        if n == 0:
            continue
        q1, k1, v1, do1, o1 = (t[b:b + 1, :n] for t in (q, k, v, do, out))
        ref, ref_lse, tol, tol_lse = R.attention_bounds(*(R.heads(t, H) for t in (q1, k1, v1)), fmt)
        within(R.heads(o1, H), ref, tol, f"out, {n} of {S}")
        within(lse[b:b + 1, :, :n], ref_lse, tol_lse, f"lse, {n} of {S}")
        refs, tols = R.attention_grad_bounds(*(R.heads(t, H) for t in (q1, k1, v1, o1, do1)),
                                             lse[b:b + 1, :, :n].double(), fmt)
        for i, name in enumerate(("dq", "dk", "dv")):
            within(R.heads(g[b:b + 1, :n, i * d:(i + 1) * d], H), refs[i], tols[i], f"{name}, {n} of {S}")


@pytest.mark.parametrize("S", [300, 250], ids=["two_tiles", "one_tile"])
@pytest.mark.parametrize("which", ["mixed", "gap", "none"])
def test_attention_gradient_of_many_elements(which, S):
    """More elements than a warp has lanes, with runs that hold no tokens: each equals itself run alone."""
    B, H, hd, fmt = 101, 3, 64, 0
    d = H * hd
    lens = [(37 * b) % (S + 1) for b in range(B)]
    if which == "gap":  # nothing in elements 20 to 79, only single tokens at the end
        lens = [0 if 20 <= b < 80 else 1 if b >= 95 else n for b, n in enumerate(lens)]
    elif which == "none":
        lens = [0] * (B - 1) + [S]
    q, k, v, do = qkv_case(B, S, H, hd, fmt, 53)
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = run_forward(q, k, v, H, hd, fmt, kl)
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt, kl)
    for b, n in enumerate(lens):
        assert not g[b, n:].any()
        if n == 0:
            continue
        q1, k1, v1, o1, do1 = (t[b:b + 1, :n] for t in (q, k, v, out, do))
        refs, tols = R.attention_grad_bounds(*(R.heads(t, H) for t in (q1, k1, v1, o1, do1)),
                                             lse[b:b + 1, :, :n].double(), fmt)
        for i, name in enumerate(("dq", "dk", "dv")):
            within(R.heads(g[b:b + 1, :n, i * d:(i + 1) * d], H), refs[i], tols[i], f"{name}, element {b}")


def test_attention_negative_counts_are_no_tokens():
    q, k, v, do = qkv_case(2, 70, 1, 64, 0, 41)
    kl = torch.tensor([-3, 70], dtype=torch.int32, device="cuda")
    out, lse = run_forward(q, k, v, 1, 64, 0, kl)
    g = run_backward(q, k, v, out, do, lse, 1, 64, 0, kl)
    assert not out[0].any() and not lse[0].any() and not g[0].any() and g[1].any()


def test_attention_views_leave_their_neighbours_alone():
    """Views into wider buffers, each with its own row stride: only the named columns are written."""
    B, S, H, hd, fmt = 2, 150, 2, 64, 0
    d = H * hd
    g = gen(43)
    wide = [randn(g, B, S, w, fmt=fmt) for w in (d + 8, 3 * d + 16, 2 * d)]
    q, k, v = wide[0][..., 8:], wide[1][..., 16:16 + d], wide[2][..., :d]
    do = randn(g, B, S, d, std=0.02, fmt=fmt)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    base = run_backward(q.contiguous(), k.contiguous(), v.contiguous(), out, do, lse, H, hd, fmt)
    bufs = [torch.full((B, S, w), 7.0, dtype=DT[fmt], device="cuda") for w in (d + 24, 2 * d + 8, d + 8)]
    views = [bufs[0][..., 8:8 + d], bufs[1][..., d:2 * d], bufs[2][..., :d]]
    ops.joint_attention_backward(q, k, v, out, do, lse, *views, H, hd,
                                 ws(ops.joint_attention_backward_workspace_bytes(B, S, H, hd)), fmt=fmt)
    for i, (buf, view) in enumerate(zip(bufs, views)):
        assert torch.equal(view, base[..., i * d:(i + 1) * d])
        view.fill_(7.0)
        assert (buf == 7.0).all()


def test_attention_offsets_past_32_bits():
    """Rows 2^19 elements apart: offsets beyond 2^32 elements in q, k, v and the gradients."""
    B, S, H, hd, fmt = 2, 4200, 1, 64, 0
    ld = 1 << 19
    g = gen(47)
    buf = torch.empty(B * S * ld, dtype=DT[fmt], device="cuda").view(B, S, ld)
    q, k, v = buf[..., :hd], buf[..., 1024:1024 + hd], buf[..., ld - hd:]
    for t in (q, k, v):
        t.copy_(randn(g, B, S, hd, fmt=fmt))
    do = randn(g, B, S, hd, std=0.02, fmt=fmt)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    out1, lse1 = run_forward(q.contiguous(), k.contiguous(), v.contiguous(), H, hd, fmt)
    assert torch.equal(out, out1) and torch.equal(lse, lse1)
    ref = run_backward(q.contiguous(), k.contiguous(), v.contiguous(), out, do, lse, H, hd, fmt)
    grads = [buf[..., 4096 * (i + 1):4096 * (i + 1) + hd] for i in range(3)]
    ops.joint_attention_backward(q, k, v, out, do, lse, *grads, H, hd,
                                 ws(ops.joint_attention_backward_workspace_bytes(B, S, H, hd)), fmt=fmt)
    for i in range(3):
        assert torch.equal(grads[i], ref[..., i * hd:(i + 1) * hd])


@FMTS
def test_attention_gradient_against_differences(fmt):
    """<gradient, direction> against central differences of the 64-bit forward along random directions."""
    B, S, H, hd = 1, 200, 2, 64
    q, k, v, do = qkv_case(B, S, H, hd, fmt, 53, do_std=1.0)
    out, lse = run_forward(q, k, v, H, hd, fmt)
    g = run_backward(q, k, v, out, do, lse, H, hd, fmt).double()
    d = H * hd
    x = [R.heads(t, H) for t in (q, k, v)]
    loss = lambda a: (R.attention(*a)[0] * R.heads(do, H)).sum().item()
    h = 1e-4
    for i in range(3):
        # along the gradient itself the derivative is its squared norm: no cancellation hides an error
        w = R.heads(g[..., i * d:(i + 1) * d], H)
        w = w / w.norm()
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + h * w, x[i] - h * w
        diff = (loss(up) - loss(dn)) / (2 * h)
        mine = (R.heads(g[..., i * d:(i + 1) * d], H) * w).sum().item()
        # roundings of P or dS, of out inside delta, and of the result: three of at most u each, in the norm
        assert abs(diff - mine) <= 3 * U[fmt] * abs(mine), (i, diff, mine)


def test_attention_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    B, S, H, hd, fmt = 2, 700, 4, 128, 1
    q, k, v, do = qkv_case(B, S, H, hd, fmt, 59)
    kl = torch.tensor([700, 431], dtype=torch.int32, device="cuda")
    out, lse = run_forward(q, k, v, H, hd, fmt, kl)
    ref = run_backward(q, k, v, out, do, lse, H, hd, fmt, kl)
    for _ in range(3):
        assert torch.equal(run_backward(q, k, v, out, do, lse, H, hd, fmt, kl), ref)
    # two streams at once, each with its own workspace
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    got = [nan_like(B, S, 3 * H * hd, fmt=fmt) for _ in s]
    wss = [ws(ops.joint_attention_backward_workspace_bytes(B, S, H, hd)) for _ in s]
    d = H * hd
    torch.cuda.synchronize()
    for i in range(2):
        ops.joint_attention_backward(q, k, v, out, do, lse, got[i][..., :d], got[i][..., d:2 * d], got[i][..., 2 * d:],
                                     H, hd, wss[i], key_lens=kl, fmt=fmt, stream=s[i])
    torch.cuda.synchronize()
    assert torch.equal(got[0], ref) and torch.equal(got[1], ref)
    # captured once, replayed on other inputs in the same buffers
    w1 = ws(ops.joint_attention_lse_workspace_bytes(B, S, H, hd))
    o2, l2, g2 = torch.empty_like(out), torch.empty_like(lse), nan_like(B, S, 3 * d, fmt=fmt)
    qb, kb, vb, dob = (t.contiguous().clone() for t in (q, k, v, do))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.joint_attention_lse(qb, kb, vb, o2, l2, H, hd, w1, key_lens=kl, fmt=fmt)
        ops.joint_attention_backward(qb, kb, vb, o2, dob, l2, g2[..., :d], g2[..., d:2 * d], g2[..., 2 * d:], H, hd,
                                     wss[0], key_lens=kl, fmt=fmt)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g2, ref)
    q3, k3, v3, do3 = qkv_case(B, S, H, hd, fmt, 61)
    kl.copy_(torch.tensor([3, 650], dtype=torch.int32))
    for dst, src in ((qb, q3), (kb, k3), (vb, v3), (dob, do3)):
        dst.copy_(src)
    graph.replay()
    o3, l3 = run_forward(q3, k3, v3, H, hd, fmt, kl)
    assert torch.equal(o2, o3) and torch.equal(g2, run_backward(q3, k3, v3, o3, do3, l3, H, hd, fmt, kl))


# ---------------------------------------------------------------- QK-norm + M-RoPE


def config(H, hd):
    c = ops.BlockConfig()
    c.d_model, c.n_heads, c.head_dim, c.d_mlp = H * hd, H, hd, 4 * H * hd
    for i, v in enumerate((8, 12, 12) if hd == 64 else (24, 20, 20)):
        c.rope_sections[i] = v
    c.rope_theta, c.eps, c.gelu_tanh = 10000.0, 1e-6, 0
    return c


def gains(seed, hd):
    g = gen(seed)
    return [(1 + 0.05 * torch.randn(hd, generator=g, device="cuda")).bfloat16() for _ in range(2)]


@FMTS
@pytest.mark.parametrize("H,hd", [(4, 64), (2, 128)])
def test_qk_out_equals_the_in_place_call(H, hd, fmt):
    cfg, (gq, gk) = config(H, hd), gains(3, hd)
    d = H * hd
    qkv = randn(gen(67), 2, 37 + 9 * 11, 3 * d, fmt=fmt)
    ref = qkv.clone()
    ops.qknorm_mrope(ref, cfg, 37, 9, 11, gq, gk, ws(256), t_img=5, fmt=fmt)
    raw = qkv.clone()
    qk = nan_like(2, qkv.shape[1], 2 * d, fmt=fmt)
    kl = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    ops.qknorm_mrope_out(qkv, qk, cfg, 37, 9, 11, gq, gk, t_img=5, key_lens=kl, fmt=fmt)
    assert torch.equal(qkv, raw) and torch.equal(qk, ref[..., :2 * d]) and kl.tolist() == [136, 136]


@FMTS
def test_qk_out_padded_equals_each_prompt_alone(fmt):
    H, hd, n_text, gh, gw = 4, 64, 30, 4, 7
    cfg, (gq, gk) = config(H, hd), gains(5, hd)
    d, S = H * hd, n_text + gh * gw
    lens = [30, 0, 1, 17]
    qkv = randn(gen(71), 4, S, 3 * d, fmt=fmt)
    qk = nan_like(4, S, 2 * d, fmt=fmt)
    kl = torch.zeros(4, dtype=torch.int32, device="cuda")
    ops.qknorm_mrope_out(qkv, qk, cfg, n_text, gh, gw, gq, gk, text_lens=torch.tensor(lens, dtype=torch.int32).cuda(),
                         key_lens=kl, fmt=fmt)
    assert kl.tolist() == [n + gh * gw for n in lens]
    for b, n in enumerate(lens):
        m = n + gh * gw
        one = nan_like(1, m, 2 * d, fmt=fmt)
        ops.qknorm_mrope_out(qkv[b:b + 1, :m].contiguous(), one, cfg, n, gh, gw, gq, gk, fmt=fmt)
        assert torch.equal(qk[b:b + 1, :m], one)


def qk_backward_case(B, n_text, gh, gw, H, hd, fmt, seed, lens=None, t_img=-1, pos=None):
    """Runs the call in place in a [B, S, 3d] gradient buffer; returns what within() needs."""
    cfg, (gq, gk) = config(H, hd), gains(seed, hd)
    d, S = H * hd, n_text + gh * gw
    g = gen(seed)
    qkv, dqkv = randn(g, B, S, 3 * d, fmt=fmt), randn(g, B, S, 3 * d, std=0.02, fmt=fmt)
    counts = [S] * B if lens is None else [n + gh * gw for n in lens]
    for b, n in enumerate(counts):
        qkv[b, n:] = float("nan")
        dqkv[b, n:, :2 * d] = float("inf")
    before = dqkv.clone()
    dg = [nan_like(hd, fmt=2) for _ in range(2)]
    tl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    ops.qknorm_mrope_backward(qkv, dqkv[..., :2 * d], dqkv[..., :2 * d], cfg, n_text, gh, gw, gq, gk, *dg,
                              ws(ops.qknorm_mrope_backward_workspace_bytes(cfg, B, S)), t_img=t_img, pos=pos,
                              text_lens=tl, fmt=fmt)
    assert torch.equal(dqkv[..., 2 * d:], before[..., 2 * d:])
    sums, sizes = [0, 0], [0, 0]
    for b, n in enumerate(counts):
        assert not dqkv[b, n:, :2 * d].any()
        p = (pos.long() if pos is not None else
             R.positions(n_text if lens is None else lens[b], gh, gw, t_img, S, "cuda"))[None, :n]
        ang = R.angles(p, cfg.rope_sections, cfg.rope_theta, hd)
        for w, gain in enumerate((gq, gk)):
            x = qkv[b:b + 1, :n, w * d:(w + 1) * d].double().view(1, n, H, hd)
            dy = before[b:b + 1, :n, w * d:(w + 1) * d].double().view(1, n, H, hd)
            dx, term, size, tsize = R.qk_backward(x, gain.double(), ang, cfg.eps, dy)
            # fp32: the angle's sine and cosine, products and a sum of hd terms: (hd / 4 + 32) steps of what enters
            tol = U[fmt] * dx.abs() + (hd / 4 + 32) * 2.0 ** -24 * size + R.TINY[fmt]
            within(dqkv[b:b + 1, :n, w * d:(w + 1) * d].view(1, n, H, hd), dx, tol, f"dx[{w}] of element {b}")
            sums[w] = sums[w] + term.sum((0, 1, 2))
            sizes[w] = sizes[w] + tsize.sum((0, 1, 2))
    for w in range(2):
        # each term within 32 fp32 steps, added in chains of at most rows / CTAs + 64
        chain = B * S / 100 + 96
        within(dg[w], sums[w], chain * 2.0 ** -24 * sizes[w] + 1e-30, f"dg[{w}]")


@FMTS
@pytest.mark.parametrize("B,n_text,gh,gw,H,hd", [(1, 1, 0, 0, 4, 64), (1, 16, 8, 8, 4, 64), (2, 37, 9, 11, 2, 128),
                                                 (1, 0, 3, 5, 12, 64), (1, 500, 20, 20, 32, 128), (1, 5, 4, 4, 64, 128)])
def test_qk_backward(B, n_text, gh, gw, H, hd, fmt):
    qk_backward_case(B, n_text, gh, gw, H, hd, fmt, 73)


@FMTS
def test_qk_backward_padded(fmt):
    qk_backward_case(5, 40, 5, 7, 4, 64, fmt, 79, lens=[40, 0, 1, 17, 39])
    qk_backward_case(3, 40, 0, 0, 2, 128, fmt, 83, lens=[0, 40, 9], t_img=4)


def test_qk_backward_explicit_positions():
    pos = torch.randint(-50, 4000, (90, 3), generator=gen(89), device="cuda", dtype=torch.int32)
    qk_backward_case(2, 10, 8, 10, 2, 128, 0, 89, pos=pos)


def test_qk_backward_against_differences():
    B, n_text, gh, gw, H, hd, fmt = 1, 9, 4, 5, 4, 64, 1
    cfg, (gq, gk) = config(H, hd), gains(97, hd)
    d, S = H * hd, n_text + gh * gw
    g = gen(97)
    qkv, dqk = randn(g, B, S, 3 * d, fmt=fmt), randn(g, B, S, 2 * d, fmt=fmt)
    dx, dg = nan_like(B, S, 2 * d, fmt=fmt), nan_like(2, hd, fmt=2)
    ops.qknorm_mrope_backward(qkv, dqk, dx, cfg, n_text, gh, gw, gq, gk, dg[0], dg[1],
                              ws(ops.qknorm_mrope_backward_workspace_bytes(cfg, B, S)), fmt=fmt)
    ang = R.angles(R.positions(n_text, gh, gw, -1, S, "cuda")[None], cfg.rope_sections, cfg.rope_theta, hd)
    h = 1e-5
    for w, gain in enumerate((gq.double(), gk.double())):
        x = qkv[..., w * d:(w + 1) * d].double().view(B, S, H, hd)
        dy = dqk[..., w * d:(w + 1) * d].double().view(B, S, H, hd)
        loss = lambda a, b: (R.qk_forward(a, b, ang, cfg.eps) * dy).sum().item()
        mine = dx[..., w * d:(w + 1) * d].double().view(B, S, H, hd)
        e = mine / mine.norm()
        diff = (loss(x + h * e, gain) - loss(x - h * e, gain)) / (2 * h)
        assert abs(diff - (mine * e).sum().item()) <= 2 * U[fmt] * abs(diff)
        e = dg[w].double() / dg[w].double().norm()
        diff = (loss(x, gain + h * e) - loss(x, gain - h * e)) / (2 * h)
        assert abs(diff - dg[w].double().norm().item()) <= 1e-5 * abs(diff)


# ---------------------------------------------------------------- RMSNorm rows


@pytest.mark.parametrize("rows,cols", [(1, 8), (80, 256), (5, 264), (3, 4096), (700, 1000), (2, 4104), (601, 8192),
                                       (1500, 512), (2500, 1024), (1190, 776), (5000, 256), (400, 1032)])
@pytest.mark.parametrize("xf,yf,of,res", [(0, 0, 0, True), (0, 1, 0, False), (2, 1, 2, True), (2, 2, 1, True),
                                          (0, 2, 2, False), (2, 0, 0, True)])
def test_rmsnorm_backward(rows, cols, xf, yf, of, res):
    g = gen(rows + cols)
    x, dy = randn(g, rows, cols, std=1.5, fmt=xf), randn(g, rows, cols, std=0.02, fmt=yf)
    gain = (1 + 0.05 * torch.randn(cols, generator=g, device="cuda")).bfloat16()
    dres = randn(g, rows, cols, std=0.02, fmt=of) if res else None
    dx, dg = nan_like(rows, cols, fmt=of), nan_like(cols, fmt=2)
    ops.rmsnorm_rows_backward(x, gain, dy, dx, dg, 1e-6, ws(ops.rmsnorm_rows_backward_workspace_bytes(rows, cols)),
                              dres=dres, x_fmt=xf, dy_fmt=yf, dx_fmt=of)
    ref, term, size = R.rms_backward(x.double(), gain.double(), dy.double(), 1e-6)
    if res:
        ref = ref + dres.double()
        size = size + dres.double().abs()
    # fp32: sums of cols / threads terms per thread, then 5 + 16 partial sums; a handful of products
    within(dx, ref, U[of] * ref.abs() + 64 * 2.0 ** -24 * size + R.TINY[of], "dx")
    chain = rows / 296 + 32 + 64
    within(dg, term.sum(0), chain * 2.0 ** -24 * term.abs().sum(0) + 1e-30, "dg")


def test_rmsnorm_backward_in_the_residual_buffer_and_no_rows():
    g = gen(101)
    x, dy, dres = randn(g, 300, 512, fmt=2), randn(g, 300, 512, fmt=1), randn(g, 300, 512, fmt=2)
    gain = torch.ones(512, device="cuda").bfloat16()
    w = ws(ops.rmsnorm_rows_backward_workspace_bytes(300, 512))
    dx, dg, dg2 = nan_like(300, 512, fmt=2), nan_like(512, fmt=2), nan_like(512, fmt=2)
    ops.rmsnorm_rows_backward(x, gain, dy, dx, dg, 1e-6, w, dres=dres, x_fmt=2, dy_fmt=1, dx_fmt=2)
    ops.rmsnorm_rows_backward(x, gain, dy, dres, dg2, 1e-6, w, dres=dres, x_fmt=2, dy_fmt=1, dx_fmt=2)
    assert torch.equal(dres, dx) and torch.equal(dg, dg2)
    none = torch.empty(0, 512, device="cuda")
    ops.rmsnorm_rows_backward(none, gain, none.half(), none.clone(), dg, 1e-6, w, x_fmt=2, dy_fmt=1, dx_fmt=2)
    assert not dg.any()


def test_rmsnorm_backward_against_differences():
    g = gen(103)
    x, dy = randn(g, 20, 256, fmt=2), randn(g, 20, 256, fmt=2)
    gain = (1 + 0.05 * torch.randn(256, generator=g, device="cuda")).bfloat16()
    dx, dg = nan_like(20, 256, fmt=2), nan_like(256, fmt=2)
    ops.rmsnorm_rows_backward(x, gain, dy, dx, dg, 1e-6, ws(ops.rmsnorm_rows_backward_workspace_bytes(20, 256)),
                              x_fmt=2, dy_fmt=2, dx_fmt=2)
    f = lambda a, b: (a * torch.rsqrt(a.square().mean(-1, keepdim=True) + 1e-6) * b * dy.double()).sum().item()
    h = 1e-5
    for mine, up in ((dx, lambda e: f(x.double() + e, gain.double())), (dg, lambda e: f(x.double(), gain.double() + e))):
        e = mine.double() / mine.double().norm()
        diff = (up(h * e) - up(-h * e)) / (2 * h)
        assert abs(diff - mine.double().norm().item()) <= 1e-5 * abs(diff)


# ---------------------------------------------------------------- both, as a program uses them


def test_elementwise_gradients_on_other_streams_and_in_graphs():
    """Two streams with their own workspaces, then a captured run replayed on other inputs: the same bits."""
    B, n_text, gh, gw, H, hd, fmt = 2, 30, 8, 8, 4, 64, 0
    cfg, (gq, gk), d, S = config(H, hd), gains(5, hd), H * hd, n_text + gh * gw
    g = gen(67)
    tl = torch.tensor([30, 11], dtype=torch.int32, device="cuda")
    gain = torch.ones(d, device="cuda").bfloat16()
    qkv, dqk = randn(g, B, S, 3 * d, fmt=fmt), randn(g, B, S, 2 * d, std=0.02, fmt=fmt)
    x, dy = randn(g, B * S, d, fmt=2), randn(g, B * S, d, std=0.02, fmt=fmt)

    def results():
        return [nan_like(B, S, 2 * d, fmt=fmt), nan_like(B, S, 2 * d, fmt=fmt), nan_like(hd, fmt=2), nan_like(hd, fmt=2),
                nan_like(B * S, d, fmt=2), nan_like(d, fmt=2)]

    def works():
        return (ws(ops.qknorm_mrope_backward_workspace_bytes(cfg, B, S)),
                ws(ops.rmsnorm_rows_backward_workspace_bytes(B * S, d)))

    def run(r, w, stream=None):
        ops.qknorm_mrope_out(qkv, r[0], cfg, n_text, gh, gw, gq, gk, text_lens=tl, fmt=fmt, stream=stream)
        ops.qknorm_mrope_backward(qkv, dqk, r[1], cfg, n_text, gh, gw, gq, gk, r[2], r[3], w[0], text_lens=tl, fmt=fmt,
                                  stream=stream)
        ops.rmsnorm_rows_backward(x, gain, dy, r[4], r[5], 1e-6, w[1], x_fmt=2, dy_fmt=fmt, dx_fmt=2, stream=stream)

    ref = results()
    run(ref, works())
    streams, got, wss = [torch.cuda.Stream() for _ in range(2)], [results() for _ in range(2)], [works() for _ in range(2)]
    torch.cuda.synchronize()
    for s, r, w in zip(streams, got, wss):
        run(r, w, s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, ref))
    graph, mine = torch.cuda.CUDAGraph(), results()
    with torch.cuda.graph(graph):
        run(mine, wss[0])
    qkv.copy_(randn(g, B, S, 3 * d, fmt=fmt))
    x.copy_(randn(g, B * S, d, fmt=2))
    tl.copy_(torch.tensor([0, 29], dtype=torch.int32))
    graph.replay()
    run(ref, wss[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(mine, ref))


def test_elementwise_offsets_past_32_bits():
    """Buffers of more than 2^32 bytes and 2^31 elements: the last tokens and rows equal a short run."""
    H, hd, fmt, n = 64, 128, 0, 512
    cfg, (gq, gk), d = config(H, hd), gains(7, hd), H * hd
    B = (1 << 31) // (3 * d * n) + 1
    g = gen(71)
    qkv = torch.zeros(B, n, 3 * d, dtype=DT[fmt], device="cuda")
    grad = torch.zeros_like(qkv)
    qkv[-1], grad[-1] = randn(g, n, 3 * d, fmt=fmt), randn(g, n, 3 * d, std=0.02, fmt=fmt)
    one, gone, dq1 = qkv[-1:].clone(), grad[-1:].clone(), grad[-1:].clone()
    qk, qk1 = torch.empty(B, n, 2 * d, dtype=DT[fmt], device="cuda"), nan_like(1, n, 2 * d, fmt=fmt)
    ops.qknorm_mrope_out(qkv, qk, cfg, n, 0, 0, gq, gk, fmt=fmt)
    ops.qknorm_mrope_out(one, qk1, cfg, n, 0, 0, gq, gk, fmt=fmt)
    assert torch.equal(qk[-1:], qk1)
    del qk
    dg, dg1 = [nan_like(hd, fmt=2) for _ in range(2)], [nan_like(hd, fmt=2) for _ in range(2)]
    for a, b, c in ((qkv, grad, dg), (one, gone, dg1)):
        ops.qknorm_mrope_backward(a, b[..., :2 * d], b[..., :2 * d], cfg, n, 0, 0, gq, gk, *c,
                                  ws(ops.qknorm_mrope_backward_workspace_bytes(cfg, a.shape[0], n)), fmt=fmt)
    assert torch.equal(grad[-1:], gone)
    # zero gradients before the last element add nothing; each sum is within its chains (as above) of the exact one
    ang = R.angles(R.positions(n, 0, 0, -1, n, "cuda")[None], cfg.rope_sections, cfg.rope_theta, hd)
    for w, gain in enumerate((gq, gk)):
        x, dy = (t[..., w * d:(w + 1) * d].double().view(1, n, H, hd) for t in (one, dq1))
        _, term, _, tsize = R.qk_backward(x, gain.double(), ang, cfg.eps, dy)
        for got in (dg[w], dg1[w]):
            within(got, term.sum((0, 1, 2)), (n / 100 + 96) * 2.0 ** -24 * tsize.sum((0, 1, 2)) + 1e-30, f"dg[{w}]")
    del qkv, grad
    rows, cols = (1 << 31) // 8192 + 9, 8192
    x, dy = torch.zeros(rows, cols, dtype=DT[fmt], device="cuda"), torch.zeros(rows, cols, dtype=DT[fmt], device="cuda")
    x[-5:], dy[-5:] = randn(g, 5, cols, fmt=fmt), randn(g, 5, cols, std=0.02, fmt=fmt)
    gain = torch.ones(cols, device="cuda").bfloat16()
    xs, dys, dx1 = x[-5:].clone(), dy[-5:].clone(), nan_like(5, cols, fmt=fmt)
    dx, dgn = dy.clone(), nan_like(cols, fmt=2)
    ops.rmsnorm_rows_backward(x, gain, dy, dx, dgn, 1e-6, ws(ops.rmsnorm_rows_backward_workspace_bytes(rows, cols)))
    ops.rmsnorm_rows_backward(xs, gain, dys, dx1, dgn.clone(), 1e-6, ws(ops.rmsnorm_rows_backward_workspace_bytes(5, cols)))
    assert torch.equal(dx[-5:], dx1) and not dx[:-5].any()
