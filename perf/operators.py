"""The operators of a training step through the joint-attention sublayer: cases, inputs, plain forms.

Each case is one pass through one operator, either through its plain form (elementary torch
operations) or, with ``own`` set, through the library's entry points:

  qk_forward    per-head QK-RMSNorm + 3D M-RoPE, written beside the raw q and k that the gradient
                needs (``ops.qknorm_mrope_out``)
  qk_backward   its gradient, with the sums of the two gains' gradients (``ops.qknorm_mrope_backward``)
  attn_forward  joint attention that also returns the log-sum-exp of every row
                (``ops.joint_attention_lse``)
  attn_backward its gradient, the probabilities recomputed (``ops.joint_attention_backward``)
  norm_backward the pre-norm's gradient with the gain's, the residual's gradient added
                (``ops.rmsnorm_rows_backward``)
"""
import math

import numpy as np
import torch

own = False

THETA = 10000.0
EPS = 1e-6
SECTIONS = {64: (8, 12, 12), 128: (24, 20, 20)}  # rotary pairs on the (t, h, w) axes
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases


def _attn(name, op, n_text, gh, gw, heads, hd, fmt, batch=1, lens=""):
    return {"name": name, "op": op, "batch": batch, "n_text": n_text, "grid_h": gh, "grid_w": gw, "heads": heads,
            "head_dim": hd, "fmt": fmt, "lens": lens}


def listed():
    return [
        # the smallest model of the tests, one prompt: every call is latency
        _attn("attn_forward tiny", "attn_forward", 16, 8, 8, 4, 64, "bf16"),
        # one 1024 px image with its prompt, in the block's own activation format
        _attn("attn_forward 1024px", "attn_forward", 512, 64, 64, 32, 128, "f16"),
        _attn("attn_backward tiny", "attn_backward", 16, 8, 8, 4, 64, "bf16"),
        # prompts of different lengths in one padded batch of a smaller image with odd sides
        _attn("attn_backward padded", "attn_backward", 512, 31, 33, 16, 64, "bf16", batch=4, lens="512,77,301,0"),
        # the training step's own size: one 1024 px image, fp16 with small gradients
        _attn("attn_backward 1024px", "attn_backward", 512, 64, 64, 32, 128, "f16"),
        # one 2048 px image, the longest sequence of the configurations
        _attn("attn_backward 2048px", "attn_backward", 512, 128, 128, 32, 128, "bf16"),
        _attn("qk_forward tiny", "qk_forward", 16, 8, 8, 4, 64, "f16"),
        # two prompts padded to one length at 1024 px
        _attn("qk_forward 1024px padded", "qk_forward", 512, 64, 64, 32, 128, "bf16", batch=2, lens="512,131"),
        _attn("qk_backward tiny", "qk_backward", 16, 8, 8, 4, 64, "bf16"),
        _attn("qk_backward 1024px", "qk_backward", 512, 64, 64, 32, 128, "f16"),
        # the first pre-norm of the smallest model
        {"name": "norm_backward tiny", "op": "norm_backward", "rows": 80, "cols": 256, "x": "bf16", "dy": "bf16",
         "dx": "bf16", "residual": True},
        # the second pre-norm at 1024 px: the fp32 residual stream in, its gradient out
        {"name": "norm_backward 1024px", "op": "norm_backward", "rows": 4608, "cols": 4096, "x": "f32", "dy": "f16",
         "dx": "f32", "residual": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["attn_forward", "attn_backward", "attn_backward", "qk_forward", "qk_backward", "norm_backward"])
    if op == "norm_backward":
        cols = 8 * _log_int(rng, 8, 1024)
        rows = _log_int(rng, 1, min(20000, (16896 * 4096) // cols))
        return {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["bf16", "f32"]),
                "dy": rng.choice(["bf16", "f16", "f32"]), "dx": rng.choice(["bf16", "f32"]),
                "residual": rng.random() < 0.7}
    hd = rng.choice([64, 128])
    heads = (256 // hd) * rng.choice([1, 2, 4, 8, 12, 16])
    batch = rng.choice([1, 1, 2, 3])
    while True:
        gh, gw = _log_int(rng, 1, 110), _log_int(rng, 1, 110)
        n_text = rng.choice([0, 1, _log_int(rng, 2, 700), _log_int(rng, 2, 700)])
        seq = n_text + gh * gw
        # never dearer than the longest listed sequence
        if batch * seq * seq * heads * hd <= 16896 ** 2 * 4096 and batch * seq * heads * hd <= 16896 * 4096:
            break
    lens = ""
    if n_text > 0 and rng.random() < 0.5:
        lens = ",".join(str(rng.randint(0, n_text)) for _ in range(batch))
    return {"op": op, "batch": batch, "n_text": n_text, "grid_h": gh, "grid_w": gw, "heads": heads, "head_dim": hd,
            "fmt": rng.choice(["bf16", "f16"]), "lens": lens}


def _lens(case):
    return [int(v) for v in case["lens"].split(",")] if case["lens"] else None


def _seq(case):
    return case["n_text"] + case["grid_h"] * case["grid_w"]


def _counts(case):
    """Tokens of each batch element that take part."""
    n_img = case["grid_h"] * case["grid_w"]
    lens = _lens(case)
    return [_seq(case)] * case["batch"] if lens is None else [n + n_img for n in lens]


# ---------------------------------------------------------------- inputs


def _randn(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    if case["op"] == "norm_backward":
        rows, cols = case["rows"], case["cols"]
        st = {"case": case,
              "x": (_randn(gen, rows, cols) * 1.5).to(DTYPES[case["x"]]),
              "g": (1.0 + _randn(gen, cols, std=0.05)).to(torch.bfloat16),
              "dy": _randn(gen, rows, cols, std=0.02).to(DTYPES[case["dy"]]),
              "dres": _randn(gen, rows, cols, std=0.02).to(DTYPES[case["dx"]]) if case["residual"] else None}
        st["dx"] = torch.empty(rows, cols, dtype=DTYPES[case["dx"]], device="cuda")
        st["dg"] = torch.empty(cols, dtype=torch.float32, device="cuda")
        if own:
            from joint_attention_block_b200 import ops
            st["ws"] = torch.empty(ops.rmsnorm_rows_backward_workspace_bytes(rows, cols), dtype=torch.uint8,
                                   device="cuda")
        return st

    B, S, H, hd = case["batch"], _seq(case), case["heads"], case["head_dim"]
    d, dt = H * hd, DTYPES[case["fmt"]]
    lens = _lens(case)
    st = {"case": case,
          # the fused projection's output: q, k and v as the block's product of unit rows gives them
          "qkv": _randn(gen, B, S, 3 * d, std=1.28).to(dt),
          "g_q": (1.0 + _randn(gen, hd, std=0.05)).to(torch.bfloat16),
          "g_k": (1.0 + _randn(gen, hd, std=0.05)).to(torch.bfloat16),
          "text_lens": None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"),
          "key_lens": None if lens is None else torch.tensor(_counts(case), dtype=torch.int32, device="cuda")}
    if case["op"] == "qk_forward":
        st["qk"] = torch.empty(B, S, 2 * d, dtype=dt, device="cuda")
        if lens is not None:
            st["counts"] = torch.empty(B, dtype=torch.int32, device="cuda")
    elif case["op"] == "qk_backward":
        dqk = _randn(gen, B, S, 2 * d, std=0.02)
        for b, n in enumerate(_counts(case)):
            dqk[b, n:] = 0  # what the attention's gradient holds behind each element's tokens
        st["dqk"] = dqk.to(dt)
        st["dx"] = torch.empty(B, S, 2 * d, dtype=dt, device="cuda")
        st["dg"] = torch.empty(2, hd, dtype=torch.float32, device="cuda")
    else:
        # normalised, gained q and k (a rotation leaves their distribution as it is)
        qk = st["qkv"][..., :2 * d].float().view(B, S, 2, H, hd)
        qk = qk * torch.rsqrt(qk.square().mean(-1, keepdim=True) + EPS)
        qk = qk * torch.stack([st["g_q"], st["g_k"]]).float()[:, None, :]
        st["qk"] = qk.reshape(B, S, 2 * d).to(dt)
        del qk
        st["out"] = torch.empty(B, S, d, dtype=dt, device="cuda")
        st["lse"] = torch.empty(B, H, S, dtype=torch.float32, device="cuda")
        if case["op"] == "attn_backward":
            out, lse = _plain_attn_forward(st)  # what the forward pass left behind
            st["out"], st["lse"] = out, lse
            st["dout"] = _randn(gen, B, S, d, std=0.02).to(dt)
            st["dqkv"] = torch.empty(B, S, 3 * d, dtype=dt, device="cuda")
    if own:
        from joint_attention_block_b200 import ops
        cfg = ops.BlockConfig()
        cfg.d_model, cfg.n_heads, cfg.head_dim, cfg.d_mlp = d, H, hd, 4 * d
        for i in range(3):
            cfg.rope_sections[i] = SECTIONS[hd][i]
        cfg.rope_theta, cfg.eps, cfg.gelu_tanh = THETA, EPS, 0
        st["cfg"] = cfg
        n = {"qk_forward": 256,
             "qk_backward": ops.qknorm_mrope_backward_workspace_bytes(cfg, B, S),
             "attn_forward": ops.joint_attention_lse_workspace_bytes(B, S, H, hd),
             "attn_backward": ops.joint_attention_backward_workspace_bytes(B, S, H, hd)}[case["op"]]
        st["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- one pass


def run(state):
    return {"qk_forward": _qk_forward, "qk_backward": _qk_backward, "attn_forward": _attn_forward,
            "attn_backward": _attn_backward, "norm_backward": _norm_backward}[state["case"]["op"]](state)


def _fmt(state):
    return {"bf16": 0, "f16": 1}[state["case"]["fmt"]]


def _split(state):
    """q, k (the rotated ones) and v as the calls take them: [B, S, d] views of the two buffers."""
    d = state["case"]["heads"] * state["case"]["head_dim"]
    return state["qk"][..., :d], state["qk"][..., d:], state["qkv"][..., 2 * d:]


def _qk_forward(st):
    c = st["case"]
    if own:
        from joint_attention_block_b200 import ops
        ops.qknorm_mrope_out(st["qkv"], st["qk"], st["cfg"], c["n_text"], c["grid_h"], c["grid_w"], st["g_q"],
                             st["g_k"], text_lens=st["text_lens"], key_lens=st.get("counts"), fmt=_fmt(st))
        return (st["qk"], st["counts"]) if c["lens"] else st["qk"]
    B, S, H, hd = c["batch"], _seq(c), c["heads"], c["head_dim"]
    x = st["qkv"][..., :2 * H * hd].float().view(B, S, 2, H, hd)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * torch.stack([st["g_q"], st["g_k"]]).float()[:, None, :]
    cos, sin = _plain_angles(c)
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    y = y.reshape(B, S, 2 * H * hd).to(st["qkv"].dtype)
    return (y, st["text_lens"] + c["grid_h"] * c["grid_w"]) if c["lens"] else y


def _qk_backward(st):
    c = st["case"]
    if own:
        from joint_attention_block_b200 import ops
        ops.qknorm_mrope_backward(st["qkv"], st["dqk"], st["dx"], st["cfg"], c["n_text"], c["grid_h"], c["grid_w"],
                                  st["g_q"], st["g_k"], st["dg"][0], st["dg"][1], st["ws"],
                                  text_lens=st["text_lens"], fmt=_fmt(st))
        return st["dx"], st["dg"]
    B, S, H, hd = c["batch"], _seq(c), c["heads"], c["head_dim"]
    d = H * hd
    x = st["qkv"][..., :2 * d].float().view(B, S, 2, H, hd)
    dy = st["dqk"].float().view(B, S, 2, H, hd)
    g = torch.stack([st["g_q"], st["g_k"]]).float()[:, None, :]
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    cos, sin = _plain_angles(c)
    a, b = dy[..., :hd // 2], dy[..., hd // 2:]
    dz = torch.cat([a * cos + b * sin, b * cos - a * sin], -1)
    dg = (dz * xh).sum((0, 1, 3), dtype=torch.float64).float()
    du = dz * g
    dx = r * (du - xh * (du * xh).mean(-1, keepdim=True))
    return dx.reshape(B, S, 2 * d).to(st["qkv"].dtype), dg


def _attn_forward(st):
    c = st["case"]
    if own:
        from joint_attention_block_b200 import ops
        q, k, v = _split(st)
        ops.joint_attention_lse(q, k, v, st["out"], st["lse"], c["heads"], c["head_dim"], st["ws"],
                                key_lens=st["key_lens"], fmt=_fmt(st))
        return st["out"], st["lse"]
    return _plain_attn_forward(st)


def _attn_backward(st):
    c = st["case"]
    H, hd = c["heads"], c["head_dim"]
    d = H * hd
    q, k, v = _split(st)
    if own:
        from joint_attention_block_b200 import ops
        g = st["dqkv"]
        ops.joint_attention_backward(q, k, v, st["out"], st["dout"], st["lse"], g[..., :d], g[..., d:2 * d],
                                     g[..., 2 * d:], H, hd, st["ws"], key_lens=st["key_lens"], fmt=_fmt(st))
        return st["dqkv"]
    res = torch.zeros_like(st["dqkv"])
    scale = 1.0 / math.sqrt(hd)
    for b, n in enumerate(_counts(c)):
        for h in range(H):
            s = slice(h * hd, (h + 1) * hd)
            qh, kh, vh, doh, oh = (t[b, :n, s].float() for t in (q, k, v, st["dout"], st["out"]))
            p = torch.exp((qh @ kh.T) * scale - st["lse"][b, h, :n, None])
            dp = doh @ vh.T
            ds = p * (dp - (doh * oh).sum(-1, keepdim=True)) * scale
            res[b, :n, h * hd:(h + 1) * hd] = ds @ kh
            res[b, :n, d + h * hd:d + (h + 1) * hd] = ds.T @ qh
            res[b, :n, 2 * d + h * hd:2 * d + (h + 1) * hd] = p.T @ doh
    return res


def _norm_backward(st):
    if own:
        from joint_attention_block_b200 import ops
        code = {"bf16": 0, "f16": 1, "f32": 2}
        c = st["case"]
        ops.rmsnorm_rows_backward(st["x"], st["g"], st["dy"], st["dx"], st["dg"], EPS, st["ws"], dres=st["dres"],
                                  x_fmt=code[c["x"]], dy_fmt=code[c["dy"]], dx_fmt=code[c["dx"]])
        return st["dx"], st["dg"]
    x, dy = st["x"].float(), st["dy"].float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    dg = (dy * xh).sum(0, dtype=torch.float64).float()
    du = dy * st["g"].float()
    dx = r * (du - xh * (du * xh).mean(-1, keepdim=True))
    if st["dres"] is not None:
        dx = dx + st["dres"].float()
    return dx.to(DTYPES[st["case"]["dx"]]), dg


def _plain_attn_forward(st):
    c = st["case"]
    B, S, H, hd = c["batch"], _seq(c), c["heads"], c["head_dim"]
    q, k, v = _split(st)
    out = torch.zeros(B, S, H * hd, dtype=st["qkv"].dtype, device="cuda")
    lse = torch.zeros(B, H, S, dtype=torch.float32, device="cuda")
    for b, n in enumerate(_counts(c)):
        for h in range(H):
            s = slice(h * hd, (h + 1) * hd)
            x = (q[b, :n, s].float() @ k[b, :n, s].float().T) / math.sqrt(hd)
            m = x.amax(-1, keepdim=True)
            p = torch.exp(x - m)
            z = p.sum(-1, keepdim=True)
            out[b, :n, s] = (p @ v[b, :n, s].float()) / z
            lse[b, h, :n] = (m + torch.log(z))[:, 0]
    return out, lse


def _plain_angles(c):
    """cos, sin fp32 [B or 1, S, 1, 1, hd/2]; the angles of far positions in 64 bits."""
    S, hd, n_img = _seq(c), c["head_dim"], c["grid_h"] * c["grid_w"]
    lens = _lens(c)
    i = torch.arange(S, device="cuda")
    pos = []
    for n in [c["n_text"]] if lens is None else lens:
        img = (i >= n) & (i < n + n_img)
        text = torch.where(i < n, i, torch.zeros_like(i))
        j = i - n
        pos.append(torch.stack([torch.where(img, torch.full_like(i, n), text), torch.where(img, j // c["grid_w"], text),
                                torch.where(img, j % c["grid_w"], text)]))
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(SECTIONS[hd], device="cuda"))
    pos = torch.stack(pos)[:, axis].transpose(1, 2).double()  # [B or 1, S, hd/2]
    freq = (THETA ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)).float().double()
    ang = (pos * freq)[:, :, None, None, :]
    return ang.cos().float(), ang.sin().float()


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] == "norm_backward":
        n = case["rows"] * case["cols"]
        per = size[case["x"]] + size[case["dy"]] + size[case["dx"]] * (2 if case["residual"] else 1)
        return {"bytes": n * per + case["cols"] * 6, "flops": n * 11}
    H, hd = case["heads"], case["head_dim"]
    d = H * hd
    rows, counts = case["batch"] * _seq(case), _counts(case)
    live, pairs = sum(counts), sum(n * n for n in counts)
    if case["op"] == "qk_forward":
        return {"bytes": (rows + rows) * 2 * d * 2 + 4 * hd, "flops": rows * 2 * d * 8}
    if case["op"] == "qk_backward":
        return {"bytes": (2 * live + rows) * 2 * d * 2 + 12 * hd, "flops": live * 2 * d * 16}
    if case["op"] == "attn_forward":
        return {"bytes": (3 * live + rows) * d * 2 + rows * H * 4, "flops": 4 * pairs * d}
    return {"bytes": (5 * live + 3 * rows) * d * 2 + live * H * 4, "flops": 10 * pairs * d}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_backward":
        x, g, dy = (st[k].double() for k in ("x", "g", "dy"))
        n = x.shape[1]
        m = (x * x).sum(1) / n + EPS
        # y_i = x_i m^(-1/2) g_i, so dx_j = g_j dy_j m^(-1/2) - x_j m^(-3/2) / n sum_i x_i g_i dy_i
        dot = torch.einsum("ri,i,ri->r", x, g, dy)
        dx = dy * g / m.sqrt()[:, None] - x * (dot / (n * m ** 1.5))[:, None]
        if st["dres"] is not None:
            dx += st["dres"].double()
        return dx, torch.einsum("ri,ri,r->i", dy, x, 1 / m.sqrt())

    B, S, H, hd = case["batch"], _seq(case), case["heads"], case["head_dim"]
    d = H * hd
    if case["op"] in ("qk_forward", "qk_backward"):
        # pair i of a head as the complex number a + ib; the rotation is a product with exp(i angle)
        rot = _exact_rotation(case)
        out = torch.zeros(B, S, 2 * d, dtype=torch.float64, device="cuda")
        dg = torch.zeros(2, hd, dtype=torch.float64, device="cuda")
        for b in range(B):
            for w, g in enumerate((st["g_q"].double(), st["g_k"].double())):
                x = st["qkv"][b, :, w * d:(w + 1) * d].double().reshape(S, H, hd)
                m = torch.einsum("shi,shi->sh", x, x) / hd + EPS
                if case["op"] == "qk_forward":
                    u = x * g / m.sqrt()[..., None]
                    z = torch.complex(u[..., :hd // 2], u[..., hd // 2:]) * rot[b][:, None, :]
                    out[b, :, w * d:(w + 1) * d] = torch.cat([z.real, z.imag], -1).reshape(S, d)
                else:
                    dy = st["dqk"][b, :, w * d:(w + 1) * d].double().reshape(S, H, hd)
                    z = torch.complex(dy[..., :hd // 2], dy[..., hd // 2:]) * rot[b].conj()[:, None, :]
                    dz = torch.cat([z.real, z.imag], -1)
                    dot = torch.einsum("shi,i,shi->sh", dz, g, x)
                    dx = dz * g / m.sqrt()[..., None] - x * (dot / (hd * m ** 1.5))[..., None]
                    out[b, :, w * d:(w + 1) * d] = dx.reshape(S, d)
                    dg[w] += torch.einsum("shi,shi,sh->i", dz, x, 1 / m.sqrt())
        if case["op"] == "qk_backward":
            return out, dg
        return (out, torch.tensor(_counts(case))) if case["lens"] else out

    q, k, v = (t.double().view(B, S, H, hd) for t in _split(st))
    if case["op"] == "attn_forward":
        out = torch.zeros(B, S, H, hd, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, H, S, dtype=torch.float64, device="cuda")
    else:
        do = st["dout"].double().view(B, S, H, hd)
        grad = torch.zeros(B, S, 3, H, hd, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_counts(case)):
        for h in range(H):
            x = torch.einsum("qi,ki->qk", q[b, :n, h], k[b, :n, h]).mul_(hd ** -0.5)
            z = torch.logsumexp(x, 1)
            p = x.sub_(z[:, None]).exp_()
            if case["op"] == "attn_forward":
                out[b, :n, h], lse[b, h, :n] = p @ v[b, :n, h], z
                continue
            grad[b, :n, 2, h] = p.T @ do[b, :n, h]
            dp = do[b, :n, h] @ v[b, :n, h].T
            mean = torch.einsum("qk,qk->q", p, dp)  # the softmax's own mean of dp
            ds = dp.sub_(mean[:, None]).mul_(p).mul_(hd ** -0.5)
            grad[b, :n, 0, h] = ds @ k[b, :n, h]
            grad[b, :n, 1, h] = ds.T @ q[b, :n, h]
    if case["op"] == "attn_forward":
        return out.view(B, S, d), lse
    return grad.view(B, S, 3 * d)


def _exact_rotation(case):
    """exp(i angle), complex128 [S, hd/2] for each batch element, from the positions written out token by token."""
    S, hd = _seq(case), case["head_dim"]
    freq = np.array([np.float32(THETA ** (-2.0 * i / hd)) for i in range(hd // 2)], dtype=np.float64)
    lens = _lens(case)
    res = []
    for n in [case["n_text"]] * case["batch"] if lens is None else lens:
        pos = np.zeros((S, 3))
        for s in range(S):
            if s < n:
                pos[s] = s
            elif s < n + case["grid_h"] * case["grid_w"]:
                pos[s] = (n, (s - n) // case["grid_w"], (s - n) % case["grid_w"])
        cols = np.concatenate([np.repeat(pos[:, a:a + 1], SECTIONS[hd][a], axis=1) for a in range(3)], axis=1)
        res.append(torch.from_numpy(np.exp(1j * cols * freq)).cuda())
    return res
