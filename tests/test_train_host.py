"""The training calls on the host: refusals before any device work, workspace sizes, the binding's checks."""
import ctypes

import pytest
import torch

from joint_attention_block_b200 import _abi, build, synth

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
WS = 1 << 16  # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.lib()


@pytest.fixture(scope="module")
def cfg():
    return _abi.make_config(synth.TINY)


def lse_call(lib, q=1024, ldq=128, k=2048, ldk=128, v=4096, ldv=128, out=8192, lse=16384, fmt=0, batch=1, seq=8,
             heads=2, hd=64, lens=None, ws=None, ws_bytes=0):
    return lib.dit_joint_attention_lse(q, ldq, k, ldk, v, ldv, out, lse, fmt, batch, seq, heads, hd, lens, ws, ws_bytes,
                                       None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(lse=None), INVALID), (dict(q=1032), INVALID), (dict(ldq=120), INVALID),
    (dict(ldk=132), INVALID), (dict(fmt=2), INVALID), (dict(batch=0), INVALID), (dict(seq=0), INVALID),
    (dict(heads=0), INVALID), (dict(hd=96), UNSUPPORTED), (dict(out=1024), INVALID), (dict(out=4096), INVALID),
    (dict(lens=512), WORKSPACE), (dict(lens=512, ws=WS, ws_bytes=100), WORKSPACE),
    (dict(lens=512, ws=WS + 16, ws_bytes=1 << 30), WORKSPACE), (dict(batch=70000), INVALID),
    (dict(seq=1 << 28), INVALID), (dict(ldv=1 << 33), INVALID), (dict(seq=1 << 20, ldk=1 << 20), UNSUPPORTED),
])
def test_attention_forward_refusals(lib, change, status):
    assert lse_call(lib, **change) == status


def backward_call(lib, **c):
    a = dict(q=1024, ldq=128, k=2048, ldk=128, v=4096, ldv=128, out=8192, dout=12288, lse=16384, dq=20480, lddq=128,
             dk=24576, lddk=128, dv=28672, lddv=128, fmt=0, batch=1, seq=8, heads=2, hd=64, lens=None, ws=WS,
             ws_bytes=1 << 30)
    a.update(c)
    return lib.dit_joint_attention_backward(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(dout=None), INVALID), (dict(dv=None), INVALID), (dict(lse=None), INVALID), (dict(lddq=64), INVALID),
    (dict(lddv=130), INVALID), (dict(dk=24584), INVALID), (dict(dq=1024), INVALID), (dict(dv=12288), INVALID),
    (dict(dk=20480), INVALID), (dict(hd=32), UNSUPPORTED), (dict(fmt=2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(ws_bytes=255), WORKSPACE), (dict(ws=WS + 128), WORKSPACE), (dict(seq=-1), INVALID),
    (dict(seq=1 << 20, lddk=1 << 20), UNSUPPORTED),
])
def test_attention_backward_refusals(lib, change, status):
    assert backward_call(lib, **change) == status


def test_qk_refusals(lib, cfg):
    c = ctypes.byref(cfg)
    bad = _abi.make_config(synth.TINY)
    bad.rope_sections[0] = 9

    def out(qkv=1024, qk=4096, fmt=0, batch=1, pos=None, lens=None, config=c, gq=16):
        return lib.dit_qknorm_mrope_out(qkv, qk, fmt, batch, 16, 8, 8, -1, pos, lens, None, config, gq, 32, None)

    assert out(qkv=None) == out(qk=1024) == out(qk=4100) == out(fmt=2) == out(batch=0) == out(gq=None) == INVALID
    assert out(pos=64, lens=64) == INVALID and out(config=ctypes.byref(bad)) == INVALID

    def back(dqk=4096, ld=512, dx=8192, ldx=512, dgq=64, dgk=128, ws=WS, n=1 << 20, pos=None, lens=None):
        return lib.dit_qknorm_mrope_backward(1024, dqk, ld, dx, ldx, dgq, dgk, 0, 1, 16, 8, 8, -1, pos, lens, c, 16, 32,
                                             ws, n, None)

    assert back(dqk=None) == back(ld=511) == back(ld=504) == back(dx=1024) == back(dgq=None) == back(dgk=64) == INVALID
    assert back(dx=4096, ldx=768) == INVALID  # in place with another stride
    assert back(pos=64, lens=64) == INVALID
    assert back(ws=None) == back(n=100) == back(ws=WS + 32) == WORKSPACE
    assert lib.dit_qknorm_mrope_backward_workspace_bytes(ctypes.byref(bad), 1, 80) == 0
    assert lib.dit_qknorm_mrope_backward_workspace_bytes(c, 1, 80) % 256 == 0


def test_rmsnorm_backward_refusals(lib):
    def call(x=1024, xf=0, g=2048, dy=4096, yf=0, dres=None, dx=8192, of=0, dg=12288, rows=4, cols=64, ws=WS, n=1 << 20):
        return lib.dit_rmsnorm_rows_backward(x, xf, g, dy, yf, dres, dx, of, dg, rows, cols, 1e-6, ws, n, None)

    assert call(x=None) == call(xf=1) == call(yf=3) == call(of=-1) == call(cols=12) == call(rows=-1) == INVALID
    assert call(dx=1024) == call(dx=4096) == call(dy=4104) == call(dg=None) == call(dres=8200) == INVALID
    assert call(cols=8200) == UNSUPPORTED
    assert call(ws=None) == call(n=16) == WORKSPACE
    assert lib.dit_rmsnorm_rows_backward_workspace_bytes(4, 12) == 0


def test_misaligned_arrays_are_refused(lib, cfg):
    """A float or int32 array off its 4 bytes would fault in the kernel."""
    assert lse_call(lib, lse=16386) == lse_call(lib, lens=513, ws=WS, ws_bytes=1 << 30) == INVALID
    assert backward_call(lib, lse=16385) == backward_call(lib, lens=514) == INVALID
    c = ctypes.byref(cfg)

    def out(pos=None, lens=None, counts=None):
        return lib.dit_qknorm_mrope_out(1024, 4096, 0, 1, 16, 8, 8, -1, pos, lens, counts, c, 16, 32, None)

    def back(dgq=64, dgk=1024, pos=None, lens=None):
        return lib.dit_qknorm_mrope_backward(1024, 4096, 512, 8192, 512, dgq, dgk, 0, 1, 16, 8, 8, -1, pos, lens, c, 16, 32,
                                             WS, 1 << 20, None)

    assert out(pos=66) == out(lens=66) == out(counts=65) == INVALID
    assert back(dgq=66) == back(dgk=1025) == back(pos=66) == back(lens=67) == INVALID


def test_counts_are_not_written_over_the_lengths(lib, cfg):
    """key_lens inside text_lens would be written by one CTA while the others read it."""
    def call(lens, counts, batch=2):
        return lib.dit_qknorm_mrope_out(1024, 4096, 0, batch, 16, 8, 8, -1, None, lens, counts, ctypes.byref(cfg), 16, 32,
                                        None)

    assert call(512, 512) == call(512, 516) == call(516, 512) == call(512, 524, batch=4) == INVALID


def test_rmsnorm_backward_takes_any_slice_of_a_gradient_buffer(lib):
    """dg is written a float at a time: 4-byte alignment is enough (the workspace is what is refused here)."""
    def call(dg):
        return lib.dit_rmsnorm_rows_backward(1024, 0, 2048, 4096, 0, None, 8192, 0, dg, 4, 64, 1e-6, None, 0, None)

    assert call(12288) == call(12292) == call(12296) == call(12300) == WORKSPACE
    assert call(12290) == call(12289) == INVALID


def test_workspace_sizes(lib):
    # one zero-padded block of 128 rows per element
    assert lib.dit_joint_attention_lse_workspace_bytes(2, 1000, 4, 64) == 2 * 128 * 4 * 64 * 2
    assert lib.dit_joint_attention_lse_workspace_bytes(1, 1000, 4, 96) == 0
    assert lib.dit_joint_attention_backward_workspace_bytes(0, 1000, 4, 64) == 0
    small, large = (lib.dit_joint_attention_backward_workspace_bytes(1, s, 32, 128) for s in (4608, 16896))
    assert 0 < small < large < 64 << 20


def test_binding_checks_types_shapes_strides_and_devices(cfg):
    B, S, H, hd = 2, 10, 4, 64
    d = H * hd
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    q, out, lse = t(B, S, d), t(B, S, d), t(B, H, S, dt=torch.float32)
    call = lambda *a, **k: _abi.joint_attention_lse(*a, H, hd, stream=0, **k)
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(q, q, q, out, lse)
    with pytest.raises(ValueError, match="dtype"):
        call(q.float(), q, q, out, lse)
    with pytest.raises(ValueError, match="dtype"):
        call(q.half(), q, q, out, lse)
    with pytest.raises(ValueError, match="shape"):
        call(q, q[:, :9], q, out, lse)
    with pytest.raises(ValueError, match="shape"):
        call(q, q, q, out, t(B, S, H, dt=torch.float32))
    with pytest.raises(ValueError, match="strides"):
        call(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, out, lse)
    with pytest.raises(ValueError, match="strides"):
        call(t(B, 2 * S, d)[:, :S], q, q, out, lse)
    with pytest.raises(ValueError, match="dtype"):
        call(q, q, q, out, lse, key_lens=t(B, dt=torch.int64))
    with pytest.raises(ValueError, match="16-bit"):
        call(q, q, q, out, lse, fmt=2)
    g = [t(hd), t(hd)]
    with pytest.raises(ValueError, match="shape"):
        _abi.qknorm_mrope_out(t(1, 80, 3 * d), t(1, 80, 3 * d), cfg, 16, 8, 8, *g, stream=0)
    with pytest.raises(ValueError, match="text_lens"):
        _abi.qknorm_mrope_out(t(1, 80, 3 * d), t(1, 80, 2 * d), cfg, 16, 8, 8, *g, stream=0,
                              text_lens=torch.zeros(2, dtype=torch.int32))
    x = t(4, 64)
    with pytest.raises(ValueError, match="dx has dtype"):
        _abi.rmsnorm_rows_backward(x, t(64), x, x, t(64, dt=torch.float32), 1e-6, x, dx_fmt=2, stream=0)


def test_unknown_formats_are_value_errors(cfg):
    x, f = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(ValueError, match="unknown fmt 7"):
        _abi.rmsnorm_rows_backward(x, x[0], x, x, f, 1e-6, x, x_fmt=7, stream=0)
    with pytest.raises(ValueError, match="unknown fmt -1"):
        _abi.qknorm_mrope_out(x, x, cfg, 16, 8, 8, x, x, fmt=-1, stream=0)


def test_single_row_views_have_a_leading_dimension():
    """The stride of a length-one dimension is arbitrary; the binding takes the one that addresses something."""
    d = 128
    one = torch.zeros(1, 1, 3 * d, dtype=torch.bfloat16)[..., d:2 * d]
    assert _abi._rows("q", one, 1, 1, d, 0) == (one.data_ptr(), d)
    batch = torch.zeros(3, 1, 2 * d, dtype=torch.bfloat16)[..., :d]
    assert _abi._rows("q", batch, 3, 1, d, 0) == (batch.data_ptr(), 2 * d)
