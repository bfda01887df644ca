"""Calls at the edges of what the embedding and the block norms allow, as far as the host
answers them: no GPU needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    from mixture_experts_ffn_04_gb300 import build
    build.build()
    m.lib()
    return m


def norm_shape(m, **kw):
    s = m.MoEBlockNormShape()
    s.tokens, s.hidden, s.dtype, s.residual_scale, s.eps = 64, 256, m.MOE_BF16, 1.0, 1e-6
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def test_norms_of_no_tokens(m):
    """Arrays of no tokens have no address; a gate for each of them is one."""
    f, b = m.lib().moe_block_norm_forward, m.lib().moe_block_norm_backward
    s = norm_shape(m, tokens=0, gate=m.MOE_GATE_TOKEN)
    n = m.moe_block_norm_workspace_bytes(s)
    assert n > 0
    assert f(ctypes.byref(s), None, None, 16, None, 16, None, None, None, None) == m.MOE_OK, m.moe_last_error()
    # nothing but gradients of no tokens
    assert b(ctypes.byref(s), None, None, None, None, 16, None, 16, None, None, None, None, None, None, 256, n,
             None) == m.MOE_OK, m.moe_last_error()
    plain = norm_shape(m, tokens=0)
    assert b(ctypes.byref(plain), None, None, None, None, None, None, None, None, None, None, None, None, None, 256, n,
             None) == m.MOE_OK, m.moe_last_error()
    # a gate for each channel has its addresses all the same, and so has one for each of some tokens
    for kw in (dict(tokens=0, gate=m.MOE_GATE_CHANNEL), dict(gate=m.MOE_GATE_TOKEN)):
        s = norm_shape(m, **kw)
        assert f(ctypes.byref(s), 16, 16, 16, None, 16, 16, 16, 16, None) == m.MOE_ERR_INVALID_ARG
        assert "gate" in m.moe_last_error()
    s = norm_shape(m)
    assert b(ctypes.byref(s), 16, 16, 16, 16, 16, None, 16, 16, None, None, None, None, None, 256, 1 << 40,
             None) == m.MOE_ERR_INVALID_ARG
    assert "no gradient" in m.moe_last_error()


def test_a_refused_table_leaves_the_shape_as_it_was(m, monkeypatch):
    """The row stride of a table belongs to its call: the calls after a refused one, and the
    gradient, which reads no table, go on."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(m, "_device", lambda t: -1)     # host tensors
    s = m.MoEEmbedShape()
    s.tokens, s.hidden, s.vocab, s.dtype, s.padding_idx, s.scale = 6, 16, 10, m.MOE_F32, -1, 1.0
    n = m.moe_embed_workspace_bytes(s)
    ids, y, ws = torch.zeros(6, dtype=torch.int32), torch.zeros(6, 16), torch.zeros(n, dtype=torch.uint8)
    with pytest.raises(m.MoEError, match="w_stride"):
        m.moe_embed_forward(s, torch.zeros(10, 20)[:, :16], ids, y, ws, stream=0)
    assert s.w_stride == 0 and m.moe_embed_workspace_bytes(s) == n
    with pytest.raises(ValueError, match="ids"):
        m.moe_embed_forward(s, torch.zeros(10, 24)[:, :16], ids[:5], y, ws, stream=0)
    assert s.w_stride == 0


def test_rows_past_31_bits_of_bytes_are_refused(m):
    """A lookup of rows of 2 GiB counted their pieces in 32 bits."""
    for dtype in (m.MOE_F32, m.MOE_BF16):
        s = m.MoEEmbedShape()
        s.tokens, s.vocab, s.dtype, s.padding_idx, s.scale = 1, 1, dtype, -1, 1.0
        s.hidden = 1 << 28
        assert m.moe_embed_workspace_bytes(s) > 0
        s.hidden = (1 << 28) + 8
        assert m.moe_embed_workspace_bytes(s) == 0 and "hidden" in m.moe_last_error()
        for call in (m.lib().moe_embed_forward, m.lib().moe_embed_backward):
            a = (16, 16, 16) if call is m.lib().moe_embed_forward else (16, 16, None, 16)
            assert call(ctypes.byref(s), *a, 256, 1 << 60, None) == m.MOE_ERR_INVALID_ARG


def test_too_much_gradient_is_refused_before_anything_runs(m):
    """2^32 pieces of sums: refused with the shape, not after the sort has been launched."""
    s = m.MoEEmbedShape()
    s.tokens, s.hidden, s.vocab, s.dtype, s.padding_idx, s.scale = 1 << 28, 1 << 20, 10, m.MOE_BF16, -1, 1.0
    assert m.moe_embed_workspace_bytes(s) == 0 and "tokens times hidden" in m.moe_last_error()
    st = m.lib().moe_embed_backward(ctypes.byref(s), 16, 16, None, 16, 256, 1 << 62, None)
    assert st == m.MOE_ERR_UNSUPPORTED and "tokens times hidden" in m.moe_last_error()
    s.hidden = 1 << 18
    assert m.moe_embed_workspace_bytes(s) > 0
