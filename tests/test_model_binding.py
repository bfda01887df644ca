"""What the Python binding of the embedding, the block norms and the orthogonalised update
refuses before the library is called: no GPU needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    from mixture_experts_ffn_04_gb300 import build
    build.build()
    m.lib()
    return m


@pytest.fixture
def device0(m, monkeypatch):
    """The checks behind the device check, on host tensors: those are device -1."""
    monkeypatch.setattr(m, "_device", lambda t: -1)


def test_host_memory_is_refused(m):
    t = torch.zeros(4, 64)
    for call in (lambda: m.moe_embed_forward(m.MoEEmbedShape(), t, t, t, t),
                 lambda: m.moe_embed_backward(m.MoEEmbedShape(), t, t, None, t, t),
                 lambda: m.moe_block_norm_forward(m.MoEBlockNormShape(), t, t, None, None, None, t, None, None),
                 lambda: m.moe_block_norm_backward(m.MoEBlockNormShape(), t, t, t, t, None, None, None, t, t, t, None,
                                                   None, None, t),
                 lambda: m.moe_orthogonalize(m.MoEOrthShape(), m.orth_coefs(), t, t, t),
                 lambda: m.moe_muon_step((m.MoEMuonTensor * 1)(), m.MoEMuonConfig(), t)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_another_device_than_the_current_one_is_refused(m, monkeypatch):
    class Elsewhere:
        is_cuda = True
        device = "cuda:1"

        def get_device(self):
            return 1

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        m._device(Elsewhere())


def embed(m, T=6, H=16, V=10):
    s = m.MoEEmbedShape()
    s.tokens, s.hidden, s.vocab, s.dtype, s.padding_idx, s.scale = T, H, V, m.MOE_F32, -1, 1.0
    return s, torch.zeros(V, H), torch.zeros(T, dtype=torch.int32), torch.zeros(T, H), torch.zeros(512, dtype=torch.uint8)


def test_embedding_arguments(m, device0):
    s, w, ids, y, ws = embed(m)
    bad = [(w.expand(10, 16)[:1].expand(10, 16), ids, y, "rows of w"), (w[:9], ids, y, "w must"),
           (w.bfloat16(), ids, y, "w must"), (w, ids.long(), y, "ids must"), (w, ids[:5], y, "ids must"),
           (w, ids, y.bfloat16(), "y must"), (w, ids, torch.zeros(16, 6).t(), "contiguous"), (w, None, y, "ids must"),
           (w, ids, None, "y must")]
    for a, b, c, word in bad:
        with pytest.raises(ValueError, match=word):
            m.moe_embed_forward(s, a, b, c, ws, stream=0)
    for ids_, dy, add, dw, word in ((ids, y, None, None, "dw must"), (ids, y, w[:3], w, "dw_add must"),
                                    (ids, y[:2], None, w, "dy must"), (ids.float(), y, None, w, "ids must"),
                                    (ids, y, None, torch.zeros(10, 32)[:, :16], "contiguous")):
        with pytest.raises(ValueError, match=word):
            m.moe_embed_backward(s, ids_, dy, add, dw, ws, stream=0)


def test_norm_arguments(m, device0):
    s = m.MoEBlockNormShape()
    s.tokens, s.hidden, s.dtype, s.gate, s.residual_scale, s.eps = 6, 16, m.MOE_BF16, m.MOE_GATE_TOKEN, 1.0, 1e-6
    x, v, g = torch.zeros(6, 16).bfloat16(), torch.zeros(16).bfloat16(), torch.zeros(6)
    r, ws = torch.zeros(6, 2), torch.zeros(512, dtype=torch.uint8)
    good = dict(x=x, y=x, w_post=v, gate=g, w_pre=v, s=x, h=x, rstd=r)
    for name, bad in (("x", x.float()), ("x", None), ("y", x[:3]), ("w_post", v.float()), ("gate", v), ("gate", g.double()),
                      ("w_pre", v[:8]), ("s", x.float()), ("h", torch.zeros(16, 6).bfloat16().t()), ("rstd", r[:2])):
        with pytest.raises(ValueError, match=name):
            m.moe_block_norm_forward(s, **{**good, name: bad}, stream=0)
    good = dict(ds=x, dh=x, x=x, y=x, w_post=v, gate=g, w_pre=v, rstd=r, dx=x, dy=x, dw_post=v, dgate=g, dw_pre=v, ws=ws)
    for name, bad in (("ds", x.float()), ("dh", x[:1]), ("x", None), ("rstd", None), ("dx", x.half()), ("dy", x[:1]),
                      ("dw_post", v.float()), ("dgate", v), ("dw_pre", torch.zeros(32).bfloat16()[::2])):
        with pytest.raises(ValueError, match=name):
            m.moe_block_norm_backward(s, **{**good, name: bad}, stream=0)


def test_update_lists(m):
    w = torch.zeros(2, 8, 16)
    with pytest.raises(ValueError, match="one gradient"):
        m.muon_tensors([w], [], [w])
    for g, v in ((w[:1], w), (w, w[0]), (w, w.bfloat16())):
        with pytest.raises(ValueError, match="same shape"):
            m.muon_tensors([w], [g], [v])
    with pytest.raises(ValueError, match="matrix"):
        m.muon_tensors([w[0, 0]], [w[0, 0]], [w[0, 0]])
    with pytest.raises(ValueError, match="CUDA"):
        m.muon_tensors([w], [w], [w])
    with pytest.raises(ValueError, match="empty"):
        m.Muon([], [])


def test_direction_arguments(m, device0):
    s = m.MoEOrthShape()
    s.batch, s.rows, s.cols, s.dtype = 2, 8, 16, m.MOE_F32
    x, ws = torch.zeros(2, 8, 16), torch.zeros(512, dtype=torch.uint8)
    for a, b in ((x.bfloat16(), x), (x[:1], x), (x, None), (x, x.transpose(1, 2))):
        with pytest.raises(ValueError):
            m.moe_orthogonalize(s, m.orth_coefs(), a, b, ws, stream=0)
