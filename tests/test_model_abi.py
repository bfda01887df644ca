"""The C ABI of the embedding, the block norms and the orthogonalised update without a
GPU: the symbols exist with the binding's arguments, and bad arguments are rejected on
the host before any CUDA call."""
import ctypes
import math
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    from mixture_experts_ffn_04_gb300 import build
    build.build()
    m.lib()
    return m


def test_exports_every_declared_symbol_with_its_arguments(m):
    src = open(os.path.join(ROOT, "include", "moe_model.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    found = re.findall(r"^[A-Za-z_][\w \*]*?\b(moe_\w+)\s*\(([^;{]*?)\)\s*;", src, flags=re.M | re.S)
    assert len(found) == 10
    for name, args in found:
        assert len(getattr(m.lib(), name).argtypes) == args.count(",") + 1, name
    assert m.moe_status_string(m.MOE_ERR_TOKEN) == "MOE_ERR_TOKEN"


def rejected(m, st, word=""):
    assert st in (m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED), st
    assert word in m.moe_last_error(), m.moe_last_error()


def embed_shape(m, **kw):
    s = m.MoEEmbedShape()
    s.tokens, s.hidden, s.vocab, s.dtype, s.padding_idx, s.scale = 64, 256, 1000, m.MOE_BF16, -1, 1.0
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,word", [
    (dict(tokens=-1), "tokens"), (dict(tokens=(1 << 28) + 1), "tokens"), (dict(hidden=0), "hidden"),
    (dict(hidden=12), "hidden"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 30) + 1), "vocab"),
    (dict(dtype=5), "dtype"), (dict(padding_idx=-2), "padding"), (dict(padding_idx=1000), "padding"),
    (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"), (dict(scale=1e300), "scale"),
    (dict(w_stride=128), "stride"), (dict(w_stride=260), "stride"), (dict(w_stride=-8), "stride")])
def test_embedding_shapes(m, kw, word):
    s = embed_shape(m, **kw)
    assert m.moe_embed_workspace_bytes(s) == 0 and word in m.moe_last_error()
    ref = ctypes.byref(s)
    rejected(m, m.lib().moe_embed_forward(ref, 16, 16, 16, 256, 1 << 40, None), word)
    rejected(m, m.lib().moe_embed_backward(ref, 16, 16, None, 16, 256, 1 << 40, None), word)


def test_embedding_arguments(m):
    f, b = m.lib().moe_embed_forward, m.lib().moe_embed_backward
    s = embed_shape(m)
    ref, n = ctypes.byref(s), m.moe_embed_workspace_bytes(s)
    rejected(m, f(None, 16, 16, 16, 256, n, None))
    for hole in range(3):
        a = [16, 16, 16]
        a[hole] = None
        rejected(m, f(ref, *a, 256, n, None), "non-NULL")
        rejected(m, b(ref, a[0], a[1], None, a[2], 256, n, None), "non-NULL")
    rejected(m, f(ref, 8, 16, 16, 256, n, None), "aligned")
    rejected(m, f(ref, 16, 2, 16, 256, n, None), "aligned")
    rejected(m, b(ref, 16, 24, None, 16, 256, n, None), "aligned")
    rejected(m, b(ref, 16, 16, 8, 16, 256, n, None), "aligned")
    for ws, size in ((None, n), (128, n), (256, n - 1)):
        assert f(ref, 16, 16, 16, ws, size, None) == m.MOE_ERR_WORKSPACE
        assert b(ref, 16, 16, None, 16, ws, size, None) == m.MOE_ERR_WORKSPACE


def norm_shape(m, **kw):
    s = m.MoEBlockNormShape()
    s.tokens, s.hidden, s.dtype, s.residual_scale, s.eps = 64, 256, m.MOE_BF16, 1.0, 1e-6
    for k, v in kw.items():
        setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw,word", [
    (dict(tokens=-1), "tokens"), (dict(hidden=0), "hidden"), (dict(hidden=20), "hidden"),
    (dict(hidden=32776), "hidden"), (dict(dtype=7), "dtype"), (dict(gate=3), "gate"), (dict(gate=-1), "gate"),
    (dict(unit_offset=2), "unit_offset"), (dict(residual_scale=math.nan), "residual"), (dict(eps=0.0), "eps"),
    (dict(eps=-1.0), "eps"), (dict(eps=math.inf), "eps"), (dict(eps=1e-60), "eps")])
def test_norm_shapes(m, kw, word):
    s = norm_shape(m, **kw)
    assert m.moe_block_norm_workspace_bytes(s) == 0 and word in m.moe_last_error()
    ref = ctypes.byref(s)
    rejected(m, m.lib().moe_block_norm_forward(ref, 16, 16, 16, None, 16, 16, 16, 16, None), word)
    rejected(m, m.lib().moe_block_norm_backward(ref, 16, 16, 16, 16, 16, None, 16, 16, 16, 16, 16, None, 16, 256, 1 << 40,
                                                None), word)


def test_norm_arguments(m):
    f, b = m.lib().moe_block_norm_forward, m.lib().moe_block_norm_backward
    s = norm_shape(m)
    ref, n = ctypes.byref(s), m.moe_block_norm_workspace_bytes(s)
    rejected(m, f(ref, None, 16, 16, None, 16, 16, 16, 16, None), "x must")
    rejected(m, f(ref, 16, None, 16, None, 16, 16, 16, 16, None), "need y")
    rejected(m, f(ref, 16, 16, 16, 16, 16, 16, 16, 16, None), "gate")          # a gate the shape has not
    rejected(m, f(ref, 16, 16, 16, None, 16, 16, None, 16, None), "h must")
    rejected(m, f(ref, 16, 16, 16, None, None, 16, 16, 16, None), "h must")
    rejected(m, f(ref, 16, 16, 16, None, None, None, None, 16, None), "one of s and h")
    for hole in (0, 1, 2, 4, 5, 6):
        a = [16, 16, 16, None, 16, 16, 16, 16]
        a[hole] = 24
        rejected(m, f(ref, *a, None), "aligned")
    rejected(m, f(ref, 16, 16, 16, None, 16, 16, 16, 4, None), "rstd")
    good = [16, 16, 16, 16, 16, None, 16, 16, 16, 16, 16, None, 16]
    def back(**kw):
        names = ("ds", "dh", "x", "y", "w_post", "gate", "w_pre", "rstd", "dx", "dy", "dw_post", "dgate", "dw_pre")
        a = dict(zip(names, good))
        a.update(kw)
        return b(ref, *[a[k] for k in names], 256, n, None)
    rejected(m, back(dh=None), "dh must")
    rejected(m, back(w_pre=None, dw_pre=None), "dh must")
    rejected(m, back(ds=None, dh=None, w_pre=None, dw_pre=None), "one of ds")
    rejected(m, back(rstd=None), "rstd")
    rejected(m, back(y=None, w_post=None, dw_post=None), "input")
    rejected(m, back(w_post=None), "input")
    rejected(m, back(dgate=16), "input")
    rejected(m, back(dx=None, dy=None, dw_post=None, dw_pre=None), "no gradient")
    rejected(m, back(dx=8), "aligned")
    rejected(m, back(dw_pre=17), "aligned")
    for ws, size in ((None, n), (128, n), (256, n - 1)):
        assert b(ref, *good, ws, size, None) == m.MOE_ERR_WORKSPACE


def test_coefficients(m):
    s = m.MoEOrthShape()
    s.batch, s.rows, s.cols, s.dtype = 2, 64, 200, m.MOE_BF16

    def bytes_of(*triples, eps=1e-7, steps=None):
        c = m.orth_coefs(triples, eps=eps)
        if steps is not None:
            c.steps = steps
        return m.moe_orthogonalize_workspace_bytes(s, c)

    assert bytes_of((3.4445, -4.7750, 2.0315)) > 0
    assert bytes_of(*[(3.4445, -4.7750, 2.0315)] * 16) > 0
    assert bytes_of((1.5, -0.5, 0.0)) > 0 and bytes_of((1.0, 0.0, 0.0)) > 0
    assert bytes_of((8.28721201814563, -23.595886519098837, 17.300387312530933)) > 0
    for bad, word in (((3.6, 0.0, 0.0), "3.5"), ((math.nan, 0.0, 0.0), "finite"), ((2.0, 0.0, 300.0), "3.5"),
                      ((0.0, -3.0, -3.0), "3.5")):
        assert bytes_of(bad) == 0 and word in m.moe_last_error(), bad
    assert bytes_of((3.0, 0.0, 0.0), (3.0, 0.0, 0.0)) == 0 and "3.5" in m.moe_last_error()
    # 30 s - 200 s^3 + 172 s^5 stays below 3.5 in size only near its ends
    assert bytes_of((30.0, -200.0, 172.0)) == 0
    assert bytes_of((102.0, -203.0, 102.0)) == 0
    for eps in (-1.0, math.inf, math.nan):
        assert bytes_of((1.0, 0.0, 0.0), eps=eps) == 0 and "eps" in m.moe_last_error()
    for steps in (0, 17, -1):
        assert bytes_of((1.0, 0.0, 0.0), steps=steps) == 0 and "steps" in m.moe_last_error()
    for bad in ([], [(1.0, 2.0)], [(1.0, 2.0, 3.0)] * 17):
        with pytest.raises(ValueError):
            m.orth_coefs(bad)
    with pytest.raises(ValueError):
        m.orth_coefs((1.0, 0.0, 0.0), steps=0)


@pytest.mark.parametrize("kw,word", [(dict(batch=-1), "batch"), (dict(batch=(1 << 24) + 1), "batch"),
                                     (dict(rows=0), "rows"), (dict(cols=65537), "rows"), (dict(dtype=3), "dtype"),
                                     (dict(reserved=1), "reserved")])
def test_direction_shapes(m, kw, word):
    s, c = m.MoEOrthShape(), m.orth_coefs()
    s.batch, s.rows, s.cols, s.dtype = 2, 64, 200, m.MOE_F32
    for k, v in kw.items():
        setattr(s, k, v)
    assert m.moe_orthogonalize_workspace_bytes(s, c) == 0 and word in m.moe_last_error()
    rejected(m, m.lib().moe_orthogonalize(ctypes.byref(s), ctypes.byref(c), 16, 16, 256, 1 << 40, None), word)


def test_direction_arguments(m):
    s, c = m.MoEOrthShape(), m.orth_coefs()
    s.batch, s.rows, s.cols, s.dtype = 2, 300, 200, m.MOE_F32
    n = m.moe_orthogonalize_workspace_bytes(s, c)
    f, a = m.lib().moe_orthogonalize, (ctypes.byref(s), ctypes.byref(c))
    rejected(m, f(None, a[1], 16, 16, 256, n, None))
    rejected(m, f(a[0], None, 16, 16, 256, n, None))
    rejected(m, f(*a, None, 16, 256, n, None), "non-NULL")
    rejected(m, f(*a, 16, 2, 256, n, None), "aligned")
    for ws, size in ((None, n), (128, n), (256, n - 1)):
        assert f(*a, 16, 16, ws, size, None) == m.MOE_ERR_WORKSPACE


def test_update_lists(m):
    def entry(**kw):
        arr = (m.MoEMuonTensor * 1)()
        e = arr[0]
        e.param, e.grad, e.momentum, e.batch, e.rows, e.cols = 16, 16, 16, 2, 300, 200
        e.param_dtype, e.grad_dtype = m.MOE_BF16, m.MOE_F32
        for k, v in kw.items():
            setattr(e, k, v)
        return arr

    def config(**kw):
        c = m.MoEMuonConfig()
        c.lr, c.momentum, c.weight_decay, c.coefs = 0.02, 0.95, 0.0, m.orth_coefs()
        for k, v in kw.items():
            setattr(c, k, v)
        return c

    n = m.moe_muon_workspace_bytes(entry(), config())
    assert n > 0
    step = m.lib().moe_muon_step
    for kw, word in ((dict(param=None), "non-NULL"), (dict(grad=None), "non-NULL"), (dict(momentum=None), "non-NULL"),
                     (dict(param=1), "aligned"), (dict(grad=18), "aligned"), (dict(momentum=6), "aligned"),
                     (dict(batch=-1), "batch"), (dict(rows=0), "rows"), (dict(cols=-4), "rows"),
                     (dict(param_dtype=9), "dtypes"), (dict(grad_dtype=9), "dtypes")):
        assert m.moe_muon_workspace_bytes(entry(**kw), config()) == 0
        rejected(m, step(entry(**kw), 1, ctypes.byref(config()), 256, 1 << 40, None), word)
    for kw, word in ((dict(lr=math.nan), "lr"), (dict(momentum=1.0), "momentum"), (dict(momentum=-0.1), "momentum"),
                     (dict(weight_decay=math.inf), "weight_decay"), (dict(nesterov=2), "nesterov"),
                     (dict(scale=3), "scale")):
        rejected(m, step(entry(), 1, ctypes.byref(config(**kw)), 256, 1 << 40, None), word)
    rejected(m, step(entry(), 1, None, 256, n, None), "config")
    rejected(m, step(entry(), -1, ctypes.byref(config()), 256, n, None), "tensors")
    rejected(m, step(None, 1, ctypes.byref(config()), 256, n, None), "tensors")
    for ws, size in ((None, n), (128, n), (256, n - 1)):
        assert step(entry(), 1, ctypes.byref(config()), ws, size, None) == m.MOE_ERR_WORKSPACE
    # a list's workspace is its largest part's, whichever way round the matrices are
    wide, tall = entry(batch=4, rows=300, cols=500), entry(batch=4, rows=500, cols=300)
    both = (m.MoEMuonTensor * 2)(wide[0], tall[0])
    assert m.moe_muon_workspace_bytes(both, config()) > m.moe_muon_workspace_bytes(wide, config())
    assert m.moe_muon_workspace_bytes(wide, config()) == m.moe_muon_workspace_bytes(tall, config())
