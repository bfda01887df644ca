"""The training operators' C ABI without a GPU: the symbols exist, and bad
arguments are rejected on the host before any CUDA call."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    from mixture_experts_ffn_04_gb300 import build
    build.build()
    m.lib()
    return m


def test_exports_every_declared_symbol(m):
    src = open(os.path.join(ROOT, "include", "moe_train.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(moe_\w+)\s*\(", src, flags=re.M)))
    assert len(names) == 8
    lib = ctypes.CDLL(m.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    assert m.moe_status_string(m.MOE_ERR_TARGET) == "MOE_ERR_TARGET"


def ce_shape(m, **kw):
    s = m.MoECeShape()
    s.tokens, s.hidden, s.vocab, s.dtype = 64, 256, 1000, m.MOE_BF16
    s.reduction, s.ignore_index = m.MOE_CE_MEAN, -100
    for k, v in kw.items():
        setattr(s, k, v)
    return s


BAD_CE = [(dict(tokens=-1), "tokens"), (dict(hidden=0), "hidden"), (dict(hidden=12), "hidden"),
          (dict(vocab=0), "vocab"), (dict(dtype=5), "dtype"), (dict(reduction=3), "reduction"),
          (dict(x_stride=128), "stride"), (dict(w_stride=260), "stride"), (dict(x_stride=-8), "stride")]


@pytest.mark.parametrize("kw,word", BAD_CE)
def test_ce_shapes_rejected(m, kw, word):
    s = ce_shape(m, **kw)
    assert m.moe_linear_ce_workspace_bytes(s) == 0
    for st in (m.lib().moe_linear_ce_forward(ctypes.byref(s), 16, 16, 16, 16, 16, 16, 16, 256, 1 << 40, None),
               m.lib().moe_linear_ce_backward(ctypes.byref(s), 16, 16, 16, 16, 16, 16, 16, 256, 1 << 40, None)):
        assert st in (m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED)
        assert word in m.moe_last_error()


def test_ce_arguments_rejected(m):
    f, b = m.lib().moe_linear_ce_forward, m.lib().moe_linear_ce_backward
    s = ce_shape(m)
    ref, n = ctypes.byref(s), m.moe_linear_ce_workspace_bytes(s)
    assert n > 0
    inv, wse = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_WORKSPACE
    assert f(None, 16, 16, 16, 16, 16, 16, 16, 256, n, None) == inv
    for hole in range(3):
        a = [16, 16, 16]
        a[hole] = None
        assert f(ref, *a, 16, 16, 16, 16, 256, n, None) == inv
        assert b(ref, *a, 16, 16, 16, 16, 256, n, None) == inv
    assert f(ref, 16, 16, 16, None, None, None, None, 256, n, None) == inv
    assert f(ref, 16, 16, 16, 16, 16, 4, 16, 256, n, None) == inv
    assert f(ref, 8, 16, 16, 16, 16, 16, 16, 256, n, None) == inv
    assert f(ref, 16, 24, 16, 16, 16, 16, 16, 256, n, None) == inv
    assert f(ref, 16, 16, 16, 16, 16, 16, 16, None, n, None) == wse
    assert f(ref, 16, 16, 16, 16, 16, 16, 16, 128, n, None) == wse
    assert f(ref, 16, 16, 16, 16, 16, 16, 16, 256, n - 1, None) == wse
    assert b(ref, 16, 16, 16, None, 16, 16, 16, 256, n, None) == inv
    assert b(ref, 16, 16, 16, 4, 16, 16, 16, 256, n, None) == inv
    assert b(ref, 16, 16, 16, 16, 16, None, None, 256, n, None) == inv
    assert b(ref, 16, 16, 16, 16, 16, 8, 16, 256, n, None) == inv
    assert b(ref, 16, 16, 16, 16, 16, 16, 16, 256, n - 1, None) == wse
    none = ce_shape(m, reduction=m.MOE_CE_NONE)
    assert f(ctypes.byref(none), 16, 16, 16, 16, 16, 16, 16, 256, n, None) == inv
    assert b(ctypes.byref(none), 16, 16, 16, 16, None, 16, 16, 256, n, None) == inv


def test_ce_binding_checks_tensors(m):
    s = ce_shape(m)
    x, w = torch.zeros(64, 256, dtype=torch.bfloat16), torch.zeros(1000, 256, dtype=torch.bfloat16)
    t, ws = torch.zeros(64, dtype=torch.int32), torch.zeros(16, dtype=torch.uint8)
    lse, st, tot = torch.zeros(64), torch.zeros(64, 4), torch.zeros(1)
    for bad in (dict(x=x.float()), dict(x=x[:63]), dict(w=w[:, :248]), dict(t=t.long()), dict(t=t[:5]),
                dict(lse=lse[:3]), dict(st=lse), dict(tot=torch.zeros(2)), dict(x=x.t().contiguous().t())):
        a = dict(x=x, w=w, t=t, lse=lse, st=st, tot=tot)
        a.update(bad)
        with pytest.raises(ValueError):
            m.moe_linear_ce_forward(s, a["x"], a["w"], a["t"], None, a["lse"], a["st"], a["tot"], ws, stream=0)


def test_router_arguments_rejected(m):
    f = m.lib().moe_router_backward
    s = m.MoEShape()
    s.tokens, s.hidden, s.moe_inter, s.topk_shape = 64, 256, 8, m.moe_topk_pack(8, 2)
    s.norm_topk, s.dtype, s.norm_eps = 1, m.MOE_BF16, 1e-6
    n, ref = m.moe_router_backward_workspace_bytes(s), ctypes.byref(s)
    assert n > 0
    inv = m.MOE_ERR_INVALID_ARG

    def call(x=16, w=16, idx=16, dw=16, dg=None, bal=0.1, z=0.1, add=16, dx=16, dwr=16, aux=16, ws=256, nb=n):
        return f(ref, x, w, idx, dw, dg, bal, z, add, dx, dwr, aux, ws, nb, None)

    for bad in (dict(x=None), dict(w=None), dict(idx=None), dict(dx=None), dict(dwr=None), dict(dg=16),
                dict(bal=-1.0), dict(z=float("nan")), dict(bal=float("inf")), dict(x=8), dict(add=4),
                dict(dx=8), dict(dwr=8)):
        assert call(**bad) == inv, bad
    assert call(nb=n - 1) == m.MOE_ERR_WORKSPACE and call(ws=None) == m.MOE_ERR_WORKSPACE
    s.shared_gate, s.shared_inter = 1, 8
    assert call(nb=1 << 40) == inv and "d_gate" in m.moe_last_error()
    s.topk_shape = 0
    assert m.moe_router_backward_workspace_bytes(s) == 0 and call() == inv


def test_clip_arguments_rejected(m):
    L = m.lib()

    def one(**kw):
        t = (m.MoEGradTensor * 1)()
        t[0].src, t[0].dst, t[0].numel, t[0].src_dtype, t[0].dst_dtype = 16, 16, 100, m.MOE_F32, m.MOE_F32
        for k, v in kw.items():
            setattr(t[0], k, v)
        return t

    n = m.moe_grad_clip_workspace_bytes(one())
    assert n > 0
    plan = m.MoEGradPlan()
    for bad in (dict(src=None), dict(numel=-1), dict(src_dtype=7), dict(dst_dtype=-1), dict(src=18),
                dict(dst=18), dict(dst_dtype=m.MOE_BF16)):
        t = one(**bad)
        assert m.moe_grad_clip_workspace_bytes(t) == 0, bad
        assert L.moe_grad_clip_plan(t, 1, ctypes.byref(plan), 256, n, None) in (
            m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED)
    assert L.moe_grad_clip_plan(one(), 1, None, 256, n, None) == m.MOE_ERR_INVALID_ARG
    assert L.moe_grad_clip_plan(one(), 1, ctypes.byref(plan), 256, n - 1, None) == m.MOE_ERR_WORKSPACE
    assert L.moe_grad_clip_plan(one(), 1, ctypes.byref(plan), 128, n, None) == m.MOE_ERR_WORKSPACE
    plan.tensors, plan.chunks, plan.chunk_elems = 1, 1, 16384
    assert L.moe_grad_clip(ctypes.byref(plan), 1.0, None, 256, n, None) == m.MOE_ERR_INVALID_ARG
    for bad in (0.0, -1.0, float("nan")):
        assert L.moe_grad_clip(ctypes.byref(plan), bad, 16, 256, n, None) == m.MOE_ERR_INVALID_ARG
    assert L.moe_grad_clip(ctypes.byref(plan), 1.0, 16, None, n, None) == m.MOE_ERR_WORKSPACE
    plan.chunk_elems = 0
    assert L.moe_grad_clip(ctypes.byref(plan), 1.0, 16, 256, n, None) == m.MOE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        m.GradClip([])
    with pytest.raises(ValueError):
        m.GradClip([torch.zeros(4)], out=[torch.zeros(5)])
    with pytest.raises(ValueError):
        m.GradClip([torch.zeros(4, 4).t()[1:]])
