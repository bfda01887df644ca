"""Calls at the edges of what the embedding and the block norms allow."""
import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("pre,post", [(True, True), (False, True), (True, False), (False, False)])
def test_norms_of_no_tokens(gate, pre, post):
    """The class on empty tensors: empty outputs, and sums over no tokens."""
    op = m.BlockNorm(0, 64, gate=gate)
    e = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    g = {None: None, "channel": w, "token": torch.empty(0, device="cuda")}[gate]
    kw = dict(w_post=w if post else None, gate=g, w_pre=w if pre else None)
    s, h = op.forward(e, e, **kw)
    d = op.backward(e, e if pre else None, e, e, **kw)
    assert s.shape == d.dx.shape == d.dy.shape == (0, 64) and (h is None) == (not pre)
    for t in (d.dw_post, d.dw_pre, d.dgate):
        assert t is None or t.numel() == 0 or float(t.abs().max()) == 0.0
    only = op.backward(e, None, e) if gate is None else None
    assert only is None or only.dx.shape == (0, 64)
    assert op.device_status() == (m.MOE_OK, 0)
