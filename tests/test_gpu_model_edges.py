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


@pytest.mark.parametrize("T,H,dt", [(50, 264, torch.bfloat16), (3000, 1024, torch.float32)])
def test_one_object_for_two_layers(T, H, dt):
    """Both forwards, then both backwards, each with its own rstd: the bits of an object each."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    layers = [(r(T, H), dict(y=r(T, H), w_post=r(H), gate=r(H), w_pre=r(H)), r(T, H), r(T, H)) for _ in range(2)]
    want = []
    for x, a, ds, dh in layers:
        op = m.BlockNorm(T, H, dtype=dt, gate="channel")
        want.append(list(op.forward(x, **a)) + list(op.backward(ds, dh, x, **a)))
    one = m.BlockNorm(T, H, dtype=dt, gate="channel")
    rstd = [torch.full((T, 2), float("nan"), device="cuda") for _ in layers]
    got = [list(one.forward(x, **a, rstd=k)) for (x, a, _, _), k in zip(layers, rstd)]
    for i in (1, 0):
        x, a, ds, dh = layers[i]
        got[i] += list(one.backward(ds, dh, x, **a, rstd=rstd[i]))
    for p, q in zip(sum(got, []), sum(want, [])):
        assert torch.equal(p, q)
    with pytest.raises(ValueError, match="rstd"):
        one.forward(layers[0][0], **layers[0][1], rstd=rstd[0][:1])
