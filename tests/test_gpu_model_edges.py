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


@pytest.mark.parametrize("gate", [None, "token", "channel"])
@pytest.mark.parametrize("T,H,dt", [(40, 256, torch.float32), (40, 2816, torch.bfloat16), (9, 8200, torch.float32)])
def test_rows_of_zeros_under_a_tiny_eps(T, H, dt, gate):
    """1 / sqrt(eps) of both norms is a number of fp32, their product is not: nothing of a row of
    zeros reaches the sums over rows, and dx, dy are ds, dh times what the formula says."""
    eps = 1e-42
    g = torch.Generator(device="cuda").manual_seed(H)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)
    z, w, ds = torch.zeros((T, H), device="cuda", dtype=dt), r(H), r(T, H)
    k = {None: None, "channel": r(H), "token": torch.rand(T, generator=g, device="cuda")}[gate]
    op = m.BlockNorm(T, H, dtype=dt, gate=gate, eps=eps)
    s, h = op.forward(z, z, w_post=w, gate=k, w_pre=w)
    assert float(s.abs().max()) == float(h.abs().max()) == 0.0
    d = op.backward(ds, torch.zeros_like(ds), z, z, w_post=w, gate=k, w_pre=w)
    for t in (d.dw_post, d.dw_pre, d.dgate):
        assert t is None or float(t.abs().max()) == 0.0
    assert torch.equal(d.dx, ds)
    # dy = g ds w_post / sqrt(eps): four roundings of fp32 and the reciprocal root's two units, then the type's.
    # eps is a subnormal of fp32 here: what it is rounded to counts
    root = float(torch.tensor(eps, dtype=torch.float32).double()) ** -0.5
    gain = 1.0 if k is None else (k.double() if gate == "channel" else k.double()[:, None])
    want = gain * ds.double() * w.double() * root
    tol = torch.finfo(dt).eps / 2 + 8 * 2.0 ** -24
    assert bool(((d.dy.double() - want).abs() <= tol * want.abs()).all())
    # rows of values beside them
    x = r(T, H)
    x[::2] = 0.0
    s, h = op.forward(x, x, w_post=w, gate=k, w_pre=w)
    d = op.backward(torch.zeros_like(ds), ds, x, x, w_post=w, gate=k, w_pre=w)
    for t in (s, h, d.dw_pre):
        assert bool(torch.isfinite(t).all())
    assert float(h[::2].abs().max()) == 0.0


@pytest.mark.parametrize("T,V,H", [(300000, 5, 16), (60001, 300, 256), (9000, 40, 64), (64, 1, 264), (64, 3, 8)])
def test_infinities_and_overflow_of_a_gradient_stay(T, V, H):
    """An infinite term gives an infinite sum, one of each sign or a NaN give NaN, and finite terms whose
    sum leaves the range its infinity; the other columns are as they were."""
    g = torch.Generator(device="cuda").manual_seed(T + 1)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    dy = torch.rand((T, H), generator=g, device="cuda")
    op = m.TokenEmbedding(T, H, V, dtype=torch.float32)
    clean = op.backward(ids, dy)
    row = int(ids[T // 2])
    mine = (ids == row).nonzero()[:, 0]
    dy[mine[len(mine) // 2], 1] = float("inf")
    dy[mine[0], 2], dy[mine[-1], 2] = float("inf"), float("-inf")
    dy[mine[-1], 3] = float("nan")
    dy[mine, 4] = 3e38
    got = op.backward(ids, dy)
    several = len(mine) > 1
    assert float(got[row, 1]) == float("inf") and bool(got[row, 3].isnan())
    assert bool(got[row, 2].isnan()) if several else float(got[row, 2]) == float("-inf")
    assert float(got[row, 4]) == (float("inf") if several else float(torch.tensor(3e38)))
    clean[row, 1:5] = got[row, 1:5] = 0.0
    assert torch.equal(got, clean)
