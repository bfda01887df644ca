"""One workspace for calls of any shapes and operators in turn: its first 256 bytes aside,
what a call finds there is another call's leavings, here also NaN bits throughout.  The results
are the same bits as from workspaces of their own."""
import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, dt=F32: torch.randn(s, generator=g, device="cuda").to(dt)


def share(ops):
    """The largest workspace for all of them; its bytes after the status words as NaN."""
    ws = max((op.ws for op in ops), key=lambda w: w.numel())
    for op in ops:
        op.ws = ws
    return lambda: ws[256:].fill_(0xFF)


# m, n around the tiles and paddings; whole and in pieces; the first steps paired and not; clusters
DIRECTIONS = [((2, 300, 2500), F32), ((1, 130, 258), BF), ((3, 777, 1001), F32), ((37, 130, 1100), BF), ((1, 129, 4100), BF),
              ((2, 513, 100), BF), ((5, 256, 512), BF), ((2, 200, 330), F32), ((1, 700, 5000), BF), ((6, 260, 1030), F32),
              ((1, 1030, 520), BF), ((2, 100, 4500), F32), ((1, 257, 300), BF)]


def test_directions_of_many_shapes():
    ops, xs, want = [], [], []
    for i, (shape, dt) in enumerate(DIRECTIONS):
        ops.append(m.Orthogonalize(*shape, dtype=dt))
        xs.append(gen(i)(*shape, dt=dt))
        want.append(ops[-1].forward(xs[-1]))
    assert all(bool(torch.isfinite(t).all()) for t in want)
    spoil = share(ops)
    order = list(range(len(ops)))
    for spoiled in (True, False):
        for i in order + order[::-1]:
            if spoiled:
                spoil()
            assert torch.equal(ops[i].forward(xs[i]), want[i]), DIRECTIONS[i]
    assert ops[0].device_status() == (0, 0)


def test_steps_of_many_lists():
    lists = [[(4, 72, 136), (4, 136, 72), (3, 140, 264)], [(2, 300, 900), (900, 300)], [(1, 200, 1200)] * 3 + [(131, 131)],
             [(40, 128, 1000), (2, 129, 70)]]
    runs = []
    for i, shapes in enumerate(lists):
        r = gen(i)
        dt = BF if i % 2 else F32
        start = [r(*s, dt=dt) for s in shapes]
        grads = [r(*s, dt=dt if i < 2 else F32) for s in shapes]
        params = [p.clone() for p in start]
        op = m.Muon(params, grads, lr=0.1, weight_decay=0.1)
        op.step()
        runs.append((op, start, params, [p.clone() for p in params], [v.clone() for v in op.momenta]))
    spoil = share([r[0] for r in runs])
    for op, start, params, want, momenta in runs + runs[::-1]:
        for p, s in zip(params, start):
            p.copy_(s)
        for v in op.momenta:
            v.zero_()
        spoil()
        op.step()
        assert all(torch.equal(p, q) for p, q in zip(params + op.momenta, want + momenta))
        assert op.device_status() == (0, 0)


def test_norms_and_embeddings_in_turn():
    calls, ops = [], []
    for i, (T, H, dt, gate) in enumerate([(50, 264, BF, "token"), (3000, 1024, F32, "channel"), (1, 2048, BF, None),
                                          (300, 8200, F32, "token"), (6000, 64, BF, "channel"), (40, 16384, BF, None)]):
        r = gen(i)
        a = dict(y=r(T, H, dt=dt), w_post=r(H, dt=dt), w_pre=r(H, dt=dt),
                 gate={None: None, "channel": r(H, dt=dt), "token": r(T)}[gate])
        x, ds, dh = r(T, H, dt=dt), r(T, H, dt=dt), r(T, H, dt=dt)
        op = m.BlockNorm(T, H, dtype=dt, gate=gate)
        op.forward(x, **a)
        ops.append(op)
        calls.append(lambda op=op, ds=ds, dh=dh, x=x, a=a: [t for t in op.backward(ds, dh, x, **a) if t is not None])
    for i, (T, V, H, dt) in enumerate([(40, 33, 8, F32), (4096, 5000, 264, BF), (20011, 3001, 64, F32), (100003, 1023, 40, F32),
                                       (300, 100001, 72, BF)]):
        r = gen(20 + i)
        ids = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
        dy, add = r(T, H, dt=dt), r(V, H, dt=dt)
        op = m.TokenEmbedding(T, H, V, dtype=dt, padding_idx=3)
        ops.append(op)
        calls.append(lambda op=op, ids=ids, dy=dy, add=add: [op.backward(ids, dy), op.backward(ids, dy, dw_add=add)])
    want = [c() for c in calls]
    spoil = share(ops)
    for spoiled in (True, False):
        for i in list(range(len(calls))) + list(range(len(calls)))[::-1]:
            if spoiled:
                spoil()
            assert all(torch.equal(p, q) for p, q in zip(calls[i](), want[i])), i
    assert ops[0].device_status() == (0, 0)
