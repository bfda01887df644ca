"""What the block norms do when a row's copy into a ring never comes: the bounded wait is
made to give up at once (the copies themselves do arrive, before their block ends), every
row that went through a ring is NaN, the backward's status word says so, and the calls
after it are as before."""
import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

pytestmark = pytest.mark.gpu


def inputs(T, H, dt, gate, post, pre, with_y):
    g = torch.Generator(device="cuda").manual_seed(T + H)

    def r(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    a = dict(y=r(T, H) if with_y else None, w_post=r(H) if post else None,
             gate={None: None, "channel": r(H), "token": r(T, dtype=torch.float32)}[gate], w_pre=r(H) if pre else None)
    return r(T, H), a, r(T, H), r(T, H) if pre else None


@pytest.fixture
def give_up():
    """Waits that give up at once, while the test asks for them."""
    before = []
    yield lambda: before.append(m.moe_testing_set_norm_wait(0))
    m.moe_testing_set_norm_wait(before[0] if before else -1)


CASES = [  # T, H, dtype, gate, post, pre, y: rings in both directions, one and two vectors a thread, short rows
    (6000, 512, torch.bfloat16, "channel", True, True, True), (4000, 2816, torch.bfloat16, "token", True, True, True),
    (25000, 72, torch.float32, None, True, True, True), (3000, 4096, torch.float32, "channel", False, True, True),
    (6000, 1000, torch.bfloat16, "token", True, False, True), (6000, 1000, torch.bfloat16, None, False, False, False),
    (6000, 264, torch.float32, None, False, True, False), (3000, 7168, torch.bfloat16, None, False, False, True)]


@pytest.mark.parametrize("T,H,dt,gate,post,pre,with_y", CASES)
def test_lost_copies(give_up, T, H, dt, gate, post, pre, with_y):
    x, a, ds, dh = inputs(T, H, dt, gate, post, pre, with_y)
    op = m.BlockNorm(T, H, dtype=dt, gate=gate)

    def both():
        return list(op.forward(x, **a)), list(op.backward(ds, dh, x, **a))

    forward, back = both()
    rstd = op.rstd.clone()
    assert op.device_status() == (m.MOE_OK, 0)
    give_up()
    for t in op.forward(x, **a):
        assert t is None or bool(t.isnan().all())
    op.rstd.copy_(rstd)      # the backward by itself
    for t in op.backward(ds, dh, x, **a):
        assert t is None or bool(t.isnan().all())
    assert op.device_status() == (m.MOE_ERR_TIMEOUT, 4)
    m.moe_testing_set_norm_wait(-1)
    again = both()
    assert op.device_status() == (m.MOE_OK, 0)
    for p, q in zip(forward + back, again[0] + again[1]):
        assert (p is None) == (q is None) and (p is None or torch.equal(p, q))


def test_a_few_lost_copies_end_in_time(give_up):
    """Many steps a block: one wait is given up, not each step's."""
    T, H = 400000, 64
    x, a, ds, dh = inputs(T, H, torch.bfloat16, None, True, True, True)
    op = m.BlockNorm(T, H)
    op.forward(x, **a)
    give_up()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    op.backward(ds, dh, x, **a)
    op.forward(x, **a)
    end.record()
    end.synchronize()
    assert start.elapsed_time(end) < 100.0
    assert op.device_status() == (m.MOE_ERR_TIMEOUT, 4)
