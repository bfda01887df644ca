"""Global gradient norm and clipping on the GPU against float64.

Bounds (derived): f = 2^-24.  A thread adds at most 80 squares in fp32 before
the tree, every square and addition rounded: the norm's relative error is at most
half of (80 + 12) f at worst, 64 f is allowed.  coef has that error and its own
rounding; the product and the store round once each: per element relative
64 f + 3 f + u of the destination.
"""
import math

import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: F}
BF, FP = torch.bfloat16, torch.float32


def make(sizes, seed=0, scale=1e-3):
    """Gradients of (numel, dtype) at odd element offsets of flat buffers."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    flat = {dt: (torch.randn(sum(n for n, d in sizes if d == dt) + len(sizes) + 1, generator=g,
                             device="cuda") * scale).to(dt) for dt in (BF, FP)}
    at, out = {BF: 1, FP: 1}, []
    for i, (n, dt) in enumerate(sizes):
        out.append(flat[dt][at[dt]: at[dt] + n])
        at[dt] += n + (i % 2)
    return out


def reference(grads, max_norm):
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))


def check(grads, max_norm, out=None):
    before = [g.clone() for g in grads]
    norm, coef = reference(before, max_norm)
    op = m.GradClip(grads, out=out)
    got = float(op.clip(max_norm))
    assert abs(got - norm) <= 64 * F * norm
    for b, o in zip(before, grads if out is None else out):
        want = b.double() * coef
        if coef == 1.0 and o.dtype == b.dtype:
            assert torch.equal(o, b)
        # values under the type's normal range round absolutely
        assert ((o.double() - want).abs() <= (67 * F + U[o.dtype]) * want.abs() + 2.0 ** -133).all()
    return op, got


LISTS = [[(1, FP)], [(1, BF), (0, FP), (3, FP)], [(7, BF), (16383, BF), (16384, FP), (16385, BF)],
         [(100003, FP), (50001, BF), (1, BF), (2, FP)],
         [(i * 37 % 1000 + 1, BF if i % 3 else FP) for i in range(300)]]


@pytest.mark.parametrize("i", range(len(LISTS)))
@pytest.mark.parametrize("clips", [True, False])
def test_in_place(i, clips):
    grads = make(LISTS[i], seed=i)
    norm, _ = reference(grads, 1.0)
    check(grads, norm * (0.25 if clips else 4.0))


@pytest.mark.parametrize("clips", [True, False])
@pytest.mark.parametrize("src", [BF, FP])
@pytest.mark.parametrize("dst", [BF, FP])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_into_another_buffer_and_type(clips, src, dst, shift):
    grads = make([(20001, src), (9, src), (65536, src)], seed=5)
    outs = [torch.full((g.numel() + 8,), 7.0, device="cuda", dtype=dst) for g in grads]
    views = [o[shift: shift + g.numel()] for o, g in zip(outs, grads)]
    keep = [g.clone() for g in grads]
    norm, _ = reference(grads, 1.0)
    check(grads, norm * (0.5 if clips else 2.0), out=views)
    for o, g, k in zip(outs, grads, keep):
        assert torch.equal(g, k)
        assert (o[:shift] == 7).all() and (o[shift + g.numel():] == 7).all()


def test_norm_alone_and_entries_without_destination():
    grads = make([(5000, BF), (70000, FP)])
    keep = [g.clone() for g in grads]
    norm, _ = reference(grads, 1.0)
    assert abs(float(m.GradClip(grads).clip(math.inf)) - norm) <= 64 * F * norm
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    check_out = torch.empty_like(grads[1])
    op = m.GradClip(grads, out=[None, check_out])
    op.clip(norm / 2)
    assert torch.equal(grads[0], keep[0])
    want = keep[1].double() * (norm / 2 / (norm + 1e-6))
    assert ((check_out.double() - want).abs() <= 70 * F * want.abs()).all()


@pytest.mark.parametrize("scale", [1e25, 1e-24, 1e-36])
def test_norms_whose_squares_leave_the_range(scale):
    grads = make([(40000, FP), (20000, BF)], scale=scale)
    norm, _ = reference(grads, 1.0)
    got = float(m.GradClip(grads).clip(math.inf))
    # bf16 and fp32 values near the bottom of the range are what they are; the
    # reference reads the same ones
    assert abs(got - norm) <= 64 * F * norm


def test_zero_gradients():
    grads = [torch.zeros(50000, device="cuda"), torch.zeros(3, device="cuda", dtype=BF)]
    assert float(m.GradClip(grads).clip(1.0)) == 0.0
    assert all((g == 0).all() for g in grads)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norm_that_is_not_finite_leaves_the_gradients(bad):
    grads = make([(40000, FP), (333, BF)])
    grads[1][7] = bad
    keep = [g.clone() for g in grads]
    norm = float(m.GradClip(grads).clip(1e-3))
    assert math.isnan(norm) if math.isnan(bad) else math.isinf(norm)
    for g, k in zip(grads, keep):
        assert torch.equal(g.view(torch.int16 if g.dtype == BF else torch.int32),
                           k.view(torch.int16 if g.dtype == BF else torch.int32))


def test_repeatable_other_stream_and_graph():
    grads = make([(300001, BF), (77777, FP)], seed=8)
    outs = [torch.empty_like(g) for g in grads]
    op = m.GradClip(grads, out=outs)
    n0 = op.clip(1e-2)
    first = [o.clone() for o in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n1 = op.clip(1e-2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n2 = op.clip(1e-2)
    for g in grads:
        g.mul_(3.0)
    graph.replay()
    norm, coef = reference(grads, 1e-2)
    assert abs(float(n2) - norm) <= 64 * F * norm


def test_more_elements_than_a_launch_has_threads():
    """Chunks several times the grid; one tensor past 2^31 bytes."""
    g = torch.full((1 << 30 | 5,), 2.0 ** -10, device="cuda", dtype=BF)
    got = float(m.GradClip([g]).clip(16.0))
    norm = math.sqrt(g.numel()) * 2.0 ** -10
    assert abs(got - norm) <= 64 * F * norm
    want = torch.tensor(2.0 ** -10 * (16.0 / (norm + 1e-6)), dtype=torch.float64)
    for part in (g[:5], g[-5:], g[1 << 29: (1 << 29) + 5]):
        assert ((part.double().cpu() - want).abs() <= 2.0 ** -8 * want).all()


@pytest.mark.parametrize("n", [2048 * 600, 2048 * 1216, 2048 * 1217, 2048 * 2433])
def test_around_the_chunk_sizes(n):
    """Lists just below and above the limits at which the chunks double, repeated:
    the counters are ready for the next call."""
    grads = make([(n - 5000, FP), (4990, BF), (10, FP)], seed=3)
    outs = [torch.empty_like(g) for g in grads]
    norm, coef = reference(grads, 1.0)
    op = m.GradClip(grads, out=outs)
    for clip in (norm * 0.5, norm * 0.25, norm * 3.0):
        got = float(op.clip(clip))
        assert abs(got - norm) <= 64 * F * norm
        c = min(1.0, clip / (norm + 1e-6))
        for g, o in zip(grads, outs):
            want = g.double() * c
            assert ((o.double() - want).abs() <= (67 * F + U[o.dtype]) * want.abs() + 2.0 ** -133).all()
    assert op.device_status() == (m.MOE_OK, 0)
