"""Orthogonalised updates against the definition in float64.

Bounds (derived).  The result of the polynomial's steps has no useful closed error
bound (an error may grow by 4 a step), so the bound is the error that the
documented roundings give on the same input: `modelled` runs the steps in float64
with X in two fp16 parts (bf16 matrices: 19 bits), the operands of every product in one
part (bf16 matrices) or two (fp32), and every product's entry off by up to 2^-19 downwards: the tensor cores cut
the fp32 accumulator at each K = 16 step, by at most 2^-23 of it (a bit of 24), 32
steps of a chunk lose up to half of each, the chunks are added in fp32.  Two draws of such
errors differ by sqrt 2 of one; 2.5 times the modelled error covers that and the
largest of some dozens of draws, u |exact| the output's rounding (bf16 2^-8, fp32
2^-24), relative to the matrix's Frobenius norm.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E24 = 2.0 ** -24
COEFS = (3.4445, -4.7750, 2.0315)
X, A, B = 13, 11, 9      # powers of two of the fp16 parts


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    return m


def exact(u, coefs=(COEFS,) * 5, eps=1e-7):
    tall = u.shape[1] > u.shape[2]
    x = u.double().transpose(1, 2) if tall else u.double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + eps)
    for a, b, c in coefs:
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(1, 2) if tall else x


def modelled(u, planes, coefs=(COEFS,) * 5, eps=1e-7):
    g = torch.Generator(device="cuda").manual_seed(5)

    def parts(v, power):
        v = (v * 2.0 ** power).float()
        hi = v.half()
        low = (v - hi.float()).half().double()
        if planes == 1:
            unit = 2.0 ** (torch.floor(torch.log2(hi.double().abs().clamp_min(2.0 ** -14))) - 18)
            low = torch.round((v.double() - hi.double()) / unit) * unit
        return hi.double() / 2.0 ** power, low / 2.0 ** power

    def product(p, q):
        r = p[0] @ q[0] if planes == 1 else p[0] @ q[0] + p[0] @ q[1] + p[1] @ q[0]
        return r * (1.0 - 2.0 ** -19 * torch.rand(r.shape, generator=g, device="cuda", dtype=torch.float64))

    flip = lambda p: (p[0].mT, p[1].mT)
    tall = u.shape[1] > u.shape[2]
    x = u.double().transpose(1, 2) if tall else u.double()
    x = parts(x / (torch.linalg.matrix_norm(x, keepdim=True) + eps), X)
    for a, b, c in coefs:
        p = parts(product(x, flip(x)), A)
        q = parts(b * (p[0] + (p[1] if planes == 2 else 0)) + c * product(p, p), B)
        x = parts(a * (x[0] + x[1]) + product(q, x), X)
    x = x[0] + x[1]
    return x.transpose(1, 2) if tall else x


def close(got, u, coefs=(COEFS,) * 5, eps=1e-7):
    """got [batch, rows, cols] against the definition, matrix by matrix."""
    want = exact(u, coefs, eps)
    off = modelled(u, 2 if got.dtype == torch.float32 else 1, coefs, eps)
    norm = lambda t: torch.linalg.matrix_norm(t.double())
    bound = 2.5 * norm(off - want) + U[got.dtype] * norm(want) + 8 * E24 * norm(want)
    err = norm(got.double() - want)
    assert bool((err <= bound).all()), (err / bound).tolist()


def draw(shape, dt, seed=0, rank=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, r, c = shape
    if rank is None:
        return torch.randn(shape, generator=g, device="cuda").to(dt)
    return (torch.randn((b, r, rank), generator=g, device="cuda")
            @ torch.randn((b, rank, c), generator=g, device="cuda")).to(dt)


SHAPES = [(1, 1, 1), (1, 1, 9), (2, 9, 1), (3, 7, 5), (2, 16, 16), (5, 8, 64), (1, 64, 200), (2, 129, 70),
          (1, 128, 2048), (1, 257, 300), (4, 100, 513), (3, 513, 100), (2, 256, 256), (2, 777, 1001), (1, 1030, 520),
          # one side at most 128: a cluster a matrix up to a length, more of them than run at once, beyond it
          (40, 128, 1000), (2, 2047, 127), (1, 4096, 100), (2, 33, 4097), (1, 9001, 64), (300, 24, 40), (2, 129, 4000)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_direction(m, shape, dt):
    u = draw(shape, dt, seed=sum(shape))
    op = m.Orthogonalize(*shape, dtype=dt)
    got = op.forward(u)
    close(got, u)
    assert torch.equal(op.forward(u), got)
    again = u.clone()
    assert torch.equal(op.forward(again, out=again), got)
    assert op.device_status() == (0, 0)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rank", [1, 3, 20])
def test_few_directions(m, dt, rank):
    """Matrices of low rank, whose rounding noise the steps amplify most."""
    u = draw((2, 200, 330), dt, seed=rank, rank=rank)
    close(m.Orthogonalize(2, 200, 330, dtype=dt).forward(u), u)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_scale_does_not_matter(m, dt):
    """Powers of two over the type's range give the same bits (eps 0)."""
    u = draw((1, 60, 90), dt, seed=4)
    op = m.Orthogonalize(1, 60, 90, dtype=dt, eps=0.0)
    got = op.forward(u)
    close(got, u, eps=0.0)
    for p in (-100, -60, 60, 100, 124):
        assert torch.equal(op.forward((u.double() * 2.0 ** p).to(dt)), got), p


def test_zeros_and_bad_matrices_stay_alone(m):
    u = draw((6, 70, 100), torch.float32, seed=9)
    op = m.Orthogonalize(6, 70, 100, dtype=torch.float32)
    clean = op.forward(u)
    u[1] = 0.0
    u[3, 5, 5] = float("nan")
    u[4, 6, 7] = float("inf")
    got = op.forward(u)
    assert float(got[1].abs().max()) == 0.0
    assert bool(got[3].isnan().all()) and bool(got[4].isnan().all())
    for i in (0, 2, 5):
        assert torch.equal(got[i], clean[i])
    close(got[1:2], u[1:2], eps=1e-7)
    assert m.Orthogonalize(0, 70, 100).forward(torch.empty((0, 70, 100), device="cuda", dtype=torch.bfloat16)).shape == (0, 70, 100)


def test_steps_of_their_own(m):
    coefs = ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5))
    u = draw((2, 90, 150), torch.float32, seed=2)
    close(m.Orthogonalize(2, 90, 150, dtype=torch.float32, coefficients=coefs).forward(u), u, coefs)
    u = u.bfloat16()
    close(m.Orthogonalize(2, 90, 150, coefficients=(1.5, -0.5, 0.0), steps=1).forward(u), u, coefs[:1])


WIDE = [(1, 129, 258), (3, 200, 400), (2, 130, 1000), (1, 2050, 300), (5, 256, 512)]


@pytest.mark.parametrize("shape", WIDE)
@pytest.mark.parametrize("rank", [None, 1, 16])
def test_first_two_steps_in_one(m, shape, rank):
    """bf16 matrices at least twice as wide as high (or the reverse); the default steps, three
    of them, and two, which stay apart."""
    u = draw(shape, torch.bfloat16, seed=sum(shape), rank=rank)
    for steps in (5, 3, 2):
        op = m.Orthogonalize(*shape, steps=steps)
        got = op.forward(u)
        close(got, u, (COEFS,) * steps)
        assert torch.equal(op.forward(u), got)
        assert op.device_status() == (0, 0)


@pytest.mark.parametrize("third", [(0.3, 0.0, 0.0), (0.9, -0.02, 0.0)])
def test_two_steps_too_large_for_one(m, third):
    """3.5 T5(s), then 3.5 T5(s / 3.5): (b A + c A A) of both and their product pass 200 together."""
    coefs = ((17.5, -70.0, 56.0), (5.0, -20.0 / 12.25, 16.0 / 12.25 ** 2), third)
    coefs = tuple(tuple(0.99 * v for v in c) for c in coefs)
    u = draw((2, 150, 310), torch.bfloat16, seed=5)
    close(m.Orthogonalize(2, 150, 310, coefficients=coefs).forward(u), u, coefs)


def reference_step(w, g, v, lr, beta, nesterov, decay, scale):
    v2 = beta * v.double() + (1.0 - beta) * g.double()
    u = beta * v2 + (1.0 - beta) * g.double() if nesterov else v2
    r, c = w.shape[-2:]
    size = {"none": 1.0, "spectral": max(1.0, r / c) ** 0.5, "rms": 0.2 * max(r, c) ** 0.5}[scale]
    u3 = u.reshape(-1, r, c)
    return v2, u3, size, w.double() * (1.0 - lr * decay)


def check_step(m, params, grads, nesterov, decay, scale, lr=0.05, beta=0.9):
    g = torch.Generator(device="cuda").manual_seed(11)
    momenta = [torch.randn(p.shape, generator=g, device="cuda") for p in params]
    before = [p.clone() for p in params]
    old = [v.clone() for v in momenta]
    op = m.Muon(params, grads, momenta=momenta, lr=lr, momentum=beta, nesterov=nesterov, weight_decay=decay, scale=scale)
    op.step()
    assert op.device_status() == (0, 0)
    for w0, w, gr, v0, v in zip(before, params, grads, old, momenta):
        v2, u, size, kept = reference_step(w0, gr, v0, lr, beta, nesterov, decay, scale)
        # three roundings, and beta and 1 - beta themselves
        mag = beta * v0.double().abs() + (1.0 - beta) * gr.double().abs()
        assert bool(((v.double() - v2).abs() <= 5 * E24 * mag).all())
        # the direction is taken from the fp32 momentum, whose rounding the steps amplify as
        # any other: the model starts from it rounded the same way
        planes = 2 if w.dtype == torch.float32 else 1
        want = exact(u)
        off = torch.linalg.matrix_norm(modelled(u.float(), planes) - want)
        full = (kept - lr * size * want.view(w.shape)).reshape(want.shape)
        norm = lambda t: torch.linalg.matrix_norm(t.double())
        bound = lr * size * (2.5 * off + 8 * E24 * norm(want)) + (U[w.dtype] + 4 * E24) * (
            norm(full) + norm(kept.reshape(want.shape)) * E24 / U[w.dtype])
        err = norm(w.reshape(want.shape).double() - full)
        assert bool((err <= bound).all()), (err / bound).tolist()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("nesterov,decay,scale", [(True, 0.1, "spectral"), (False, 0.0, "rms"), (True, 0.0, "none")])
def test_step_of_a_layer(m, dt, nesterov, decay, scale):
    """gate, up and down of one layer share their launches; a router and 2-D matrices
    have their own."""
    shapes = [(4, 72, 136), (4, 72, 136), (4, 136, 72), (10, 136), (200, 33), (3, 140, 264), (3, 264, 140), (131, 131)]
    params = [torch.randn(s, device="cuda").to(dt) for s in shapes]
    grads = [torch.randn(s, device="cuda").to(dt) for s in shapes]
    check_step(m, params, grads, nesterov, decay, scale)


def test_step_of_mixed_types_and_odd_addresses(m):
    """Gradients of the other type; views at odd element offsets."""
    N = 200000
    flat = torch.randn(N, device="cuda")
    half = torch.randn(N, device="cuda").bfloat16()
    params = [flat[1:1 + 40 * 60].view(40, 60), half[3:3 + 2 * 31 * 17].view(2, 31, 17), flat[5001:5001 + 17 * 31].view(17, 31),
              half[20001:20001 + 130 * 151].view(130, 151), flat[60003:60003 + 150 * 133].view(150, 133)]
    grads = [half[7001:7001 + 2400].view(40, 60), flat[9003:9003 + 1054].view(2, 31, 17), half[12001:12001 + 527].view(17, 31),
             flat[100001:100001 + 130 * 151].view(130, 151), half[150003:150003 + 150 * 133].view(150, 133)]
    guard = flat.clone(), half.clone()
    check_step(m, params, grads, True, 0.01, "spectral")
    for now, was, used in ((flat, guard[0], [(1, 2401), (5001, 5528), (60003, 60003 + 150 * 133)]),
                           (half, guard[1], [(3, 1057), (20001, 20001 + 130 * 151)])):
        keep = torch.ones(N, dtype=torch.bool, device="cuda")
        for lo, hi in used:
            keep[lo:hi] = False
        assert torch.equal(now[keep], was[keep])


def test_long_list_of_small_matrices(m):
    """More tensors of one size than a launch carries."""
    params = [torch.randn((1 + i % 3, 12, 20) if i % 2 else (1 + i % 3, 20, 12), device="cuda") for i in range(41)]
    grads = [torch.randn(p.shape, device="cuda") for p in params]
    check_step(m, params, grads, True, 0.0, "spectral")


def test_step_in_a_graph_and_on_a_stream(m):
    w = torch.randn((3, 130, 90), device="cuda").bfloat16()
    g = torch.randn((3, 130, 90), device="cuda").bfloat16()
    one, two, three = w.clone(), w.clone(), w.clone()
    a, b, c = (m.Muon([t], [g], lr=0.1) for t in (one, two, three))
    a.step()
    a.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.step(stream=side)
    b.step(stream=side)
    side.synchronize()
    assert torch.equal(one, two) and torch.equal(a.momenta[0], b.momenta[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(one, three) and torch.equal(a.momenta[0], c.momenta[0])


def test_a_list_that_meets_itself_is_refused(m):
    z = lambda *n: torch.zeros(n, device="cuda", dtype=torch.float32)
    w, g, v = z(4, 160, 160), z(4, 160, 160), z(4, 160, 160)
    with pytest.raises(ValueError, match="no two"):
        m.Muon([w, w], [g, g.clone()], [v, v.clone()])
    with pytest.raises(ValueError, match="no two"):
        m.Muon([w, w[3:]], [g, g[:1]], [v, z(1, 160, 160)])
    with pytest.raises(ValueError, match="no two"):
        m.Muon([w[:2], w[2:]], [g[:2], g[2:]], [v[:2], v[1:3]])
    with pytest.raises(ValueError, match="gradient"):
        m.Muon([w], [w], [v])
    with pytest.raises(ValueError, match="gradient"):
        m.Muon([w[:1], w[1:2]], [g[:1], w[1:2]], [v[:1], v[1:2]])
    # side by side, and one gradient for two
    m.Muon([w[:2], w[2:]], [g[:2], g[:2]], [v[:2], v[2:]]).step()


@pytest.mark.parametrize("shape", [(5, 160, 400), (5, 400, 160)])
def test_bad_wide_matrices_stay_alone(m, shape):
    u = draw(shape, torch.bfloat16, seed=9)
    op = m.Orthogonalize(*shape)
    clean = op.forward(u)
    u[1] = 0.0
    u[2, 5, 5] = float("nan")
    u[4, 6, 7] = float("-inf")
    got = op.forward(u)
    assert float(got[1].abs().max()) == 0.0
    assert bool(got[2].isnan().all()) and bool(got[4].isnan().all())
    assert torch.equal(got[0], clean[0]) and torch.equal(got[3], clean[3])


# few matrices with a long side: A's sums in pieces
LONG = [(1, 129, 4100), (2, 300, 2500), (1, 700, 5000), (6, 260, 1030), (1, 9000, 140), (37, 130, 1100), (1, 1030, 1100)]


@pytest.mark.parametrize("shape", LONG)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_long_sides(m, shape, dt):
    u = draw(shape, dt, seed=sum(shape))
    op = m.Orthogonalize(*shape, dtype=dt)
    got = op.forward(u)
    close(got, u)
    assert torch.equal(op.forward(u), got)
    # the workspace of a call of another batch in between
    two = m.Orthogonalize(*shape, dtype=dt)
    two.forward(-u)
    assert torch.equal(two.forward(u), got) and two.device_status() == (0, 0)


def test_long_sides_in_a_list(m):
    """More tensors than a launch carries: rounds of different sizes."""
    gs = [draw((1, 200, 1200) if i % 2 else (1, 1200, 200), torch.float32, seed=i) for i in range(19)]
    ps = [torch.zeros_like(g) for g in gs]
    m.Muon(ps, gs, lr=0.1, momentum=0.0, nesterov=False, scale="none").step()
    for p, g in zip(ps, gs):
        close(p / -0.1, g)   # of zeros: two more roundings of the direction
