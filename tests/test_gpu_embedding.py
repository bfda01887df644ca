"""Token embedding and its gradient against the definition in float64.

Bounds (derived): a lookup is one fp32 product and one rounding to the type (u: bf16
2^-8, fp32 2^-24), so u + 2^-23 relative to each element.  A gradient row is an fp32
sum of n terms in some order, at most n + 2 roundings of 2^-24 of sum |term|, the
product with the scale, the addition of dw_add and one rounding:
u |exact| + (n + 6) 2^-24 (|scale| sum |dy| + |dw_add|).  The scales here are exact in
fp32.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E24 = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    return m


def draw_ids(T, V, kind, g):
    if kind == "one":
        return torch.full((T,), V // 2, dtype=torch.int32, device="cuda")
    if kind == "few":
        return torch.randint(0, min(V, 5), (T,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "skewed":
        u = torch.rand((T,), generator=g, device="cuda", dtype=torch.float64)
        return ((V + 1.0) ** u - 1.0).long().clamp_(0, V - 1).int()
    return torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)


def reference(ids, dy, V, scale, pad, add):
    """Gradient in float64, the sum of the terms' magnitudes, tokens of each row."""
    at = ids.long()
    ok = (at >= 0) & (at < V) & (at != (-1 if pad is None else pad))
    d = dy.double()[ok] * scale
    zero = torch.zeros((V, dy.shape[1]), dtype=torch.float64, device="cuda")
    dw = zero.clone().index_add_(0, at[ok], d)
    mag = zero.index_add_(0, at[ok], d.abs())
    n = torch.bincount(at[ok], minlength=V).double()[:, None]
    if add is not None:
        dw += add.double()
        mag += add.double().abs()
    return dw, mag, n


def close_rows(got, ids, dy, V, scale, pad, add):
    dw, mag, n = reference(ids, dy, V, scale, pad, add)
    bound = U[got.dtype] * dw.abs() + (n + 6) * E24 * mag
    err = (got.double() - dw).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


CASES = [  # T, V, H, ids, dtype, scale, padding, add
    (1, 1, 8, "any", "bf16", 1.0, None, None), (1, 50257, 2048, "any", "bf16", 0.5, None, "out"),
    (7, 3, 264, "few", "f32", 2.0, 0, None), (33, 17, 1000, "any", "bf16", 1.0, None, "out"),
    (257, 511, 72, "skewed", "f32", 64.0, None, "in"), (2048, 512, 512, "any", "bf16", 1.0, 5, None),
    (4096, 131072, 264, "skewed", "bf16", 1.0, None, "in"), (8192, 100, 2048, "skewed", "bf16", 1.0, 0, "out"),
    (8192, 7, 8, "one", "f32", 1.0, None, None), (8193, 32001, 520, "skewed", "bf16", 0.25, None, None),
    (20011, 300001, 64, "any", "f32", 1.0, 3, "in"), (30000, 4000, 256, "one", "bf16", 1.0, None, "out"),
    (100003, 1023, 40, "skewed", "f32", 1.0, 0, "out"), (600001, 513, 16, "few", "bf16", 1.0, None, None)]


@pytest.mark.parametrize("T,V,H,kind,dtype,scale,pad,add", CASES)
def test_lookup_and_gradient(m, T, V, H, kind, dtype, scale, pad, add):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(T + V)
    ids = draw_ids(T, V, kind, g)
    w = torch.randn((V, H), generator=g, device="cuda").to(dt)
    dy = torch.randn((T, H), generator=g, device="cuda").to(dt)
    op = m.TokenEmbedding(T, H, V, dtype=dt, scale=scale, padding_idx=pad)
    y = op.forward(w, ids)
    want = w.double()[ids.long()] * scale
    assert bool(((y.double() - want).abs() <= (U[dt] + 2 * E24) * want.abs()).all())
    base = torch.randn((V, H), generator=g, device="cuda").to(dt) if add else None
    out = torch.full((V, H), float("nan"), device="cuda", dtype=dt)
    if add == "in":
        out = base.clone()
        got = op.backward(ids, dy, dw_add=out, dw=out)
    else:
        got = op.backward(ids, dy, dw_add=base, dw=out)
    close_rows(got, ids, dy, V, scale, pad, base)
    if add:
        untouched = torch.ones(V, dtype=torch.bool, device="cuda")
        untouched[ids[ids != (-1 if pad is None else pad)].long()] = False
        assert torch.equal(got[untouched], base[untouched])
    again = base.clone() if add == "in" else torch.empty_like(out)
    op.backward(ids, dy, dw_add=again if add == "in" else base, dw=again)
    assert torch.equal(again, got)      # the same bits in every run
    assert op.device_status() == (0, 0)


@pytest.mark.parametrize("T", [5, 300, 9000])
def test_ids_out_of_range(m, T):
    """A zero row, no gradient, a bit of the status; neighbours are as they would be."""
    V, H = 40, 72
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = draw_ids(T, V, "any", g)
    ids[0], ids[T // 2], ids[-1] = -1, V, 2 ** 31 - 1
    w = torch.randn((V, H), generator=g, device="cuda").bfloat16()
    dy = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    op = m.TokenEmbedding(T, H, V)
    y = op.forward(w, ids)
    assert op.device_status() == (m.MOE_ERR_TOKEN, 32)
    bad = (ids < 0) | (ids >= V)
    assert float(y[bad].abs().max()) == 0.0 and torch.equal(y[~bad], w[ids[~bad].long()])
    dy[bad] = float("nan")
    close_rows(op.backward(ids, dy), ids, dy.nan_to_num(), V, 1.0, None, None)
    assert op.device_status() == (m.MOE_ERR_TOKEN, 32) and op.device_status() == (0, 0)


def test_no_tokens(m):
    op = m.TokenEmbedding(0, 64, 100)
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    none = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.randn((100, 64), device="cuda").bfloat16()
    assert op.forward(w, ids).shape == (0, 64)
    assert float(op.backward(ids, none, dw=torch.ones_like(w)).abs().max()) == 0.0
    assert torch.equal(op.backward(ids, none, dw_add=w), w)


def test_table_in_a_wider_buffer(m):
    wide = torch.randn((50, 96), device="cuda").bfloat16()
    ids = torch.randint(0, 50, (70,), device="cuda", dtype=torch.int32)
    y = m.TokenEmbedding(70, 64, 50).forward(wide[:, 8:72], ids)
    assert torch.equal(y, wide[ids.long(), 8:72])


def test_padding_rows_may_hold_anything(m):
    """The rows of dy at padding tokens are not read into a sum."""
    T, V, H = 500, 30, 128
    ids = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    dy = torch.randn((T, H), device="cuda")
    clean = m.TokenEmbedding(T, H, V, dtype=torch.float32, padding_idx=7).backward(ids, dy)
    dy[ids == 7] = float("inf")
    dirty = m.TokenEmbedding(T, H, V, dtype=torch.float32, padding_idx=7).backward(ids, dy)
    assert torch.equal(clean, dirty) and float(dirty[7].abs().max()) == 0.0


def test_rows_past_31_bits(m):
    """Table and gradient elements beyond 2^31."""
    V, H = 70000, 32768
    w = torch.zeros((V, H), device="cuda", dtype=torch.bfloat16)
    w[-1] = 3.0
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda", dtype=torch.int32)
    op = m.TokenEmbedding(3, H, V)
    y = op.forward(w, ids)
    assert float(y[0].min()) == 3.0 and float(y[1].abs().max()) == 0.0
    dw = op.backward(ids, torch.ones((3, H), device="cuda", dtype=torch.bfloat16), dw=w)
    assert float(dw[-1].min()) == 2.0 and float(dw[0].min()) == 1.0 and float(dw[1:-1].abs().max()) == 0.0


def test_one_workspace_for_many_shapes_a_stream_and_a_graph(m):
    big = m.TokenEmbedding(9000, 256, 5000)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((5000, 256), generator=g, device="cuda").bfloat16()
    ids = draw_ids(9000, 5000, "skewed", g)
    dy = torch.randn((9000, 256), generator=g, device="cuda").bfloat16()
    want = big.backward(ids, dy).clone()
    small = m.TokenEmbedding(100, 256, 5000)
    small.ws = big.ws
    part = small.backward(ids[:100], dy[:100]).clone()
    close_rows(part, ids[:100], dy[:100], 5000, 1.0, None, None)
    assert torch.equal(big.backward(ids, dy), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = big.backward(ids, dy, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    y, dw = torch.empty((9000, 256), device="cuda", dtype=torch.bfloat16), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        big.forward(w, ids, y=y)
        big.backward(ids, dy, dw=dw)
    ids.copy_(ids.flip(0))
    dy.copy_(dy.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, w[ids.long()])
    close_rows(dw, ids, dy, 5000, 1.0, None, None)


FEW = [  # around the number of tokens that need no sorted list
    (64, 5, 264, "few", "bf16", 1.0, None, "in"), (64, 1, 2048, "one", "f32", 0.5, None, None),
    (63, 1000, 7168, "skewed", "bf16", 1.0, 0, "out"), (65, 1000, 520, "skewed", "bf16", 1.0, 0, "out"),
    (40, 33, 8, "any", "f32", 3.0, 7, "in"), (64, 70001, 40, "any", "bf16", 1.0, None, None),
    (2, 2, 16, "one", "f32", 1.0, None, "out"), (33, 9, 1288, "one", "bf16", 1.0, 4, "out")]


@pytest.mark.parametrize("T,V,H,kind,dtype,scale,pad,add", FEW)
def test_few_tokens(m, T, V, H, kind, dtype, scale, pad, add):
    test_lookup_and_gradient(m, T, V, H, kind, dtype, scale, pad, add)


@pytest.mark.parametrize("T", [5, 64, 65])
def test_few_tokens_out_of_range(m, T):
    test_ids_out_of_range(m, T)
