"""What the Python binding of the training operators refuses before the library is
called: no GPU needed."""
import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    from mixture_experts_ffn_04_gb300 import build
    build.build()
    m.lib()
    return m


def ce_args(m, T=64, H=256, V=1000, dtype=torch.bfloat16):
    s = m.MoECeShape()
    s.tokens, s.hidden, s.vocab, s.dtype = T, H, V, m._dtype_code(dtype)
    s.reduction, s.ignore_index = m.MOE_CE_MEAN, -100
    return s, dict(x=torch.zeros(T, H, dtype=dtype), w=torch.zeros(V, H, dtype=dtype),
                   t=torch.zeros(T, dtype=torch.int32), lse=torch.zeros(T), stats=torch.zeros(T, 4),
                   total=torch.zeros(1), dx=torch.zeros(T, H, dtype=dtype), dw=torch.zeros(V, H, dtype=dtype),
                   ws=torch.zeros(16, dtype=torch.uint8))


def ce_forward(m, s, a):
    m.moe_linear_ce_forward(s, a["x"], a["w"], a["t"], None, a["lse"], a["stats"], a["total"], a["ws"], stream=0)


def ce_backward(m, s, a):
    m.moe_linear_ce_backward(s, a["x"], a["w"], a["t"], a["stats"], None, a["dx"], a["dw"], a["ws"], stream=0)


@pytest.mark.parametrize("call", [ce_forward, ce_backward])
@pytest.mark.parametrize("name", ["x", "w"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_share_memory_are_refused(m, call, name, dtype):
    """A broadcast row has the stride 0, which the C shape reads as "dense"; rows that
    overlap are no matrix of the ABI either."""
    s, a = ce_args(m, dtype=dtype)
    n, H = a[name].shape
    for bad in (a[name][:1].expand(n, H), torch.zeros(n * 8 + H, dtype=dtype).as_strided((n, H), (8, 1))):
        b = dict(a)
        b[name] = bad
        with pytest.raises(ValueError, match="rows of %s" % name):
            call(m, s, b)


@pytest.mark.parametrize("name", ["x", "w"])
def test_one_row_has_any_stride(m, name):
    """The stride of a single row means nothing: it is not looked at."""
    s, a = ce_args(m, T=1, V=1)
    H = a[name].shape[1]
    for stride in (0, 8, 10 * H):
        b = dict(a)
        b[name] = torch.zeros(16 * H, dtype=a[name].dtype).as_strided((1, H), (stride, 1))
        assert m._rows(b[name], 1, H, torch.bfloat16, name)[1] == H
