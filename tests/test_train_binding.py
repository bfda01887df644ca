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


def router_args(m, T=32, H=64, E=8, k=2):
    s = m.MoEShape()
    s.tokens, s.hidden, s.moe_inter, s.topk_shape = T, H, 8, m.moe_topk_pack(E, k)
    s.norm_topk, s.dtype, s.norm_eps = 1, m.MOE_BF16, 1e-6
    x = torch.zeros(T, H, dtype=torch.bfloat16)
    w = torch.zeros(E, H, dtype=torch.bfloat16)
    n = m.moe_router_backward_workspace_bytes(s)
    return s, [x, w, torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k), None, 0.1, 0.1, None,
               torch.zeros_like(x), torch.zeros_like(w), torch.zeros(2), torch.zeros(n, dtype=torch.uint8)]


def test_host_memory_is_refused(m):
    """Addresses of host tensors must not reach a kernel: with a host workspace, and
    with a host tensor beside a workspace on a device."""
    s, a = ce_args(m)
    a["ws"] = torch.zeros(m.moe_linear_ce_workspace_bytes(s), dtype=torch.uint8)
    for call in (ce_forward, ce_backward):
        with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
            call(m, s, a)
    s, r = router_args(m)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        m.moe_router_backward(s, *r, stream=0)
    plan = m.MoEGradPlan()
    plan.tensors, plan.chunks, plan.chunk_elems = 1, 1, 2048
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        m.moe_grad_clip(plan, 1.0, torch.zeros(1), torch.zeros(4096, dtype=torch.uint8), stream=0)
    with pytest.raises(ValueError, match="one CUDA device"):
        m.GradClip([torch.zeros(4)])

    class DeviceBytes:   # what a workspace on a GPU answers
        is_cuda, device = True, torch.device("cuda", 0)

        def get_device(self):
            return 0

    for name in ("x", "w", "dx", "stats"):
        with pytest.raises(ValueError, match="%s is on cpu" % name):
            m._on_device(DeviceBytes(), **{name: torch.zeros(3)})
    m._on_device(DeviceBytes(), dloss=None)


def test_lists_of_gradients_may_be_generators(m):
    """The refusal is that of the tensors (on the host here), not of the list."""
    with pytest.raises(ValueError, match="one CUDA device"):
        m.GradClip(torch.zeros(4) for _ in range(3))
    with pytest.raises(ValueError, match="one CUDA device"):
        m.GradClip((torch.zeros(4) for _ in range(3)), out=(torch.zeros(4) for _ in range(3)))
    with pytest.raises(ValueError, match="empty"):
        m.GradClip(torch.zeros(4) for _ in range(0))


def test_the_current_stream_without_torch_internals(m, monkeypatch):
    """The handle comes from torch's public interface where the shorter way is absent."""
    class Current:
        cuda_stream = 1234
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 5)
    monkeypatch.setattr(m, "_raw_stream", None)
    assert m._stream(None) == 1234
    monkeypatch.setattr(m, "_raw_stream", lambda device: 100 + device)
    assert m._stream(None) == 105
    assert m._stream(17) == 17


def test_a_plan_needs_device_memory(m):
    table = (m.MoEGradTensor * 1)()
    table[0].src, table[0].numel, table[0].src_dtype, table[0].dst_dtype = 256, 100, m.MOE_F32, m.MOE_F32
    ws = torch.zeros(m.moe_grad_clip_workspace_bytes(table) + 256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        m.moe_grad_clip_plan(table, ws, stream=0)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        m.moe_grad_clip_plan(table, None, stream=0)
