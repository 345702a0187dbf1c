"""The binding's `stream=`: a call on another stream allocates, launches and
frees under that stream, and its new outputs are known to the caller's stream.

Memory that the caching allocator hands out belongs to the stream that is
current at that moment.  Written on another stream it may still be in use on
its own, and scratch dropped at the call's end would be handed out again while
the kernels run.  Here (CPU) the library is a stub, tensors are fake, and the
current stream is a variable: each allocation is logged with it.  On the GPU
the same calls run behind a delayed stream, with the caller's stream taking
and filling blocks of the same sizes meanwhile."""
import ctypes

import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode

import block_scaled_fp4_amd as m

T, H, N, E = 128, 256, 384, 2


def calls(t):
    """{name: call(stream) -> outputs} over tensors made by t(dtype, *shape)."""
    u8, f32, bf, i64 = torch.uint8, torch.float32, torch.bfloat16, torch.int64
    x, y, off = t(bf, T, H), t(bf, T, H), t(i64, E + 1)
    p, s, f = t(u8, T, H // 2), t(u8, T, H // 32), t(f32, T, H // 64)
    w, ws = t(u8, E, N, H // 2), t(u8, E, N, H // 32)
    g, r = t(f32, H), t(f32, T)
    nb = -(-T // 128) + E
    c, cs = t(u8, T * H), t(f32, H * nb)
    return {
        "fp4_quantize": lambda st: m.fp4_quantize(x, "nvfp4", stream=st),
        "fp4_dequantize": lambda st: m.fp4_dequantize(p, s, T, H, "mxfp4", stream=st),
        "fp4quant_encode": lambda st: m.fp4quant_encode(x, 64, stream=st),
        "fp4quant_encode_ex": lambda st: m.fp4quant_encode_ex(x, 64, stream=st),
        "fp4quant_decode": lambda st: m.fp4quant_decode(p, f, f, T, H, 64, stream=st),
        "fp4_errfeedback_qdq": lambda st: m.fp4_errfeedback_qdq(x, stream=st),
        "mxfp4_row_to_fp8_col": lambda st: m.mxfp4_row_to_fp8_col(p, s, off, H, stream=st),
        "mxfp4_row_to_fp8_col_tokblk": lambda st: m.mxfp4_row_to_fp8_col_tokblk(p, s, off, H, stream=st),
        "mxfp4_row_to_fp8_row": lambda st: m.mxfp4_row_to_fp8_row(p, s, H, stream=st),
        "mxfp4_matmul": lambda st: m.mxfp4_matmul(p, s, w[0], ws[0], stream=st),
        "mxfp4_matmul_grouped": lambda st: m.mxfp4_matmul_grouped(p, s, w, ws, off, stream=st),
        "fp8_matmul_tokblk": lambda st: m.fp8_matmul_tokblk(c, cs, c, cs, off, H, H, stream=st),
        "rmsnorm_quantize": lambda st: m.rmsnorm_quantize(x, g, residual=y, stream=st),
        "rmsnorm_backward": lambda st: m.rmsnorm_backward(x, y, g, r, stream=st),
    }


class FakeStream:
    device = torch.device("cuda", 0)

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def fake_gpu(monkeypatch):
    """(log, mode): the log's "new" (current handle of each allocation), "launch"
    (handle of each library call) and "recorded" ({id of tensor: handle})."""
    log = {"new": [], "launch": [], "recorded": {}}
    current = [FakeStream(1)]

    def set_stream(s):
        current[0] = s

    class Stub:
        def __getattr__(self, name):
            def call(*args):
                if name.endswith("_workspace"):
                    return 4096
                log["launch"].append(args[-1])
                return 0
            return call

    class Allocations(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            if "empty" in str(func):
                log["new"].append(current[0].cuda_stream)
            return func(*args, **(kwargs or {}))

    monkeypatch.setattr(m, "_lib", Stub())
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[0])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "set_stream", set_stream)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: current[0].cuda_stream, raising=False)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 4096)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log["recorded"].update({id(t): s.cuda_stream}))
    return log, Allocations


@pytest.mark.parametrize("given", ["stream", "handle", "pointer"])
@pytest.mark.parametrize("name", sorted(calls(lambda dt, *shape: torch.empty(shape, dtype=dt, device="meta"))))
def test_allocations_belong_to_the_launch_stream(fake_gpu, name, given):
    log, allocations = fake_gpu
    st = {"stream": FakeStream(2), "handle": 2, "pointer": ctypes.c_void_p(2)}[given]
    with FakeTensorMode(allow_non_fake_inputs=True):
        call = calls(lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda:0"))[name]
        with allocations():
            out = call(st)
        assert log["new"] and set(log["new"]) == {2}
        assert log["launch"] == [2]
        for t in out if isinstance(out, tuple) else (out,):
            assert log["recorded"].get(id(t)) == 1


def test_without_a_stream_the_current_one_is_used(fake_gpu):
    log, allocations = fake_gpu
    with FakeTensorMode(allow_non_fake_inputs=True):
        for name, call in calls(lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda:0")).items():
            with allocations():
                call(None)
    assert set(log["new"]) == set(log["launch"]) == {1} and not log["recorded"]


def _gpu_inputs(seed):
    """t(dtype, *shape) with plausible contents for each of `calls`' tensors."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def t(dt, *shape):
        if dt == torch.int64:
            return torch.tensor([0, 50, T], device="cuda")
        if dt == torch.uint8:
            return torch.randint(100, 120, shape, generator=g, device="cuda", dtype=dt)
        if dt == torch.float32:                    # powers of two serve as FP8 scales too
            return torch.ones(shape, device="cuda")
        return torch.randn(shape, generator=g, device="cuda").to(dt)
    return t


def test_nothing_to_allocate(fake_gpu):
    """Outputs given: the launch goes to the stream, and nothing else happens."""
    log, allocations = fake_gpu
    with FakeTensorMode(allow_non_fake_inputs=True):
        t = lambda dt, *shape: torch.empty(shape, dtype=dt, device="cuda:0")
        x, q, s, f = t(torch.bfloat16, T, H), t(torch.uint8, T, H // 2), t(torch.uint8, T, H // 32), t(torch.float32, T)
        g, o8, s8, o = t(torch.float32, H), t(torch.uint8, T, H), t(torch.float32, T, 2), t(torch.bfloat16, T, T)
        ws = t(torch.uint8, 4096)
        with allocations():
            m.fp4_quantize(x, "mxfp4", packed=q, scales=s, stream=2)
            m.fp4_dequantize(q, s, T, H, "mxfp4", y=x, stream=FakeStream(2))
            m.mxfp4_row_to_fp8_row(q, s, H, o8, s8, stream=2)
            m.mxfp4_matmul(q, s, q, s, out=o, stream=2)
            m.rmsnorm_quantize(x, g, fmt="mxfp4", q=q, scales=s, row_scale=f, stream=2)
            m.rmsnorm_backward(x, x, g, f, dx=x, dweight=g, workspace=ws, stream=2)
    assert log["launch"] == [2] * 6 and not log["new"] and not log["recorded"]


def test_an_error_leaves_the_current_stream(fake_gpu):
    log, _ = fake_gpu
    with FakeTensorMode(allow_non_fake_inputs=True):
        x = torch.empty((T, H), dtype=torch.bfloat16, device="cuda:0")
        with pytest.raises(ValueError):
            m.rmsnorm_quantize(x, torch.empty(H - 1, device="cuda:0"), stream=2)
        m.rmsnorm_quantize(x, torch.empty(H, device="cuda:0"))
    assert log["launch"] == [1]


@pytest.mark.gpu
@pytest.mark.parametrize("given", ["stream", "handle"])
def test_outputs_and_scratch_hold_on_a_delayed_stream(given):
    """Blocks just freed with work pending on the caller's stream, and blocks
    dropped by a call whose kernels wait, meet nobody else's writes."""
    side = torch.cuda.Stream()
    for name in calls(_gpu_inputs(0)):
        print(name, flush=True)
        call = calls(_gpu_inputs(1))[name]
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = call(side if given == "stream" else side.cuda_stream)
        got = got if isinstance(got, tuple) else (got,)
        sizes = [t.numel() * t.element_size() for t in got if t is not None] + [m.rmsnorm_backward_workspace(T, H)]
        junk = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        if name == "mxfp4_row_to_fp8_col_tokblk":          # slots of scales that no shard uses are not written
            got, want = ((o[0], o[1][:H], o[1][2 * H:]) for o in (got, want))
        for a, b in zip(got, want):
            if a is None:
                assert b is None
                continue
            a, b = (v.view(torch.uint8).cpu().numpy() for v in (a, b))
            np.testing.assert_array_equal(a, b, err_msg=name)
        del junk


@pytest.mark.gpu
def test_null_stream_handle():
    """0 is the default stream, also while another one is current."""
    t = _gpu_inputs(2)
    x, g = t(torch.bfloat16, 64, 256), t(torch.float32, 256)
    want = m.rmsnorm_quantize(x, g)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = m.rmsnorm_quantize(x, g, stream=0)
    torch.cuda.synchronize()
    for a, b in zip(got[:3], want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_side_stream_inside_a_capture():
    """A stream forked inside a capture: its allocations belong to the graph."""
    t, side, g = _gpu_inputs(3), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    x, y, w, r = t(torch.bfloat16, T, H), t(torch.bfloat16, T, H), t(torch.float32, H), t(torch.float32, T)
    want = m.rmsnorm_backward(x, y, w, r)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = m.rmsnorm_backward(x, y, w, r, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        for o in got:
            o.zero_()
        junk = torch.full((1 << 20,), 7.0, device="cuda")
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and float(junk[0]) == 7.0
