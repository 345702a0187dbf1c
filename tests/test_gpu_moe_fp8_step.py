"""The FP8 operators together: examples/moe_fp8_train_step.py against the same step in
64 bits on unquantized weights, captured graphs, other streams, and sizes past 32
bits.

Bounds of the example: E4M3 rounds Gaussian values by 2.7% (relative RMS), so a product
of two rounded operands is off by 4%.  `out` holds h unrounded beside a chain of two
products and three roundings of rows (below 8%); dx holds dout unrounded beside them
and two products back (below 10%); the norm's weight and the router sum such terms
(below 15%, a few percent each); the weights' gradients are products of two MXFP4
roundings, to nearest by 11% and stochastic by 16%, of rows that were already off by 5%
(together 20%, below 30%).  The loss takes logits off by 4% of their spread of
about 1 into probabilities (below 5%)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import moe_ref as M
import ops_ref as R
from gpu_util import dev_f32, dev_i64, dev_u8, need_gpu
from test_gpu_graphs import _replay_check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.mark.parametrize("tokens,hidden,ffn,experts,masked", [
    (300, 512, 256, 8, False), (1, 256, 128, 4, False), (1000, 1024, 384, 40, True), (2500, 512, 256, 3, True)])
def test_train_step(tokens, hidden, ffn, experts, masked):
    need_gpu()
    spec = importlib.util.spec_from_file_location("moe_fp8_train_step", os.path.join(ROOT, "examples", "moe_fp8_train_step.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    off_by = ex.main(tokens, hidden, ffn, experts, masked)
    for name, most in (("out", 0.08), ("loss", 0.05), ("dx", 0.10), ("dgamma", 0.15), ("drouter", 0.15), ("dw1", 0.30), ("dw2", 0.30)):
        assert off_by[name] < most, off_by


def tensors(seed=0):
    """Inputs of every operator, at sizes that reach each kind of kernel."""
    m = need_gpu()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    x = rand(1100, 512).to(BF)
    q, s = m.fp8_quantize(x)
    w = rand(3, 700, 512)
    wq, ws, _, _ = m.fp8_quantize_blocks(w)
    logits = rand(1100, 40)
    return m, x, q, s, w, wq, ws, logits, torch.topk(logits, 2).indices, dev_i64(np.array([0, 400, 400, 1100]))


def calls():
    """{name: (call() -> outputs, call(outputs), outputs as given)}; every call has its
    outputs passed in, for graphs."""
    m, x, q, s, w, wq, ws, logits, top, off = tensors()
    mask = torch.arange(1100, device="cuda") % 7 != 0
    c = {}
    o = m.fp8_quantize(x)
    c["rows"] = (lambda o=o: m.fp8_quantize(x, *o), o)
    w2 = w[:, :640].contiguous()
    o = m.fp8_quantize_blocks(w2, True)
    c["blocks"] = (lambda o=o: m.fp8_quantize_blocks(w2, True, *o), o)
    for rows in (1, 40, 130, 1100):
        for dt in (BF, F32):
            o = torch.empty((rows, 700), dtype=dt, device="cuda")
            c[f"linear {rows} {dt}"] = (lambda o=o, rows=rows: m.fp8_matmul(q[:rows], s[:rows], wq[0], ws[0], out=o), (o,))
    for dt in (BF, F32):
        o = torch.empty((1100, 700), dtype=dt, device="cuda")
        c[f"experts {dt}"] = (lambda o=o: m.fp8_matmul_grouped(q, s, wq, ws, off, out=o), (o,))
    o = m.swiglu_quantize(x, "fp8")
    c["swiglu"] = (lambda o=o: m.swiglu_quantize(x, "fp8", True, *o), o)
    dy = x[:, :256].contiguous()
    kept = o[2].clone(), o[3].clone()
    o = (torch.empty_like(x), *m.swiglu_backward(dy, *kept, "mxfp4")[1:])
    c["swiglu gradient"] = (lambda o=o: m.swiglu_backward(dy, *kept, "mxfp4", *o), o)
    for rows in (20, 1100):                                  # one workgroup, and the second launch
        o = m.router_balance(logits[:rows], top[:rows], 0.1, mask[:rows])
        work = torch.empty(m.router_balance_workspace(rows, 40), dtype=U8, device="cuda")
        c[f"balance {rows}"] = (lambda o=o, work=work, rows=rows: m.router_balance(logits[:rows], top[:rows], 0.1, mask[:rows], *o, work), o)
    v, dl = o[3].clone(), torch.ones(1, device="cuda")
    o = torch.empty_like(logits)
    c["balance gradient"] = (lambda o=o: m.router_balance_backward(logits, v, dl, mask, logits, o), (o,))
    return c


def test_captured_and_replayed():
    for name, (call, outs) in calls().items():
        print(name, flush=True)
        call()
        _replay_check(call, [o for o in outs if o is not None])


def test_a_step_in_one_graph():
    """Router, products and activation, forward and back, in one capture, its
    allocations among it."""
    m, x, q, s, w, wq, ws, logits, top, off = tensors(1)
    w1 = w[:, :512].contiguous()

    def step():
        w1q, w1s, w1t, w1ts = m.fp8_quantize_blocks(w1, transposed=True)
        loss, counts, _, v = m.router_balance(logits, top, 0.1)
        u = m.fp8_matmul_grouped(q, s, w1q, w1s, off)
        a, sa, c, sc = m.swiglu_quantize(u)
        dx, _, _ = m.swiglu_backward(a.view(torch.float8_e4m3fn).to(BF), c, sc)
        dq, ds = m.fp8_quantize(dx)
        return loss, counts, a, sa, m.fp8_matmul_grouped(dq, ds, w1t, w1ts, off), m.router_balance_backward(logits, v)
    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(4):
        for t in got:
            t.view(U8).fill_(0x5A)
        torch.randn(1 << 20, device="cuda").sum().item()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(U8), b.view(U8))


@pytest.mark.parametrize("given", ["stream", "handle"])
def test_on_a_delayed_stream(given):
    """stream=: outputs and scratch are allocated there, and the caller's stream may
    read them after a wait, whatever it allocates meanwhile."""
    m, x, q, s, w, wq, ws, logits, top, off = tensors(2)
    c, sc = m.swiglu_quantize(x)[2:]
    dy, v = x[:, :256].contiguous(), torch.rand(40, device="cuda")
    side = torch.cuda.Stream()
    st = side if given == "stream" else side.cuda_stream
    for call in (lambda st: m.fp8_quantize(x, stream=st), lambda st: m.fp8_quantize_blocks(w[:, :640].contiguous(), True, stream=st),
                 lambda st: m.fp8_matmul(q, s, wq[0], ws[0], stream=st), lambda st: m.fp8_matmul_grouped(q, s, wq, ws, off, stream=st),
                 lambda st: m.swiglu_quantize(x, stream=st), lambda st: m.swiglu_backward(dy, c, sc, stream=st),
                 lambda st: m.swiglu_backward(dy, c, sc, "fp8", stream=st), lambda st: m.router_balance(logits, top, stream=st),
                 lambda st: m.router_balance_backward(logits, v, stream=st)):
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got = call(st)
        got = got if isinstance(got, tuple) else (got,)
        junk = [torch.full((t.numel() * t.element_size(),), 0xA5, dtype=U8, device="cuda") for t in got if t is not None for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None) == (b is None)
            assert a is None or torch.equal(a.view(U8), b.view(U8))
        del junk


def test_two_calls_at_once():
    """The same operands on two streams, with outputs and scratch of their own."""
    m, x, q, s, w, wq, ws, logits, top, off = tensors(3)
    sides = [torch.cuda.Stream() for _ in range(2)]
    want = m.router_balance(logits, top), m.fp8_matmul_grouped(q, s, wq, ws, off), m.swiglu_quantize(x)
    torch.cuda.synchronize()
    for _ in range(3):
        got = [(m.router_balance(logits, top, stream=t), m.fp8_matmul_grouped(q, s, wq, ws, off, stream=t), m.swiglu_quantize(x, stream=t))
               for t in sides]
        torch.cuda.synchronize()
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(one[0], want[0])) and torch.equal(one[1], want[1])
            assert all(torch.equal(a, b) for a, b in zip(one[2], want[2]))


def test_offsets_past_32_bits():
    """Operands and outputs over 4 GiB, or 2^32 elements: their last rows."""
    m = need_gpu()
    rng = np.random.default_rng(5)
    T, N, K = 1_200_000, 4096, 128                            # outputs of 4.9e9 elements
    qa, sa = R.random_fp8(rng, 640, K)
    qb, sb = R.random_fp8(rng, N, K)
    a = torch.zeros((T, K), dtype=U8, device="cuda")
    s = torch.ones((T, 1), device="cuda")
    a[-640:], s[-640:] = dev_u8(qa), dev_f32(sa)
    c = m.fp8_matmul(a, s, dev_u8(qb), dev_f32(sb))
    torch.cuda.synchronize()
    want, bound = M.product_bounds(M.values(qa, sa), M.values(qb, sb), None, True)
    R.assert_product(c[-640:].float().cpu().numpy(), want, bound, True)
    assert not c[:1000].any()
    del a, s, c
    E, N, K = 9, 16384, 29184                                 # weights of 4.3 GB
    w = torch.zeros((E, N, K), dtype=U8, device="cuda")
    ws = torch.ones((E, N, K // 128), device="cuda")
    qb, sb = R.random_fp8(rng, 48, K)
    w[-1, -48:], ws[-1, -48:] = dev_u8(qb), dev_f32(sb)
    for rows in (5, 300):
        qa, sa = R.random_fp8(rng, rows, K)
        off = dev_i64(np.array([0] * E + [rows]))
        want, bound = M.product_bounds(M.values(qa, sa), M.values(qb, sb), None, False)
        c = m.fp8_matmul_grouped(dev_u8(qa), dev_f32(sa), w, ws, off, out_dtype=F32)
        torch.cuda.synchronize()
        R.assert_product(c[:, -48:].cpu().numpy(), want, bound, False)
        c = m.fp8_matmul_grouped(dev_u8(qa), dev_f32(sa), w, ws, off)
        torch.cuda.synchronize()
        want, bound = M.product_bounds(M.values(qa, sa), M.values(qb, sb), None, True)
        R.assert_product(c[:, -48:].float().cpu().numpy(), want, bound, True)
    del w, ws, c
    tail = torch.randn((128, 4096), device="cuda").to(BF)
    x = torch.zeros((1_100_032, 4096), dtype=BF, device="cuda")    # 4.5e9 elements
    x[-128:] = tail
    for got, one in ((m.fp8_quantize(x), m.fp8_quantize(tail)), (m.swiglu_quantize(x), m.swiglu_quantize(tail))):
        torch.cuda.synchronize()
        assert all(torch.equal(p[-128:], q) for p, q in zip(got, one))
    c, s = got[2:]
    del got
    one = m.swiglu_backward(tail[:, :2048].contiguous(), c[-128:], s[-128:])[0]
    dx = m.swiglu_backward(x[:, :2048].contiguous(), c, s)[0]
    torch.cuda.synchronize()
    assert torch.equal(dx[-128:], one)
    del dx, c, s
    q, s, qt, st = m.fp8_quantize_blocks(x, transposed=True)
    q1, s1, qt1, st1 = m.fp8_quantize_blocks(tail, transposed=True)
    torch.cuda.synchronize()
    assert torch.equal(q[-128:], q1) and torch.equal(s[-1:], s1)
    assert torch.equal(qt[:, -128:], qt1) and torch.equal(st[:, -1:], st1)
    del q, qt, x
    t = 17_000_000                                            # logits of 4.4e9 elements
    x = torch.zeros((t, 256), dtype=BF, device="cuda")
    x[-1000:] = torch.randn((1000, 256), device="cuda").to(BF)
    idx = torch.randint(0, 256, (t, 1), device="cuda", dtype=torch.int32)
    mask = torch.zeros(t, dtype=torch.bool, device="cuda")
    mask[-1000:] = True
    got, one = m.router_balance(x, idx, mask=mask), m.router_balance(x[-1000:].clone(), idx[-1000:].clone())
    assert torch.equal(got[1], one[1]) and torch.equal(got[2], one[2]) and torch.equal(got[3], one[3])
    assert abs(float(got[0]) - float(one[0])) < 1e-5 * float(one[0])        # fp32 sums in another order
    d, e = m.router_balance_backward(x, got[3], mask=mask), m.router_balance_backward(x[-1000:].clone(), got[3])
    torch.cuda.synchronize()
    assert torch.equal(d[-1000:], e) and not d[:1000].any()
