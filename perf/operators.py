"""Cases and plain forms of the products over microscaled rows and of the quantising RMS norm.

Four families:
  linear   C[M, N] = A[M, K] . B[N, K]^T, B in MXFP4, A in MXFP4 or in FP8 rows
  experts  the same product per expert over ragged shards of tokens
  wgrad    dW[e] = A_e . B_e^T over each expert's tokens, from FP8 columns with
           scale blocks of 128 tokens
  norm     residual addition, RMS norm and FP8 rows with scales ("fwd"), and
           its gradient ("bwd").  The rows hold h * weight; the norm's factor
           1/rms stays apart as one fp32 per row, which the products take as
           the scale of their output rows

Layouts: MXFP4 rows are [rows, cols/2] bytes (element 2j in the low nibble)
with UE8M0 bytes [rows, cols/32]; FP8 rows are E4M3 [rows, cols] with
power-of-two fp32 scales [rows, cols/128]; FP8 columns are, per expert, a dense
E4M3 [channels, n_e] at byte channels * off[e], with fp32 scales
[channels, ceil(n_e/128)] at element channels * (ceil(off[e]/128) + e).
"""
import numpy as np
import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token through a 7168 -> 4096 projection while serving: weight bytes and launch latency
        {"name": "linear_token", "op": "linear", "m": 1, "n": 4096, "k": 7168, "act": "mxfp4", "row": True, "out": "bf16"},
        # a small odd batch into an odd head width, FP8 activations, fp32 logits
        {"name": "linear_odd", "op": "linear", "m": 77, "n": 1001, "k": 2176, "act": "fp8", "row": True, "out": "f32"},
        # a square weight against a long prefill or training batch: compute bound
        {"name": "linear_large", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "act": "mxfp4", "row": False, "out": "bf16"},
        # decode: 64 routed tokens over one GPU's 32 experts, most with a few tokens, some with none
        {"name": "experts_decode", "op": "experts", "t": 64, "e": 32, "n": 2048, "k": 7168, "act": "mxfp4", "row": True, "out": "bf16"},
        # training or prefill: Zipf shards through the fused gate and up projection
        {"name": "experts_up", "op": "experts", "t": 16384, "e": 32, "n": 4096, "k": 7168, "act": "mxfp4", "row": True, "out": "bf16"},
        # the projection back to the hidden size from FP8 rows: odd token count, odd expert count, fp32 out
        {"name": "experts_down_odd", "op": "experts", "t": 5001, "e": 13, "n": 7168, "k": 2048, "act": "fp8", "row": False, "out": "f32"},
        # a few ragged shards, fp32 gradients
        {"name": "wgrad_odd", "op": "wgrad", "t": 1009, "e": 5, "m": 2048, "n": 1024, "out": "f32"},
        # one GPU's experts in a training step: the gradient of the up projection
        {"name": "wgrad_up", "op": "wgrad", "t": 16384, "e": 16, "m": 4096, "n": 7168, "out": "bf16"},
        # a decode batch of four tokens: launch latency
        {"name": "norm_token", "op": "norm", "dir": "fwd", "rows": 4, "cols": 7168, "dt": "bf16", "res": True},
        # a training batch of hidden size 7168 with its residual stream
        {"name": "norm_train", "op": "norm", "dir": "fwd", "rows": 16384, "cols": 7168, "dt": "bf16", "res": True},
        # an odd number of fp32 rows, with no gradient from the residual branch
        {"name": "norm_grad_odd", "op": "norm", "dir": "bwd", "rows": 333, "cols": 2048, "dt": "f32", "res": False},
        # the gradient of a training batch with the residual branch's gradient added
        {"name": "norm_grad_train", "op": "norm", "dir": "bwd", "rows": 16384, "cols": 7168, "dt": "bf16", "res": True},
    ]


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "experts", "experts", "wgrad", "norm"])
    act, out = rng.choice(["mxfp4", "mxfp4", "fp8"]), rng.choice(["bf16", "bf16", "f32"])
    row = rng.random() < 0.5
    q = 128 if act == "fp8" else 32
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 256, 8192), "k": max(2, _log(rng, 256, 8192) // q) * q, "act": act, "row": row, "out": out}
    if op == "experts":
        return {"op": op, "t": _log(rng, 16, 16384), "e": _log(rng, 2, 32), "n": _log(rng, 512, 4096), "k": max(4, _log(rng, 512, 7168) // q) * q, "act": act, "row": row, "out": out}
    if op == "wgrad":
        return {"op": op, "t": _log(rng, 64, 16384), "e": _log(rng, 1, 16), "m": 128 * _log(rng, 2, 32), "n": 128 * _log(rng, 2, 32), "out": out}
    return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "rows": _log(rng, 1, 16384), "cols": 128 * _log(rng, 4, 64), "dt": out, "res": rng.random() < 0.7}


def _counts(case):
    """Tokens of each expert: Zipf-like shares, the same for every seed (their order is not)."""
    p = np.arange(1, case["e"] + 1, dtype=np.float64) ** -1.1
    return np.random.default_rng(7).multinomial(case["t"], p / p.sum())


def work(case):
    o = 4 if case.get("out", case.get("dt")) == "f32" else 2
    if case["op"] == "norm":
        n, r, c = case["rows"] * case["cols"], case["rows"], case["cols"]
        if case["dir"] == "fwd":
            b = n * (o * (3 if case["res"] else 2) + 1) + n // 32 + 4 * (r + c)
        else:
            b = n * o * (4 if case["res"] else 3) + 4 * r + 8 * c
        return {"bytes": b, "flops": 10 * n}
    if case["op"] == "wgrad":
        t, m, n, e = case["t"], case["m"], case["n"], case["e"]
        blocks = int(sum(-(-x // 128) for x in _counts(case)))
        return {"bytes": (m + n) * (t + 4 * blocks) + 8 * (e + 1) + e * m * n * o, "flops": 2 * t * m * n}
    n, k = case["n"], case["k"]
    m, e = (case["m"], 1) if case["op"] == "linear" else (case["t"], int((_counts(case) > 0).sum()))
    a = m * k // 2 + m * k // 32 if case["act"] == "mxfp4" else m * k + m * k // 32
    return {"bytes": a + e * (n * k // 2 + n * k // 32) + m * n * o + (4 * m if case["row"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ inputs
def _e2m1_code(q):
    """RTN codes of q (ties to the even code, 6 where q is larger)."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=q.device)
    a = q.abs()
    up, down = torch.bucketize(a, edges, right=True), torch.bucketize(a, edges)
    mag = torch.where(up % 2 == 0, up, down)
    return (mag + torch.where(torch.signbit(q), 8, 0)).to(torch.uint8)


def _mx_rows(x):
    """fp32 [rows, cols] -> unpacked codes [rows, cols], UE8M0 bytes [rows, cols/32]."""
    b = x.reshape(x.shape[0], -1, 32)
    _, e = torch.frexp(b.abs().amax(-1))
    byte = (e - 1 - 2 + 127).clamp(0, 254)
    return _e2m1_code(torch.ldexp(b, (127 - byte).unsqueeze(-1))).reshape(x.shape), byte.to(torch.uint8)


def _pack(c):
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _fp8_rows(x):
    """fp32 [rows, cols] -> E4M3 bytes, power-of-two scales [rows, cols/128] (amax / scale <= 448)."""
    b = x.reshape(x.shape[0], -1, 128)
    s = _pow2_scale(b.abs().amax(-1))
    return (b / s.unsqueeze(-1)).to(torch.float8_e4m3fn).reshape(x.shape), s


def _pow2_scale(amax):
    """The least power of two that brings amax to 448 or less (448 = 0.875 * 2^9), at least 2^-126 for amax > 0, and 2^-127 for 0."""
    f, e = torch.frexp(amax)
    k = torch.where(f <= 0.875, e - 9, e - 8).clamp(-126, 127)
    k = torch.where(amax > 0, k, torch.full_like(k, -127))
    return torch.ldexp(torch.ones_like(amax), k)


def _acts(g, dev, rows, cols):
    """Activations: Gaussian rows of differing size with a few hot channels."""
    x = torch.randn(rows, cols, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=dev))
    hot = torch.randint(0, cols, (max(1, cols // 900),), generator=g, device=dev)
    x[:, hot] *= 30.0
    return x


def _operand(g, dev, case, rows, k):
    x = _acts(g, dev, rows, k)
    if case["act"] == "fp8":
        q, s = _fp8_rows(x)
        return q.view(torch.uint8), s
    c, s = _mx_rows(x)
    return _pack(c), s


def _row_scale(g, dev, case, rows):
    return torch.exp(0.5 * torch.randn(rows, generator=g, device=dev)) if case["row"] else None


def _weights(g, dev, n, k):
    c, s = _mx_rows(torch.randn(n, k, generator=g, device=dev) * (1.0 / k) ** 0.5)
    return _pack(c), s


def _offsets(case, g, dev):
    n = _counts(case)[torch.randperm(case["e"], generator=g, device=dev).cpu().numpy()]
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _cols(g, dev, off, ch, size):
    """FP8 columns of MXFP4-rounded rows: per block of 128 tokens and channel, the scale is the largest of its rows'."""
    t, e = int(off[-1]), len(off) - 1
    x = torch.randn(t, ch, generator=g, device=dev) * torch.exp(torch.randn(t, 1, generator=g, device=dev)) * size
    code, byte = _mx_rows(x)
    val = torch.tensor(_E2M1, device=dev)[code.int()]
    q = torch.empty(t * ch, dtype=torch.uint8, device=dev)
    s = torch.zeros(ch * (-(-t // 128) + e), dtype=torch.float32, device=dev)
    for i in range(e):
        a, b = int(off[i]), int(off[i + 1])
        if a == b:
            continue
        nb = -(-(b - a) // 128)
        by = torch.zeros(nb * 128, ch // 32, dtype=torch.int32, device=dev)
        by[:b - a] = byte[a:b].int()
        tgt = by.view(nb, 128, -1).amax(1)
        d = (by - tgt.repeat_interleave(128, 0))[:b - a].repeat_interleave(32, 1)
        q[ch * a:ch * b] = torch.ldexp(val[a:b], d).t().to(torch.float8_e4m3fn).contiguous().view(torch.uint8).view(-1)
        at = ch * (-(-a // 128) + i)
        s[at:at + ch * nb] = torch.ldexp(torch.ones(1, device=dev), tgt - 127).repeat_interleave(32, 1).t().reshape(-1)
    return q, s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "linear":
        st["a"], st["as"] = _operand(g, dev, case, case["m"], case["k"])
        st["b"], st["bs"] = _weights(g, dev, case["n"], case["k"])
        st["row"] = _row_scale(g, dev, case, case["m"])
    elif case["op"] == "experts":
        off = _offsets(case, g, dev)
        st["a"], st["as"] = _operand(g, dev, case, case["t"], case["k"])
        w = [_weights(g, dev, case["n"], case["k"]) for _ in range(case["e"])]
        st["b"], st["bs"] = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
        st["row"] = _row_scale(g, dev, case, case["t"])
        st["off"], st["at"] = torch.from_numpy(off).to(dev), [int(x) for x in off]
    elif case["op"] == "wgrad":
        off = _offsets(case, g, dev)
        st["a"], st["as"] = _cols(g, dev, off, case["m"], 1e-3)
        st["b"], st["bs"] = _cols(g, dev, off, case["n"], 1.0)
        st["off"], st["at"] = torch.from_numpy(off).to(dev), [int(x) for x in off]
    else:
        r, c, dt = case["rows"], case["cols"], _DT[case["dt"]]
        st["w"] = 1.0 + 0.1 * torch.randn(c, generator=g, device=dev)
        x = _acts(g, dev, r, c)
        if case["dir"] == "fwd":
            st["x"] = x.to(dt)
            st["res"] = (2.0 * torch.randn(r, c, generator=g, device=dev)).to(dt) if case["res"] else None
        else:
            st["h"] = x.to(dt)
            st["rstd"] = 1.0 / torch.sqrt(st["h"].float().square().mean(-1) + 1e-6)
            st["dy"] = (1e-3 * torch.randn(r, c, generator=g, device=dev)).to(dt)
            st["dh"] = (1e-3 * torch.randn(r, c, generator=g, device=dev)).to(dt) if case["res"] else None
    return st


# -------------------------------------------------------------- the passes
def _mx_values(p, s):
    """MXFP4 rows as fp32 values."""
    v = torch.tensor(_E2M1, device=p.device)[torch.stack([p & 15, p >> 4], -1).int()]
    return (v.view(*s.shape, 32) * _e8m0(s).unsqueeze(-1)).view(p.shape[0], -1)


def _e8m0(b):
    return torch.ldexp(torch.ones(1, device=b.device), b.int() - 127)


def _a_values(a, s):
    if s.dtype == torch.uint8:
        return _mx_values(a, s)
    return (a.view(torch.float8_e4m3fn).float().view(*s.shape, 128) * s.unsqueeze(-1)).view(a.shape)


def _col_values(q, s, ch, a, b, i):
    """Expert i's columns (tokens a .. b) as fp32 values [ch, b - a]."""
    nb, at = -(-(b - a) // 128), ch * (-(-a // 128) + i)
    x = q[ch * a:ch * b].view(torch.float8_e4m3fn).float().view(ch, b - a)
    return x * s[at:at + ch * nb].view(ch, nb).repeat_interleave(128, 1)[:, :b - a]


def _run_plain(st):
    case = st["case"]
    if case["op"] in ("linear", "experts"):
        x = _a_values(st["a"], st["as"])
        if case["op"] == "linear":
            c = x @ _mx_values(st["b"], st["bs"]).t()
        else:
            at = st["at"]
            c = torch.cat([x[at[i]:at[i + 1]] @ _mx_values(st["b"][i], st["bs"][i]).t()
                           for i in range(case["e"]) if at[i] < at[i + 1]])
        return (c if st["row"] is None else c * st["row"].unsqueeze(-1)).to(_DT[case["out"]])
    if case["op"] == "wgrad":
        m, n, at = case["m"], case["n"], st["at"]
        dw = torch.zeros(case["e"], m, n, dtype=_DT[case["out"]], device=st["a"].device)
        for i in range(case["e"]):
            if at[i] < at[i + 1]:
                dw[i] = (_col_values(st["a"], st["as"], m, at[i], at[i + 1], i)
                         @ _col_values(st["b"], st["bs"], n, at[i], at[i + 1], i).t()).to(dw.dtype)
        return dw
    dt, w = _DT[case["dt"]], st["w"]
    if case["dir"] == "fwd":
        h = st["x"] if st["res"] is None else (st["x"].float() + st["res"].float()).to(dt)
        hf = h.float()
        rstd = 1.0 / torch.sqrt(hf.square().mean(-1) + 1e-6)
        q, s = _fp8_rows(hf * w)
        out = {"q": q, "scales": s, "rstd": rstd}
        return out if st["res"] is None else {**out, "h": h}
    hf, r = st["h"].float(), st["rstd"].unsqueeze(-1)
    dy = st["dy"].float()
    gr = dy * w
    dx = r * (gr - hf * r * r * (gr * hf).mean(-1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return {"dx": dx.to(dt), "dweight": (dy * hf * r).sum(0)}


def _run_own(st):
    import block_scaled_fp4_amd as fp4
    case = st["case"]
    if case["op"] == "linear":
        return fp4.mxfp4_matmul(st["a"], st["as"], st["b"], st["bs"], a_row_scale=st["row"], out_dtype=_DT[case["out"]])
    if case["op"] == "experts":
        return fp4.mxfp4_matmul_grouped(st["a"], st["as"], st["b"], st["bs"], st["off"], a_row_scale=st["row"], out_dtype=_DT[case["out"]])
    if case["op"] == "wgrad":
        return fp4.fp8_matmul_tokblk(st["a"], st["as"], st["b"], st["bs"], st["off"], case["m"], case["n"], out_dtype=_DT[case["out"]])
    if case["dir"] == "fwd":
        q, s, rstd, h = fp4.rmsnorm_quantize(st["x"], st["w"], residual=st["res"], eps=1e-6, fmt="fp8")
        out = {"q": q.view(torch.float8_e4m3fn), "scales": s, "rstd": rstd}
        return out if st["res"] is None else {**out, "h": h}
    dx, dw = fp4.rmsnorm_backward(st["dy"], st["h"], st["w"], st["rstd"], dh=st["dh"])
    return {"dx": dx, "dweight": dw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ in 64 bits
def _exact_mx(p, s):
    """From the fields of the codes: sign, two exponent bits of bias 1, one bit of fraction."""
    c = torch.stack([p & 15, p >> 4], -1).reshape(p.shape[0], -1).long()
    e, f = (c >> 1) & 3, (c & 1).double()
    mag = torch.where(e > 0, (1.0 + f / 2) * torch.pow(2.0, (e - 1).double()), f / 2)
    sc = torch.pow(2.0, s.double() - 127.0).repeat_interleave(32, 1)
    return torch.where(c >= 8, -mag, mag) * sc


def _exact_e4m3(q):
    b = q.long()
    e, f = (b >> 3) & 15, (b & 7).double() / 8
    mag = torch.where(e > 0, (1.0 + f) * torch.pow(2.0, (e - 7).double()), f * 2.0 ** -6)
    return torch.where(b >= 128, -mag, mag)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("linear", "experts"):
        a = _exact_mx(st["a"], st["as"]) if case["act"] == "mxfp4" else _exact_e4m3(st["a"]) * st["as"].double().repeat_interleave(128, 1)
        if st["row"] is not None:
            a *= st["row"].double()[:, None]
        if case["op"] == "linear":
            return torch.mm(a, _exact_mx(st["b"], st["bs"]).t())
        c = torch.zeros(case["t"], case["n"], dtype=torch.float64, device=a.device)
        for i, (lo, hi) in enumerate(zip(st["at"], st["at"][1:])):
            if hi > lo:
                c[lo:hi] = torch.mm(a[lo:hi], _exact_mx(st["b"][i], st["bs"][i]).t())
        return c
    if case["op"] == "wgrad":
        t, m, n = case["t"], case["m"], case["n"]
        dw = torch.zeros(case["e"], m, n, dtype=torch.float64, device=st["a"].device)
        for i, (lo, hi) in enumerate(zip(st["at"], st["at"][1:])):
            if hi > lo:
                side = []
                for q, s, ch in ((st["a"], st["as"], m), (st["b"], st["bs"], n)):
                    x = _exact_e4m3(q[ch * lo:ch * hi]).view(ch, hi - lo)
                    first = ch * ((lo + 127) // 128 + i)
                    blocks = (hi - lo + 127) // 128
                    col = torch.arange(hi - lo, device=x.device) // 128
                    side.append(x * s[first:first + ch * blocks].view(ch, blocks)[:, col].double())
                dw[i] = torch.mm(side[0], side[1].t())
        return dw
    w = st["w"].double()
    if case["dir"] == "fwd":
        h = st["x"].double() + (st["res"].double() if st["res"] is not None else 0.0)
        hr = h.to(_DT[case["dt"]]).double()
        rstd = (hr.pow(2).sum(-1) / case["cols"] + 1e-6).pow(-0.5)
        y = (hr * w).view(case["rows"], -1, 128)
        k = torch.ceil(torch.log2(y.abs().amax(-1) / 448.0))
        out = {"q": (y * torch.pow(2.0, -k)[..., None]).view(hr.shape), "scales": torch.pow(2.0, k), "rstd": rstd}
        return out if st["res"] is None else {**out, "h": h}
    h, r, dy = st["h"].double(), st["rstd"].double()[:, None], st["dy"].double()
    x = h * r
    gr = dy * w
    dx = r * (gr - x * ((gr * x).sum(-1, keepdim=True) / case["cols"]))
    if st["dh"] is not None:
        dx = dx + st["dh"].double()
    return {"dx": dx, "dweight": (dy * x).sum(0)}
