"""Cases and plain forms of the FP8 products and the quantizer that makes their operands, of
SwiGLU with an 8-bit checkpoint, and of the router's balance loss.

Families:
  rows     bf16 or fp32 -> FP8 rows: E4M3 codes and one power-of-two scale for 128 values of a row
  blocks   weights -> FP8 with one scale for a tile of 128 x 128, and the transposed copy
  linear   C[M, N] = A[M, K] . B[N, K]^T, both in FP8, B's scales for each row or for each tile
  experts  the same product per expert over ragged shards of tokens
  swiglu   y = silu(gate) * up as FP8 rows, and a checkpoint of [gate | up] in FP8 rows ("fwd");
           its gradient from the checkpoint, in the gradient's type or as FP8 rows ("bwd")
  balance  the balance loss of a router with counts and shard offsets ("fwd"), its gradient ("bwd")

FP8 rows are E4M3 [rows, cols] with power-of-two fp32 scales [rows, cols/128]; tiles have scales
[ceil(rows/128), cols/128].  The codes come back as float8 values.
"""
import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch of three tokens into FP8 rows: launch latency
        {"name": "rows_token", "op": "rows", "rows": 3, "cols": 7168, "dt": "bf16"},
        # one layer's weights after an optimizer step: four experts' fp32 masters, with the copy that the input gradient reads
        {"name": "blocks_weights", "op": "blocks", "e": 4, "rows": 4096, "cols": 7168, "dt": "f32", "copy": True},
        # one token through a 7168 -> 4096 projection while serving: weight bytes and launch latency
        {"name": "linear_token", "op": "linear", "m": 1, "n": 4096, "k": 7168, "tile": True, "row": False, "out": "bf16"},
        # a small odd batch into an odd head width, scales for each row on both sides, fp32 logits
        {"name": "linear_odd", "op": "linear", "m": 77, "n": 1001, "k": 2176, "tile": False, "row": True, "out": "f32"},
        # a square weight against a long prefill or training batch: compute bound
        {"name": "linear_large", "op": "linear", "m": 8192, "n": 8192, "k": 8192, "tile": True, "row": False, "out": "bf16"},
        # decode: 64 routed tokens over one GPU's 32 experts, most with a few tokens, some with none
        {"name": "experts_decode", "op": "experts", "t": 64, "e": 32, "n": 2048, "k": 7168, "tile": True, "row": False, "out": "bf16"},
        # training: Zipf shards of an odd token count through the fused gate and up projection
        {"name": "experts_up", "op": "experts", "t": 16383, "e": 32, "n": 4096, "k": 7168, "tile": True, "row": True, "out": "bf16"},
        # decode through the activation, nothing kept: launch latency
        {"name": "swiglu_token", "op": "swiglu", "dir": "fwd", "rows": 8, "f": 2048, "dt": "bf16", "keep": False, "fmt": "fp8"},
        # a training batch of routed tokens (8192 tokens, 8 experts each) through the activation, checkpoint kept
        {"name": "swiglu_train", "op": "swiglu", "dir": "fwd", "rows": 65536, "f": 2048, "dt": "bf16", "keep": True, "fmt": "fp8"},
        # the gradient of an odd batch in bf16, as the quantizers of the weight gradient take it
        {"name": "swiglu_grad_odd", "op": "swiglu", "dir": "bwd", "rows": 20011, "f": 2176, "dt": "bf16", "keep": True, "fmt": "same"},
        # a training batch's router: 256 experts, 8 a token, padding at the sequences' ends
        {"name": "balance_train", "op": "balance", "dir": "fwd", "t": 65536, "e": 256, "k": 8, "dt": "f32", "mask": True},
        # the gradient of a small router with an odd number of experts
        {"name": "balance_grad_odd", "op": "balance", "dir": "bwd", "t": 4097, "e": 61, "k": 4, "dt": "bf16", "mask": True},
    ]


def _log(rng, lo, hi):
    return int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))


def draw(rng):
    op = rng.choice(["rows", "blocks", "linear", "linear", "experts", "experts", "swiglu", "swiglu", "balance", "balance"])
    dt, tile, row = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7, rng.random() < 0.4
    if op == "rows":
        return {"op": op, "rows": _log(rng, 1, 16384), "cols": 128 * _log(rng, 2, 64), "dt": dt}
    if op == "blocks":
        copy = rng.random() < 0.7
        rows = 128 * _log(rng, 2, 32) if copy else _log(rng, 100, 4096)
        return {"op": op, "e": _log(rng, 1, 4), "rows": rows, "cols": 128 * _log(rng, 2, 56), "dt": dt, "copy": copy}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 256, 8192), "k": 128 * _log(rng, 2, 64), "tile": tile, "row": row, "out": dt}
    if op == "experts":
        return {"op": op, "t": _log(rng, 16, 16384), "e": _log(rng, 2, 32), "n": _log(rng, 512, 4096), "k": 128 * _log(rng, 4, 56), "tile": tile, "row": row, "out": dt}
    if op == "swiglu":
        way, fmt = rng.choice(["fwd", "bwd"]), rng.choice(["fp8", "same"])
        return {"op": op, "dir": way, "rows": _log(rng, 1, 65536), "f": 128 * _log(rng, 2, 16), "dt": dt, "keep": way == "bwd" or rng.random() < 0.7, "fmt": "fp8" if way == "fwd" else fmt}
    e = _log(rng, 8, 256)
    return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "t": _log(rng, 1, 65536), "e": e, "k": rng.randint(1, min(8, e)), "dt": dt, "mask": rng.random() < 0.5}


def _counts(case):
    """Tokens of each expert: Zipf-like shares, the same for every seed (their order is not)."""
    p = np.arange(1, case["e"] + 1, dtype=np.float64) ** -1.1
    return np.random.default_rng(7).multinomial(case["t"], p / p.sum())


def work(case):
    op, o = case["op"], 4 if case.get("out", case.get("dt")) == "f32" else 2
    if op == "rows":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (o + 1) + n // 32, "flops": 5 * n}
    if op == "blocks":
        n = case["e"] * case["rows"] * case["cols"]
        s = 4 * case["e"] * -(-case["rows"] // 128) * (case["cols"] // 128)
        return {"bytes": n * (o + 1) + s + (n + s if case["copy"] else 0), "flops": 5 * n}
    if op == "swiglu":
        r, f = case["rows"], case["f"]
        if case["dir"] == "fwd":
            return {"bytes": r * f * (2 * o + 1 + (2 if case["keep"] else 0)) + r * f // 32 * (3 if case["keep"] else 1), "flops": 15 * r * f}
        out = 2 * r * f + r * f // 16 if case["fmt"] == "fp8" else 2 * r * f * o
        return {"bytes": 2 * r * f + r * f // 16 + r * f * o + out, "flops": 20 * r * f}
    if op == "balance":
        t, e = case["t"], case["e"]
        m = t if case["mask"] else 0
        if case["dir"] == "fwd":
            return {"bytes": t * (e * o + 8 * case["k"]) + m + 16 * e, "flops": 5 * t * e}
        return {"bytes": 2 * t * e * o + m + 4 * e, "flops": 8 * t * e}
    n, k = case["n"], case["k"]
    m, e = (case["m"], 1) if op == "linear" else (case["t"], int((_counts(case) > 0).sum()))
    s = 4 * (k // 128) * (m + e * (-(-n // 128) if case["tile"] else n))
    return {"bytes": m * k + e * n * k + s + m * n * o + (4 * m if case["row"] else 0), "flops": 2 * m * n * k}


# ------------------------------------------------------------------ inputs
def _pow2_scale(amax):
    """The least power of two that brings amax to 448 or less (448 = 0.875 * 2^9), at least 2^-126 for amax > 0, and 2^-127 for 0."""
    f, e = torch.frexp(amax)
    k = torch.where(f <= 0.875, e - 9, e - 8).clamp(-126, 127)
    k = torch.where(amax > 0, k, torch.full_like(k, -127))
    return torch.ldexp(torch.ones_like(amax), k)


def _fp8_rows(x):
    """fp32 [rows, cols] -> E4M3 [rows, cols], scales [rows, cols/128]."""
    b = x.view(x.shape[0], -1, 128)
    s = _pow2_scale(b.abs().amax(-1))
    return (b / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(x.shape), s


def _fp8_tiles(x):
    """fp32 [rows, cols] -> E4M3 [rows, cols], scales [ceil(rows/128), cols/128]."""
    r, c = x.shape
    pad = torch.nn.functional.pad(x, (0, 0, 0, -r % 128)) if r % 128 else x
    b = pad.view(-1, 128, c // 128, 128)
    s = _pow2_scale(b.abs().amax((1, 3)))
    return (b / s[:, None, :, None]).view(-1, c)[:r].to(torch.float8_e4m3fn), s


def _acts(g, dev, rows, cols):
    """Activations: Gaussian rows of differing size with a few hot channels."""
    x = torch.randn(rows, cols, generator=g, device=dev)
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device=dev))
    hot = torch.randint(0, cols, (max(1, cols // 900),), generator=g, device=dev)
    x[:, hot] *= 30.0
    return x


def _weight(g, dev, case):
    w = torch.randn(case["n"], case["k"], generator=g, device=dev) * (1.0 / case["k"]) ** 0.5
    q, s = _fp8_tiles(w) if case["tile"] else _fp8_rows(w)
    return q.view(torch.uint8), s


def _logits(g, dev, case):
    """Router logits with experts that differ in popularity, their top k, and which tokens count."""
    t, e = case["t"], case["e"]
    x = 1.5 * torch.randn(t, e, generator=g, device=dev) + torch.randn(e, generator=g, device=dev)
    x = x.to(_DT[case["dt"]])
    top = torch.topk(x.float(), case["k"], dim=-1).indices
    mask = torch.rand(t, generator=g, device=dev) < 0.9 if case["mask"] else None
    return x, top, mask


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    st, op = {"case": case}, case["op"]
    if op == "rows":
        st["x"] = _acts(g, dev, case["rows"], case["cols"]).to(_DT[case["dt"]])
    elif op == "blocks":
        w = torch.randn(case["e"], case["rows"], case["cols"], generator=g, device=dev)
        w *= (1.0 / case["cols"]) ** 0.5 * torch.exp(torch.randn(case["e"], case["rows"], 1, generator=g, device=dev))
        st["x"] = w.to(_DT[case["dt"]])
    elif op in ("linear", "experts"):
        rows = case["m"] if op == "linear" else case["t"]
        q, st["as"] = _fp8_rows(_acts(g, dev, rows, case["k"]))
        st["a"] = q.view(torch.uint8)
        st["row"] = torch.exp(0.5 * torch.randn(rows, generator=g, device=dev)) if case["row"] else None
        if op == "linear":
            st["b"], st["bs"] = _weight(g, dev, case)
        else:
            w = [_weight(g, dev, case) for _ in range(case["e"])]
            st["b"], st["bs"] = torch.stack([x[0] for x in w]), torch.stack([x[1] for x in w])
            n = _counts(case)[torch.randperm(case["e"], generator=g, device=dev).cpu().numpy()]
            off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
            st["off"], st["at"] = torch.from_numpy(off).to(dev), [int(x) for x in off]
    elif op == "swiglu":
        x = _acts(g, dev, case["rows"], 2 * case["f"])
        if case["dir"] == "fwd":
            st["x"] = x.to(_DT[case["dt"]])
        else:
            q, st["cs"] = _fp8_rows(x)
            st["c"] = q.view(torch.uint8)
            st["dy"] = (1e-3 * torch.randn(case["rows"], case["f"], generator=g, device=dev)).to(_DT[case["dt"]])
    else:
        st["x"], st["top"], st["mask"] = _logits(g, dev, case)
        if case["dir"] == "bwd":
            n = case["t"] if st["mask"] is None else max(1, int(st["mask"].sum()))
            one = torch.ones(case["t"], device=dev) if st["mask"] is None else st["mask"].float()
            c = torch.zeros(case["e"], device=dev).index_add_(0, st["top"].reshape(-1), one.repeat_interleave(case["k"]))
            st["v"] = c * (0.01 * case["e"] / (case["k"] * float(n) ** 2))
            st["dl"] = 0.5 + torch.rand(1, generator=g, device=dev)
            st["add"] = (1e-6 * torch.randn(case["t"], case["e"], generator=g, device=dev)).to(_DT[case["dt"]])
    return st


# -------------------------------------------------------------- the passes
def _values(q, s):
    return (q.view(torch.float8_e4m3fn).float().view(*s.shape, 128) * s.unsqueeze(-1)).view(q.shape)


def _b_values(q, s, tile):
    return _values(q, s.repeat_interleave(128, 0)[:q.shape[0]] if tile else s)


def _rows_out(q, s):
    """FP8 rows whose values went through exp: codes, and the scales in the 8-bit type for powers of two
    where there are many (of some ten million maxima one lies between two scales by its last place)."""
    return {"q": q.view(torch.float8_e4m3fn), "scales": s if s.numel() <= 4096 else s.to(torch.float8_e8m0fnu)}


def _run_plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "rows":
        q, s = _fp8_rows(st["x"].float())
        return {"q": q, "scales": s}
    if op == "blocks":
        x = st["x"].float()
        e, r, c = x.shape
        if r % 128:   # every matrix begins with a tile of its own
            x = torch.nn.functional.pad(x, (0, 0, 0, -r % 128))
        q, s = _fp8_tiles(x.reshape(-1, c))
        q, s = q.view(e, -1, c)[:, :r].contiguous(), s.view(e, -1, c // 128)
        if not case["copy"]:
            return {"q": q, "scales": s}
        return {"q": q, "scales": s, "qt": q.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn), "scales_t": s.transpose(1, 2).contiguous()}
    if op in ("linear", "experts"):
        x, at = _values(st["a"], st["as"]), st.get("at")
        if op == "linear":
            c = x @ _b_values(st["b"], st["bs"], case["tile"]).t()
        else:
            c = torch.cat([x[at[i]:at[i + 1]] @ _b_values(st["b"][i], st["bs"][i], case["tile"]).t()
                           for i in range(case["e"]) if at[i] < at[i + 1]])
        return (c if st["row"] is None else c * st["row"].unsqueeze(-1)).to(_DT[case["out"]])
    if op == "swiglu":
        f = case["f"]
        if case["dir"] == "fwd":
            x = st["x"].float()
            g, u = x[:, :f], x[:, f:]
            out = _rows_out(*_fp8_rows(g / (1.0 + torch.exp(-g)) * u))
            if not case["keep"]:
                return out
            c, cs = _fp8_rows(x)
            return {**out, "kept": c, "kept_scales": cs}
        x, dy = _values(st["c"], st["cs"]), st["dy"].float()
        g, u = x[:, :f], x[:, f:]
        sg = 1.0 / (1.0 + torch.exp(-g))
        dx = torch.cat([dy * u * sg * (1.0 + g * (1.0 - sg)), dy * g * sg], -1)
        return _rows_out(*_fp8_rows(dx)) if case["fmt"] == "fp8" else dx.to(_DT[case["dt"]])
    x, e, k = st["x"].float(), case["e"], case["k"]
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    m = None if st["mask"] is None else st["mask"].unsqueeze(-1)
    if case["dir"] == "bwd":
        d = st["dl"] * p * (st["v"] - (p * st["v"]).sum(-1, keepdim=True))
        return ((d if m is None else d * m) + st["add"].float()).to(_DT[case["dt"]])
    one = torch.ones_like(st["top"]) if m is None else m.expand_as(st["top"]).long()
    c = torch.zeros(e, dtype=torch.int64, device=x.device).index_add_(0, st["top"].reshape(-1), one.reshape(-1))
    n = torch.full((), float(case["t"]), dtype=torch.float64, device=x.device) if m is None else m.sum().double()
    n = n.clamp(min=1)
    v = 0.01 * e * c.double() / (k * n * n)
    s = (p if m is None else p * m).sum(0, dtype=torch.float64)
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=x.device), torch.cumsum(c, 0)])
    return {"loss": (v * s).sum().float().reshape(1), "counts": c.int(), "offsets": off, "v": v.float()}


def _run_own(st):
    import block_scaled_fp4_amd as fp4
    case, op = st["case"], st["case"]["op"]
    f8 = torch.float8_e4m3fn
    if op == "rows":
        q, s = fp4.fp8_quantize(st["x"])
        return {"q": q.view(f8), "scales": s}
    if op == "blocks":
        q, s, qt, t = fp4.fp8_quantize_blocks(st["x"], transposed=case["copy"])
        out = {"q": q.view(f8), "scales": s}
        return {**out, "qt": qt.view(f8), "scales_t": t} if case["copy"] else out
    if op == "linear":
        return fp4.fp8_matmul(st["a"], st["as"], st["b"], st["bs"], a_row_scale=st["row"], out_dtype=_DT[case["out"]])
    if op == "experts":
        return fp4.fp8_matmul_grouped(st["a"], st["as"], st["b"], st["bs"], st["off"], a_row_scale=st["row"], out_dtype=_DT[case["out"]])
    if op == "swiglu":
        if case["dir"] == "fwd":
            q, s, c, cs = fp4.swiglu_quantize(st["x"], fmt="fp8", checkpoint=case["keep"])
            out = _rows_out(q, s)
            return {**out, "kept": c.view(f8), "kept_scales": cs} if case["keep"] else out
        if case["fmt"] == "fp8":
            _, q, s = fp4.swiglu_backward(st["dy"], st["c"], st["cs"], fmt="fp8")
            return _rows_out(q, s)
        return fp4.swiglu_backward(st["dy"], st["c"], st["cs"])[0]
    if case["dir"] == "bwd":
        return fp4.router_balance_backward(st["x"], st["v"], st["dl"], mask=st["mask"], add=st["add"])
    loss, counts, off, v = fp4.router_balance(st["x"], st["top"], coef=0.01, mask=st["mask"])
    return {"loss": loss, "counts": counts, "offsets": off, "v": v}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------ in 64 bits
def _exact_e4m3(q):
    b = q.long()
    e, f = (b >> 3) & 15, (b & 7).double() / 8
    mag = torch.where(e > 0, (1.0 + f) * torch.pow(2.0, (e - 7).double()), f * 2.0 ** -6)
    return torch.where(b >= 128, -mag, mag)


def _exact_scaled(y, rows):
    """Blocks of `rows` by 128 values over their scales, not rounded, and the scales."""
    r, c = y.shape
    b = y.view(r // rows, rows, c // 128, 128)
    top = b.abs().amax((1, 3))
    s = torch.pow(2.0, torch.where(top > 0, torch.ceil(torch.log2(top / 448.0)).clamp(min=-126), -127.0))
    return (b / s[:, None, :, None]).view(r, c), s


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rows":
        q, s = _exact_scaled(st["x"].double(), 1)
        return {"q": q, "scales": s}
    if op == "blocks":
        e, r, c = st["x"].shape
        q, s = [], []
        for i in range(e):
            full = torch.zeros(-(-r // 128) * 128, c, dtype=torch.float64, device=st["x"].device)
            full[:r] = st["x"][i]
            a, b = _exact_scaled(full, 128)
            q.append(a[:r])
            s.append(b)
        q, s = torch.stack(q), torch.stack(s)
        out = {"q": q, "scales": s}
        return {**out, "qt": q.permute(0, 2, 1), "scales_t": s.permute(0, 2, 1)} if case["copy"] else out
    if op in ("linear", "experts"):
        k, n = case["k"], case["n"]
        a = _exact_e4m3(st["a"]) * st["as"].double().repeat_interleave(128, 1)
        if st["row"] is not None:
            a *= st["row"].double()[:, None]
        row = torch.arange(n, device=a.device) // (128 if case["tile"] else 1)
        weight = lambda q, s: _exact_e4m3(q) * s.double()[row].repeat_interleave(128, 1)  # noqa: E731
        if op == "linear":
            return torch.mm(a, weight(st["b"], st["bs"]).t())
        c = torch.zeros(case["t"], n, dtype=torch.float64, device=a.device)
        for i, (lo, hi) in enumerate(zip(st["at"], st["at"][1:])):
            if hi > lo:
                c[lo:hi] = torch.mm(a[lo:hi], weight(st["b"][i], st["bs"][i]).t())
        return c
    if op == "swiglu":
        f = case["f"]
        if case["dir"] == "fwd":
            x = st["x"].double()
            q, s = _exact_scaled(x[:, :f] * torch.sigmoid(x[:, :f]) * x[:, f:], 1)
            if not case["keep"]:
                return {"q": q, "scales": s}
            c, cs = _exact_scaled(x, 1)
            return {"q": q, "scales": s, "kept": c, "kept_scales": cs}
        x = _exact_e4m3(st["c"]) * st["cs"].double().repeat_interleave(128, 1)
        g, u, dy = x[:, :f], x[:, f:], st["dy"].double()
        h = torch.tanh(g / 2)
        dx = torch.cat([dy * u * (0.5 * (1 + h) + g * (1 - h * h) / 4), dy * g * 0.5 * (1 + h)], 1)
        if case["fmt"] != "fp8":
            return dx
        q, s = _exact_scaled(dx, 1)
        return {"q": q, "scales": s}
    x, e, t = st["x"].double(), case["e"], case["t"]
    keep = torch.ones(t, dtype=torch.float64, device=x.device) if st["mask"] is None else st["mask"].double()
    p = torch.softmax(x, -1)
    if case["dir"] == "bwd":
        v = st["v"].double()
        return st["dl"].double() * p * (v - torch.mv(p, v)[:, None]) * keep[:, None] + st["add"].double()
    n = max(1.0, float(keep.sum()))
    c = torch.bincount(st["top"].reshape(-1), weights=keep.repeat_interleave(case["k"]), minlength=e)
    mean = torch.mv(p.t(), keep) / n
    share = c / (case["k"] * n)
    return {"loss": (0.01 * e * torch.dot(share, mean)).reshape(1), "counts": None, "offsets": None, "v": 0.01 * e * share / n}
