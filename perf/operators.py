"""Measured cases of the 8-bit projection operators.

A backbone layer with 8-bit projections runs: the residual's addition and RMSNorm with
e4m3 output, the block-scaled product (SiLU to bf16, or plain), attention, the GLN gate with
e4m3 output, the block-scaled product with the residual.  Weights and gradients enter through
the quantiser; training returns through the norm's backward pass.

Quantised form everywhere: a group is 128 columns of one row (activations) or a block of
128 x 128 (weights), the last ones ragged; with m = max(|v|, 2^-100) over the group,
scale = m / 448 and q = e4m3(v * (448 / m)), rounded to nearest even.

``own`` False: plain torch forms in fp32.  True: the framework's entry points.
"""
import math
import random

import torch

own = False

F8 = torch.float8_e4m3fn
GROUP = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2, None: 0}
EPS_RMS = 1e-6
EPS_GLN = 1e-5


def listed():
    return [
        # one newly arrived candidate of the 512-wide backbone: pure latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "dim": 512, "x": "f32", "delta": "bf16"},
        # the 64-user batch of the 768-wide backbone: fp32 residual stream, bf16 layer output
        {"name": "norm_batch768", "op": "norm", "rows": 57023, "dim": 768, "x": "f32", "delta": "bf16"},
        # training step of the 32-user batch, 512 wide: fp32 stream, fp32 gradient from the product
        {"name": "norm_bwd_pair512", "op": "norm_bwd", "rows": 25959, "dim": 512, "x": "f32", "dy": "f32", "dres": "f32"},
        # a wide bf16 stream with a ragged number of rows and the gradient of its residual branch
        {"name": "norm_bwd_wide", "op": "norm_bwd", "rows": 8191, "dim": 4096, "x": "bf16", "dy": "bf16", "dres": "bf16"},
        # Target layer of the 32-user batch: T rows only
        {"name": "gate_target_pair", "op": "gate", "users": 32, "target": True, "hq": 8, "hkv": 2, "head_dim": 64, "gln": True},
        # Full layer of the 64-user batch at the 768-wide head shape: all rows
        {"name": "gate_full_768", "op": "gate", "users": 64, "target": False, "hq": 3, "hkv": 1, "head_dim": 256, "gln": True},
        # gradient of a layer's output before its product, odd rows and columns
        {"name": "quant_rows_odd", "op": "quant", "rows": 12345, "cols": 1000, "x": "bf16", "block_rows": 1},
        # a large weight at load time, or every step while it is trained
        {"name": "quant_weight", "op": "quant", "rows": 8192, "cols": 8192, "x": "f32", "block_rows": 128},
        # one candidate through a wide projection: the weight is read once, nothing else counts
        {"name": "gemm_one_token", "op": "gemm", "m": 1, "n": 8192, "k": 4096, "out": "bf16", "act": "silu", "residual": None},
        # output projection of T rows into the fp32 residual stream, nothing a multiple of a tile
        {"name": "gemm_residual_odd", "op": "gemm", "m": 4911, "n": 1000, "k": 1000, "out": "f32", "act": None, "residual": "f32"},
        # U, Q, K, V projection of the 64-user batch, 512 wide
        {"name": "gemm_uqkv_512", "op": "gemm", "m": 53133, "n": 1280, "k": 512, "out": "bf16", "act": "silu", "residual": None},
        # bound by the tensor pipe
        {"name": "gemm_square", "op": "gemm", "m": 8192, "n": 8192, "k": 8192, "out": "bf16", "act": None, "residual": None},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = [(2, 1, 32), (8, 2, 64), (4, 1, 128), (8, 1, 32), (3, 1, 256), (5, 5, 64), (4, 2, 32)]


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gate", "quant", "gemm", "gemm"])
    kind = lambda: rng.choice(["f32", "bf16"])
    if op == "norm":
        dim = _log(rng, 1, 16384)
        rows = _log(rng, 1, min(65536, 57023 * 768 // dim))
        return {"op": op, "rows": rows, "dim": dim, "x": kind(), "delta": rng.choice([None, "f32", "bf16"])}
    if op == "norm_bwd":
        dim = _log(rng, 1, 16384)
        rows = _log(rng, 1, min(65536, 8191 * 4096 // dim))
        return {"op": op, "rows": rows, "dim": dim, "x": kind(), "dy": kind(), "dres": rng.choice([None, "f32", "bf16"])}
    if op == "gate":
        hq, hkv, dh = rng.choice(HEADS)
        return {"op": op, "users": _log(rng, 1, 64), "target": rng.random() < 0.5, "hq": hq, "hkv": hkv, "head_dim": dh,
                "gln": rng.random() < 0.75}
    if op == "quant":
        cols = _log(rng, 1, 16384)
        return {"op": op, "rows": _log(rng, 1, min(65536, 8192 * 8192 // cols)), "cols": cols, "x": kind(),
                "block_rows": rng.choice([1, 128])}
    k = _log(rng, 1, 8192)
    n = _log(rng, 1, 8192)
    m = _log(rng, 1, 65536)
    while m * n * k > 2 ** 37 or m * max(n, k) > 2 ** 28:
        m = (m + 1) // 2
    out = kind()
    return {"op": op, "m": m, "n": n, "k": k, "out": out, "act": rng.choice([None, "silu"]), "residual": rng.choice([None, out])}


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------- inputs

def _padded(rows, cols, dtype, dev="cuda"):
    """A [rows, cols] view whose rows start on 16-byte boundaries, as the product reads them."""
    step = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty(rows, _cdiv(cols, step) * step, dtype=dtype, device=dev)[:, :cols]


def _outputs(rows, cols, rows_per_scale=1):
    return (_padded(rows, cols, F8),
            torch.empty(_cdiv(rows, rows_per_scale), _cdiv(cols, GROUP), dtype=torch.float32, device="cuda"))


def _lengths(users):
    """H, R and T lengths of the users of a batch: uniform in [256, 1024], [32, 256] and [16, 128]."""
    rng = random.Random(users)
    return [[rng.randint(lo, hi) for _ in range(users)] for lo, hi in ((256, 1024), (32, 256), (16, 128))]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, dim = case["rows"], case["dim"]
        # rows of different size, a few columns that stand out
        x = (randn(rows, dim) * torch.exp(0.5 * randn(rows, 1)) * torch.exp(0.3 * randn(dim))).to(TYPES[case["x"]])
        w = 1.0 + 0.2 * randn(dim)
        if op == "norm":
            delta = None if case["delta"] is None else (0.5 * randn(rows, dim)).to(TYPES[case["delta"]])
            q, s = _outputs(rows, dim)
            return {"op": op, "x": x, "delta": delta, "w": w, "q": q, "s": s,
                    "x_out": None if delta is None else torch.empty_like(x),
                    "rstd": torch.empty(rows, dtype=torch.float32, device="cuda")}
        dy = randn(rows, dim).to(TYPES[case["dy"]])
        dres = None if case["dres"] is None else randn(rows, dim).to(TYPES[case["dres"]])
        rstd = torch.rsqrt(x.float().square().mean(1) + EPS_RMS)
        state = {"op": op, "x": x, "w": w, "rstd": rstd, "dy": dy, "dres": dres, "dx": torch.empty_like(x),
                 "dw": torch.empty(dim, dtype=torch.float32, device="cuda")}
        if own:
            import hybrid_masked_attention_b200 as M
            state["ws"] = torch.empty(M.rmsnorm_bwd_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")
        return state
    if op == "gate":
        B, D = case["users"], case["hq"] * case["head_dim"]
        lh, lr, lt = lens = torch.tensor(_lengths(B), dtype=torch.int32, device="cuda")
        lens = lens.t()
        kinds = torch.arange(3, device="cuda").repeat(B).repeat_interleave(lens.reshape(-1).long())
        if case["target"]:
            kinds = kinds[kinds == 2]
        rows = kinds.numel()
        a, u = 0.3 * randn(rows, D), randn(rows, D).bfloat16()
        gamma = 1.0 + 0.2 * randn(3, D) if case["gln"] else None
        beta = 0.1 * randn(3, D) if case["gln"] else None
        q, s = _outputs(rows, D)
        state = {"op": op, "a": a, "u": u, "gamma": gamma, "beta": beta, "kinds": kinds, "q": q, "s": s,
                 "stats": torch.empty(rows, 2, dtype=torch.float32, device="cuda") if case["gln"] else None,
                 "target": case["target"]}
        if own:
            import hybrid_masked_attention_b200 as M
            total, R, T = int(lens.sum()), int(lr.sum()), int(lt.sum())
            state["cfg"] = M.Config(batch=B, total_tokens=total, total_r=R, total_t=T, hq=case["hq"], hkv=case["hkv"],
                                    head_dim=case["head_dim"])
            state["meta"] = M.alloc_meta(state["cfg"])
            M.pack(state["cfg"], lh, lr, lt, torch.zeros(R, dtype=torch.int64, device="cuda"),
                   torch.zeros(T, dtype=torch.int64, device="cuda"), state["meta"])
        return state
    if op == "quant":
        x = (randn(case["rows"], case["cols"]) * torch.exp(randn(case["rows"], 1))).to(TYPES[case["x"]])
        q, s = _outputs(case["rows"], case["cols"], case["block_rows"])
        return {"op": op, "x": x, "block_rows": case["block_rows"], "q": q, "s": s}
    m, n, k = case["m"], case["n"], case["k"]
    a, a_scale = _outputs(m, k)
    b, b_scale = _outputs(n, k, GROUP)
    for to, scale, v, per in ((a, a_scale, randn(m, k) * torch.exp(0.5 * randn(m, 1)), 1),
                              (b, b_scale, randn(n, k) * (1.0 / math.sqrt(k)), GROUP)):
        q, s = _quantised(v, per)
        to.copy_(q)
        scale.copy_(s)
    out = _padded(m, n, TYPES[case["out"]])
    res = None
    if case["residual"] is not None:
        res = _padded(m, n, TYPES[case["residual"]])
        res.copy_(randn(m, n))
    return {"op": op, "a": a, "a_scale": a_scale, "b": b, "b_scale": b_scale, "out": out, "act": case["act"], "res": res,
            "status": torch.zeros(1, dtype=torch.int32, device="cuda")}


# ------------------------------------------------------------------------- one pass

def _quantised(v, rows_per_scale):
    """(q, scale) of an fp32 matrix, one scale for each rows_per_scale x 128 block."""
    R, C = v.shape
    pr, pc = _cdiv(R, rows_per_scale) * rows_per_scale, _cdiv(C, GROUP) * GROUP
    t = torch.nn.functional.pad(v, (0, pc - C, 0, pr - R)).view(pr // rows_per_scale, rows_per_scale, pc // GROUP, GROUP)
    m = t.abs().amax(dim=(1, 3), keepdim=True).clamp_min(2.0 ** -100)
    q = (t * (448.0 / m)).view(pr, pc)[:R, :C].to(F8)
    return q, (m / 448.0).view(pr // rows_per_scale, pc // GROUP)


def _spread(scale, rows, cols, rows_per_scale):
    return scale.repeat_interleave(rows_per_scale, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]


def run(state):
    op = state["op"]
    if own:
        import hybrid_masked_attention_b200 as M
        if op == "norm":
            M.add_rmsnorm_fp8(state["x"], state["delta"], state["w"], state["x_out"], state["q"], state["s"], state["rstd"], EPS_RMS)
            return {"x_out": state["x_out"], "q": state["q"], "scale": state["s"], "rstd": state["rstd"]}
        if op == "norm_bwd":
            M.rmsnorm_bwd(state["x"], state["w"], state["rstd"], state["dy"], state["dres"], state["dx"], state["dw"], state["ws"])
            return {"dx": state["dx"], "dw": state["dw"]}
        if op == "gate":
            M.gate_fwd_fp8(state["cfg"], state["meta"], state["target"], state["a"], state["u"], state["gamma"], state["beta"],
                           state["q"], state["s"], state["stats"])
            return {"q": state["q"], "scale": state["s"], "stats": state["stats"]}
        if op == "quant":
            M.fp8_quant(state["x"], state["q"], state["s"], state["block_rows"])
            return {"q": state["q"], "scale": state["s"]}
        M.fp8_gemm(state["a"], state["a_scale"], state["b"], state["b_scale"], state["out"], state["status"], state["act"], state["res"])
        return {"out": state["out"]}
    if op == "norm":
        x, delta = state["x"], state["delta"]
        h = x.float() if delta is None else x.float() + delta.float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS_RMS)
        q, s = _quantised(h * rstd[:, None] * state["w"], 1)
        return {"x_out": None if delta is None else h.to(x.dtype), "q": q, "scale": s, "rstd": rstd}
    if op == "norm_bwd":
        x, dy, r = state["x"].float(), state["dy"].float(), state["rstd"][:, None]
        xh, gw = x * r, dy * state["w"]
        dx = r * (gw - xh * (gw * xh).mean(1, keepdim=True))
        if state["dres"] is not None:
            dx = dx + state["dres"].float()
        return {"dx": dx.to(state["x"].dtype), "dw": (dy * xh).sum(0)}
    if op == "gate":
        a, u = state["a"], state["u"].float()
        if state["gamma"] is None:
            q, s = _quantised(a * u, 1)
            return {"q": q, "scale": s, "stats": None}
        mean = a.mean(1, keepdim=True)
        c = a - mean
        rstd = torch.rsqrt(c.square().mean(1, keepdim=True) + EPS_GLN)
        q, s = _quantised((c * rstd * state["gamma"][state["kinds"]] + state["beta"][state["kinds"]]) * u, 1)
        return {"q": q, "scale": s, "stats": torch.cat([mean, rstd], 1)}
    if op == "quant":
        q, s = _quantised(state["x"].float(), state["block_rows"])
        return {"q": q, "scale": s}
    a, b = state["a"], state["b"]
    c = (a.float() * _spread(state["a_scale"], a.shape[0], a.shape[1], 1)) @ \
        (b.float() * _spread(state["b_scale"], b.shape[0], b.shape[1], GROUP)).t()
    if state["act"] == "silu":
        c = c * torch.sigmoid(c)
    if state["res"] is not None:
        c = c + state["res"].float()
    return {"out": c.to(state["out"].dtype)}


# ------------------------------------------------------------------------- accounting

def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["dim"]
        per = BYTES[case["x"]] * (1 if case["delta"] is None else 2) + BYTES[case["delta"]] + 1
        return {"bytes": n * per + 4 * case["rows"] * (_cdiv(case["dim"], GROUP) + 1) + 4 * case["dim"], "flops": 7 * n}
    if op == "norm_bwd":
        n = case["rows"] * case["dim"]
        per = 2 * BYTES[case["x"]] + BYTES[case["dy"]] + BYTES[case["dres"]]
        return {"bytes": n * per + 4 * case["rows"] + 8 * case["dim"], "flops": 10 * n}
    if op == "gate":
        h, r, t = (sum(v) for v in _lengths(case["users"]))
        rows = t if case["target"] else h + r + t
        D = case["hq"] * case["head_dim"]
        return {"bytes": rows * (7 * D + 4 * _cdiv(D, GROUP) + (8 if case["gln"] else 0)) + (24 * D if case["gln"] else 0),
                "flops": rows * D * (10 if case["gln"] else 3)}
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (BYTES[case["x"]] + 1) + 4 * _cdiv(case["rows"], case["block_rows"]) * _cdiv(case["cols"], GROUP),
                "flops": 3 * n}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": m * k + n * k + 4 * _cdiv(k, GROUP) * (m + _cdiv(n, GROUP)) + m * n * (BYTES[case["out"]] + BYTES[case["residual"]]),
            "flops": 2 * m * n * k}


# ------------------------------------------------------------------------- in 64 bits

def _exact_quant(v, br):
    """The quantised values before their rounding, and the scales, block by block of the definition."""
    R, C = v.shape
    row = torch.arange(R, device=v.device) // br
    col = torch.arange(C, device=v.device) // GROUP
    blocks = torch.full((_cdiv(R, br) * _cdiv(C, GROUP),), 2.0 ** -100, dtype=torch.float64, device=v.device)
    at = row[:, None] * _cdiv(C, GROUP) + col[None, :]
    blocks.scatter_reduce_(0, at.reshape(-1), v.abs().reshape(-1), "amax")
    return v * 448.0 / blocks[at], (blocks / 448.0).view(_cdiv(R, br), -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    d = lambda t: None if t is None else t.double()
    if op == "norm":
        h = d(st["x"]) if st["delta"] is None else d(st["x"]) + d(st["delta"])
        r = 1.0 / torch.sqrt((h * h).sum(1) / h.shape[1] + EPS_RMS)
        q, s = _exact_quant(torch.einsum("ij,i,j->ij", h, r, d(st["w"])), 1)
        return {"x_out": None if st["delta"] is None else h, "q": q, "scale": s, "rstd": r}
    if op == "norm_bwd":
        x, dy, r = d(st["x"]), d(st["dy"]), d(st["rstd"])
        g = dy * d(st["w"])
        c = torch.einsum("ij,ij->i", g, x) * r ** 3 / x.shape[1]
        dx = r[:, None] * g - c[:, None] * x
        if st["dres"] is not None:
            dx = dx + d(st["dres"])
        return {"dx": dx, "dw": torch.einsum("ij,ij,i->j", dy, x, r)}
    if op == "gate":
        a, u = d(st["a"]), d(st["u"])
        if st["gamma"] is None:
            q, s = _exact_quant(a * u, 1)
            return {"q": q, "scale": s, "stats": None}
        mean = a.sum(1) / a.shape[1]
        rstd = 1.0 / torch.sqrt(((a - mean[:, None]) ** 2).sum(1) / a.shape[1] + EPS_GLN)
        one = torch.nn.functional.one_hot(st["kinds"], 3).double()
        z = (a - mean[:, None]) * rstd[:, None]
        q, s = _exact_quant((z * (one @ d(st["gamma"])) + one @ d(st["beta"])) * u, 1)
        return {"q": q, "scale": s, "stats": torch.stack([mean, rstd], 1)}
    if op == "quant":
        q, s = _exact_quant(d(st["x"]), st["block_rows"])
        return {"q": q, "scale": s}
    a, b, sa, sb = d(st["a"]), d(st["b"]), d(st["a_scale"]), d(st["b_scale"])
    ka = torch.arange(a.shape[1], device=a.device) // GROUP
    nb = torch.arange(b.shape[0], device=b.device) // GROUP
    c = (a * sa[:, ka]) @ (b * sb[nb][:, ka]).t()
    if st["act"] == "silu":
        c = c / (1.0 + torch.exp(-c))
    if st["res"] is not None:
        c = c + d(st["res"])
    return {"out": c}
