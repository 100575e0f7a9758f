"""The 8-bit operators on the GPU against plain 64-bit forms: norm with e4m3 output and its
backward, gate, quantiser, block-scaled product.  Tolerances count roundings (fp8_ref)."""
import pytest
import torch

import fp8_ref as R
import mtfm_synth as syn
from fp8_ref import F8, HALF, U, groups, guards_kept, padded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def rnd(seed, *shape, scale=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def strided(t, extra):
    """t in a buffer with `extra` elements between its rows."""
    base = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), device=t.device).to(t.dtype)
    base[:, :t.shape[1]] = t
    return base[:, :t.shape[1]]


def out8(rows, cols, block_rows=1):
    return padded(rows, cols, F8), padded(-(-rows // block_rows), groups(cols), F32)


# fp32 sums of squares: a lane adds at most 32 terms, then 5 shuffles and up to 16 warps
SUM_TERMS = 32 + 5 + 16


# ------------------------------------------------------------------------------- norm

@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 512), (3, 127), (5, 128), (9, 129), (17, 640), (8, 768), (33, 1000),
                                      (7, 1024), (4, 2049), (3, 4096), (5, 4100), (2, 9001), (2, 16384), (300, 512)])
@pytest.mark.parametrize("xt,dt", [(F32, None), (F32, BF16), (F32, F32), (BF16, None), (BF16, BF16), (BF16, F32)])
def test_add_rmsnorm(rows, dim, xt, dt, cuda_ok):
    import hybrid_masked_attention_b200 as M
    x = rnd(1, rows, dim, dtype=xt) * torch.exp(rnd(2, rows, 1)).to(xt)
    d = None if dt is None else rnd(3, rows, dim, scale=0.5, dtype=dt)
    w = 1 + 0.3 * rnd(4, dim)
    x_out = None if d is None else padded(rows, dim, xt)
    q, s = out8(rows, dim)
    rstd = torch.full((rows,), -1.0, device="cuda")
    M.add_rmsnorm_fp8(x, d, w, x_out, q, s, rstd)
    h, r, v = R.add_rmsnorm(x, d, w, 1e-6)
    # h: one rounding; mean of squares: the sum's and two more; square root halves it; then 1 / sqrt
    rel_r = (SUM_TERMS + 4) / 2 * U + 3 * U
    assert ((rstd.double() - r).abs() <= rel_r * r).all()
    R.check_quant(q, s, v, v.abs() * (rel_r + 4 * U))
    if d is not None:
        assert ((x_out.double() - h).abs() <= HALF[xt] * h.abs() + 2 * U * h.abs()).all()
        assert guards_kept(x_out)
    assert guards_kept(q) and guards_kept(s)


def test_add_rmsnorm_strides_and_in_place(cuda_ok):
    """Rows at odd pitches and offsets give the same bits as packed rows; x_out may be x."""
    import hybrid_masked_attention_b200 as M
    for xt, dt in ((F32, BF16), (BF16, F32)):
        rows, dim = 37, 520
        x, d, w = rnd(5, rows, dim, dtype=xt), rnd(6, rows, dim, dtype=dt), 1 + 0.1 * rnd(7, dim)
        q0, s0 = out8(rows, dim)
        x0 = torch.empty_like(x)
        M.add_rmsnorm_fp8(x, d, w, x0, q0, s0)
        for ex in (1, 3, 8):
            xs, ds = strided(x, ex), strided(d, ex + 2)
            buf = torch.zeros(rows * (dim + ex) + 1, dtype=torch.uint8, device="cuda").view(F8)
            q = buf[1:].view(rows, dim + ex)[:, :dim]     # an odd base too
            s = torch.zeros(rows, groups(dim) + ex, device="cuda")[:, :groups(dim)]
            M.add_rmsnorm_fp8(xs, ds, w, xs, q, s)
            # the lane-to-column assignment differs, and so may the last bit of a row's sum
            assert ((s - s0).abs() <= 64 * U * s0).all()
            flips = (q.float() != q0.float()).float().mean()
            assert flips < 0.01
            assert torch.equal(xs, x0)


def test_norm_extreme_rows(cuda_ok):
    """Rows of zeros, of tiny and huge values; NaN and infinity stay in their own row."""
    import hybrid_masked_attention_b200 as M
    dim = 300
    x = rnd(8, 8, dim)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e15
    x[4, 7] = float("nan")
    x[5, 200] = float("inf")
    w = torch.ones(dim, device="cuda")
    q, s = out8(8, dim)
    rstd = torch.empty(8, device="cuda")
    M.add_rmsnorm_fp8(x, None, w, None, q, s, rstd)
    assert (q[0].float() == 0).all() and (s[0].double() - R.FLOOR / 448).abs().max() <= 4 * U * R.FLOOR
    assert torch.isnan(rstd[4]) and torch.isnan(q[4].float()).all()
    assert rstd[5] == 0 and torch.isnan(q[5, 200].float())
    ok = [0, 1, 2, 3, 6, 7]
    _, r, v = R.add_rmsnorm(x[ok], None, w, 1e-6)
    rel = (SUM_TERMS + 4) / 2 * U + 7 * U
    assert ((rstd[ok].double() - r).abs() <= rel * r).all()
    R.check_quant(q[ok], s[ok], v, v.abs() * rel)


def test_norm_without_rows(cuda_ok):
    import hybrid_masked_attention_b200 as M
    x = torch.empty(0, 64, device="cuda")
    M.add_rmsnorm_fp8(x, None, torch.ones(64, device="cuda"), None, *out8(0, 64))
    dw = torch.full((64,), 3.0, device="cuda")
    ws = torch.empty(M.rmsnorm_bwd_workspace_bytes(0, 64), dtype=torch.uint8, device="cuda")
    M.rmsnorm_bwd(x, torch.ones(64, device="cuda"), torch.empty(0, device="cuda"), x, None, x, dw, ws)
    assert (dw == 0).all()


# ------------------------------------------------------------------------------- backward

@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 512), (3, 127), (700, 129), (2000, 512), (41, 768), (33, 1000), (29, 2049),
                                      (9, 4096), (700, 4100), (5, 9001), (3, 16384)])
@pytest.mark.parametrize("xt,yt,rt", [(F32, F32, F32), (F32, BF16, None), (BF16, BF16, BF16), (BF16, F32, F32)])
def test_rmsnorm_bwd(rows, dim, xt, yt, rt, cuda_ok):
    import hybrid_masked_attention_b200 as M
    x, dy, w = rnd(11, rows, dim, dtype=xt), rnd(12, rows, dim, dtype=yt), 1 + 0.3 * rnd(13, dim)
    dres = None if rt is None else rnd(14, rows, dim, dtype=rt)
    rstd = torch.rsqrt(x.float().square().mean(1) + 1e-6)
    dx, dw = padded(rows, dim, xt), torch.full((dim,), 7.0, device="cuda")
    ws = torch.full((M.rmsnorm_bwd_workspace_bytes(rows, dim),), 0xFF, dtype=torch.uint8, device="cuda")
    M.rmsnorm_bwd(x, w, rstd, dy, dres, dx, dw, ws)
    rx, rw = R.rmsnorm_bwd(x, w, rstd, dy, dres)
    X, G, r = x.double().abs(), (dy.double() * w.double()).abs(), rstd.double()[:, None]
    res = 0 if dres is None else dres.double().abs()
    # the dot product's sum and its factors, then the two terms and the sum with dres
    tol = r * (4 * U * G + X * r * r * (G * X).mean(1, keepdim=True) * (SUM_TERMS + 8) * U) + 3 * U * (res + rx.abs())
    assert ((dx.double() - rx).abs() <= tol + HALF[xt] * rx.abs()).all()
    # dw: every row once, in a fixed order; at most rows + 40 additions deep
    S = (dy.double().abs() * X * r).sum(0)
    assert ((dw.double() - rw).abs() <= (min(rows, 1200) + 40) * U * S).all()
    assert guards_kept(dx)
    again = torch.empty_like(dw)
    M.rmsnorm_bwd(x, w, rstd, dy, dres, dx, again, ws)
    assert torch.equal(again, dw)


def test_rmsnorm_bwd_differences(cuda_ok):
    """The gradient against central differences of the forward formula in 64 bits."""
    import hybrid_masked_attention_b200 as M
    rows, dim = 3, 70
    x, w, dy, dres = rnd(15, rows, dim), 1 + 0.2 * rnd(16, dim), rnd(17, rows, dim), rnd(18, rows, dim)
    rstd = torch.rsqrt(x.square().mean(1) + 1e-6)
    dx, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
    M.rmsnorm_bwd(x, w, rstd, dy, dres, dx, dw, torch.empty(M.rmsnorm_bwd_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda"))

    def loss(xx, ww):
        h, r, v = R.add_rmsnorm(xx, None, ww, 1e-6)
        return ((v * dy.double()).sum() + (h * dres.double()).sum()).item()

    eps = 1e-5
    for i, j in ((0, 0), (1, 33), (2, 69)):
        a, b = x.double().clone(), x.double().clone()
        a[i, j] += eps
        b[i, j] -= eps
        assert abs((loss(a, w) - loss(b, w)) / (2 * eps) - dx[i, j].item()) < 1e-4
        a, b = w.double().clone(), w.double().clone()
        a[j] += eps
        b[j] -= eps
        assert abs((loss(x, a) - loss(x, b)) / (2 * eps) - dw[j].item()) < 1e-4


def test_rmsnorm_bwd_in_place(cuda_ok):
    """dx may be dy or dres; odd pitches give the packed result to the last bits of the row's sum."""
    import hybrid_masked_attention_b200 as M
    rows, dim = 130, 260
    x, w, dy, dres = rnd(19, rows, dim), 1 + 0.2 * rnd(20, dim), rnd(21, rows, dim), rnd(22, rows, dim)
    rstd = torch.rsqrt(x.square().mean(1) + 1e-6)
    ws = torch.empty(M.rmsnorm_bwd_workspace_bytes(rows, dim), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(dim, device="cuda")
    M.rmsnorm_bwd(x, w, rstd, dy, dres, dx, dw, ws)
    for name in ("dy", "dres"):
        t = {"dy": dy.clone(), "dres": dres.clone()}
        M.rmsnorm_bwd(x, w, rstd, t["dy"], t["dres"], t[name], dw, ws)
        assert torch.equal(t[name], dx)
    xs, ys, rs, os_ = strided(x, 1), strided(dy, 3), strided(dres, 5), strided(x, 2)
    M.rmsnorm_bwd(xs, w, rstd, ys, rs, os_, dw, ws)
    assert (os_ - dx).abs().max() <= 1e-5


# ------------------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 127), (128, 128), (129, 129), (5, 1000), (260, 516), (7, 4097),
                                       (1, 16400)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant(rows, cols, dtype, block_rows, cuda_ok):
    import hybrid_masked_attention_b200 as M
    x = rnd(31, rows, cols, dtype=dtype) * torch.exp(rnd(32, rows, 1)).to(dtype)
    q, s = out8(rows, cols, block_rows)
    M.fp8_quant(x, q, s, block_rows)
    R.check_quant(q, s, x.double(), 0.0, block_rows)
    assert guards_kept(q) and guards_kept(s)
    for ex in (1, 4):   # other pitches, same bits: nothing is summed
        q2 = padded(rows, cols, F8, extra=ex)
        s2 = padded(s.shape[0], s.shape[1], F32, extra=ex)
        M.fp8_quant(strided(x, ex), q2, s2, block_rows)
        assert torch.equal(q2.float(), q.float()) and torch.equal(s2, s)
    odd = torch.zeros(rows * cols + 1, dtype=torch.uint8, device="cuda").view(F8)[1:].view(rows, cols)
    M.fp8_quant(x, odd, s, block_rows)
    assert torch.equal(odd.float(), q.float())


def test_quant_ties_and_specials(cuda_ok):
    """Exact powers of two keep their values; ties round to even; NaN and infinity as documented."""
    import hybrid_masked_attention_b200 as M
    x = torch.zeros(4, 128, device="cuda")
    x[0, :8] = torch.tensor([448., -448., 17., 18., 19., 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10])
    x[1, 3] = float("nan")
    x[1, 5] = 2.0
    x[2, 1] = float("inf")
    x[2, 2] = 1.0
    x[3, 0] = 1e-40
    q, s = out8(4, 128)
    M.fp8_quant(x, q, s)
    assert s[0].item() == 1.0
    # steps of 2 in [16, 32): 17 and 19 are ties; 2^-10 is half the smallest step of 2^-9
    assert q[0, :8].float().tolist() == [448., -448., 16., 18., 20., 2.0 ** -9, 0.0, 2.0 ** -8]
    assert torch.isnan(q[1, 3].float()) and q[1, 5].float().item() == 448.0 and s[1].item() == (torch.tensor(2.0) / 448).item()
    assert torch.isinf(s[2]) and torch.isnan(R.dequant(q, s)[2]).all()
    assert (q[3].float() == 0).all() and torch.isfinite(s[3]).all()


# ------------------------------------------------------------------------------- gate

HEADS = [syn.Heads(2, 1, 32), syn.Heads(8, 2, 64), syn.Heads(5, 5, 32), syn.Heads(3, 1, 256), syn.Heads(4, 1, 256)]


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("target", [False, True])
@pytest.mark.parametrize("gln", [False, True])
def test_gate_fp8(heads, target, gln, cuda_ok):
    import hybrid_masked_attention_b200 as M
    from gpu_cases import edge_batch
    from gpu_helpers import packed
    b = edge_batch()
    s = packed(b, heads)
    cfg = s.cfg
    rows, D = cfg.total_t if target else cfg.total_tokens, cfg.D
    a, u = rnd(41, rows, D, scale=0.2) + 0.1, rnd(42, rows, D, dtype=BF16)
    gamma = 1 + 0.3 * rnd(43, 3, D) if gln else None
    beta = 0.2 * rnd(44, 3, D) if gln else None
    kinds = torch.from_numpy(M.meta_read(cfg, s.meta)["row_type"]).long().cuda()
    kinds = kinds[kinds == 2] if target else kinds
    q, sc = out8(rows, D)
    stats = torch.empty(rows, 2, device="cuda") if gln else None
    M.gate_fwd_fp8(cfg, s.meta, target, a, u, gamma, beta, q, sc, stats)
    M.pack_check(s.meta)
    A, Ud = a.double(), u.double()
    if gln:
        mean = A.mean(1, keepdim=True)
        c = A - mean
        r = 1 / torch.sqrt(c.square().mean(1, keepdim=True) + 1e-5)
        g, bt = gamma.double()[kinds], beta.double()[kinds]
        v = (c * r * g + bt) * Ud
        # the mean's sum error shifts every element; the variance as the norm's sum of squares
        dmean = (SUM_TERMS + 2) * U * A.abs().mean(1, keepdim=True)
        rel = (SUM_TERMS + 8) * U
        err = (((dmean + A.abs() * 2 * U) * r + c.abs() * r * rel) * g.abs() + (c * r * g).abs() * 2 * U + bt.abs() * 2 * U) \
            * Ud.abs() + v.abs() * 2 * U
        assert ((stats[:, :1].double() - mean).abs() <= dmean + U * mean.abs()).all()
        assert ((stats[:, 1:].double() - r).abs() <= rel * r).all()
    else:
        v, err = A * Ud, (A * Ud).abs() * 2 * U
    R.check_quant(q, sc, v, err)
    assert guards_kept(q) and guards_kept(sc)


# ------------------------------------------------------------------------------- product

def operands(m, n, k, seed=51, extra=0):
    import hybrid_masked_attention_b200 as M
    a, sa = padded(m, k, F8, extra), padded(m, groups(k), F32, extra)
    b, sb = padded(n, k, F8, extra), padded(groups(n), groups(k), F32, extra)
    M.fp8_quant(rnd(seed, m, k) * torch.exp(rnd(seed + 1, m, 1)), a, sa)
    M.fp8_quant(rnd(seed + 2, n, k, scale=k ** -0.5), b, sb, 128)
    return a, sa, b, sb


def check_gemm(out, a, sa, b, sb, act, res):
    """Tolerance: the tensor cores add the 32 products of one instruction, and the sum so far,
    aligned to the largest and cut to no less than 24 bits: at most 33 units of 2^-23 of the
    block's sum of magnitudes for each of its 4 instructions; then one fp32 rounding per block.
    SiLU: slope at most 1.1.  fp32: evaluated to 9 roundings (exponential 3, 1 +, product of two,
    reciprocal 2, its two products) and 2 |x| for the exponential's argument.  bf16: h + h tanh(h)
    with h = x / 2 and a tanh of relative error 2^-11: |x| / 2 * 2^-11, and two roundings."""
    ref, S = R.gemm(a, sa, b, sb, act, res)
    nk = groups(a.shape[1])
    tol = S * (4 * 33 * 2.0 ** -23 + (nk + 2) * U)
    if act == "silu":
        pre, _ = R.gemm(a, sa, b, sb, None, None)
        own = pre.abs() * (9 + 2 * pre.abs()) * U if out.dtype == F32 else pre.abs() * (2.0 ** -12 + 2 * U)
        tol = 1.1 * tol + own
    tol = tol + HALF[out.dtype] * (ref.abs() + tol) + U * (0 if res is None else res.double().abs())
    d = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (d <= tol).all(), f"off by {float((d / tol).max())} tolerances"


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 17, 33), (5, 1280, 512), (16, 300, 1000), (33, 1000, 129), (64, 64, 2000),
          (65, 512, 4096), (127, 255, 384), (128, 256, 256), (129, 257, 130), (300, 1000, 1000), (1000, 33, 640),
          (777, 1280, 512), (2049, 640, 96), (1, 5000, 8192), (40, 2048, 8190),
          # more tiles than CTA pairs: 256 x 128 and 256 x 256 tiles, short and long K
          (2200, 2000, 512), (2200, 2000, 130), (2200, 1990, 1100), (5000, 2048, 512), (5000, 2050, 130), (4500, 2100, 1300)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype,act,res", [(BF16, None, False), (BF16, "silu", True), (F32, "silu", False), (F32, None, True)])
def test_gemm(m, n, k, dtype, act, res, cuda_ok):
    import hybrid_masked_attention_b200 as M
    a, sa, b, sb = operands(m, n, k)
    r = rnd(55, m, n, dtype=dtype) if res else None
    out = padded(m, n, dtype)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.fp8_gemm(a, sa, b, sb, out, status, act, r)
    M.fp8_check(status)
    check_gemm(out, a, sa, b, sb, act, r)
    assert guards_kept(out)


@pytest.mark.parametrize("m,n,k", [(3, 200, 300), (150, 200, 300)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gemm_strides_and_in_place(m, n, k, dtype, cuda_ok):
    """Wide pitches, output rows at odd element offsets, and the residual in the output itself."""
    import hybrid_masked_attention_b200 as M
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, sa, b, sb = operands(m, n, k, extra=2)
    r = rnd(56, m, n, dtype=dtype)
    want = torch.empty(m, n, dtype=dtype, device="cuda")
    M.fp8_gemm(a, sa, b, sb, want, status, None, r)
    check_gemm(want, a, sa, b, sb, None, r)
    buf = torch.full((m * (n + 3) + 1,), 5.0, dtype=dtype, device="cuda")
    odd = buf[1:].view(m, n + 3)[:, :n]
    odd.copy_(r)
    M.fp8_gemm(a, sa, b, sb, odd, status, None, odd)
    assert torch.equal(odd, want)
    assert (buf[0] == 5) and (buf[1:].view(m, n + 3)[:, n:] == 5).all()
    M.fp8_check(status)


def test_gemm_scale_borders(cuda_ok):
    """One element differs from zero at a time: its own scales, and no neighbour's, apply."""
    import hybrid_masked_attention_b200 as M
    m, n, k = 130, 300, 300
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sa, sb = torch.rand(m, 3, device="cuda") + 0.5, torch.rand(3, 3, device="cuda") + 0.5
    for i, j, c in ((0, 0, 0), (129, 299, 299), (127, 127, 127), (128, 128, 128), (64, 255, 256), (1, 256, 255)):
        a, b = padded(m, k, F8), padded(n, k, F8)
        a.copy_(torch.zeros(m, k))
        b.copy_(torch.zeros(n, k))
        a[i, c], b[j, c] = 3.0, 5.0
        out = torch.full((m, n), 9.0, device="cuda")
        M.fp8_gemm(a, sa, b, sb, out, status)
        want = 15.0 * sa[i, c // 128].double() * sb[j // 128, c // 128].double()
        assert abs(out[i, j].double() - want) <= 3 * U * want
        out[i, j] = 0
        assert (out == 0).all()


def test_gemm_nan_stays_in_its_row(cuda_ok):
    import hybrid_masked_attention_b200 as M
    for m in (20, 200):
        a, sa, b, sb = operands(m, 260, 256)
        a[11, 200] = float("nan")
        out = padded(m, 260, F32)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.fp8_gemm(a, sa, b, sb, out, status)
        assert torch.isnan(out[11]).all()
        rest = [i for i in range(m) if i != 11]
        check_gemm(out[rest], a[rest], sa[rest], b, sb, None, None)


def test_gemm_status_word_stops_later_calls(cuda_ok):
    import hybrid_masked_attention_b200 as M
    a, sa, b, sb = operands(10, 64, 128)
    status = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    out = torch.full((10, 64), 2.0, device="cuda")
    M.fp8_gemm(a, sa, b, sb, out, status)
    assert (out == 2).all()
    with pytest.raises(M.MtfmError) as e:
        M.fp8_check(status)
    assert e.value.status == 6
    status.zero_()
    M.fp8_gemm(a[:0], sa[:0], b, sb, out[:0], status)
    M.fp8_check(status)


def test_offsets_past_31_bits(cuda_ok):
    """More than 2^31 elements: the last rows of the quantiser, the norm and the product."""
    import hybrid_masked_attention_b200 as M
    rows, cols = 140_000, 16_384
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x[-3:] = rnd(61, 3, cols, dtype=BF16)
    x[:-3] = 1.0
    q, s = torch.empty(rows, cols, dtype=F8, device="cuda"), torch.empty(rows, cols // 128, device="cuda")
    M.fp8_quant(x, q, s)
    R.check_quant(q[-3:], s[-3:], x[-3:].double(), 0.0)
    w = 1 + 0.1 * rnd(62, cols)
    M.add_rmsnorm_fp8(x, None, w, None, q, s)
    _, _, v = R.add_rmsnorm(x[-3:], None, w, 1e-6)
    R.check_quant(q[-3:], s[-3:], v, v.abs() * 64 * U)
    a, sa, b, sb = operands(rows, cols, 128)
    out, status = x, torch.zeros(1, dtype=torch.int32, device="cuda")
    M.fp8_gemm(a, sa, b, sb, out, status)
    M.fp8_check(status)
    check_gemm(out[-130:], a[-130:], sa[-130:], b, sb, None, None)


def test_two_streams_at_once(cuda_ok):
    """Products and norms in flight on two streams, sharing a status word: each as if alone."""
    import hybrid_masked_attention_b200 as M
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    jobs = [(operands(m, n, k, seed), torch.empty(m, n, device="cuda")) for m, n, k, seed in
            ((700, 1280, 512, 71), (20, 4096, 2048, 75), (900, 640, 1024, 79), (9, 1280, 512, 83))]
    want = []
    for ops, out in jobs:
        M.fp8_gemm(*ops, out, status)
        want.append(out.clone())
        out.zero_()
    x, w = rnd(87, 3000, 512), torch.ones(512, device="cuda")
    q, s = out8(3000, 512)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(10):
        for i, (ops, out) in enumerate(jobs):
            M.fp8_gemm(*ops, out, status, stream=streams[(i + rep) % 2])
        M.add_rmsnorm_fp8(x, None, w, None, q, s, stream=streams[rep % 2])
        torch.cuda.synchronize()
        for (_, out), t in zip(jobs, want):
            assert torch.equal(out, t)
            out.zero_()
        torch.cuda.synchronize()
    M.fp8_check(status)


# ------------------------------------------------------------------------------- refusals

def test_wrapper_refusals(cuda_ok):
    import hybrid_masked_attention_b200 as M
    a, sa, b, sb = operands(8, 64, 128)
    out, st = torch.empty(8, 64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="residual"):
        M.fp8_gemm(a, sa, b, sb, out, st, None, out.bfloat16())
    with pytest.raises(ValueError, match="a_scale"):
        M.fp8_gemm(a, sa[:, :0], b, sb, out, st)
    with pytest.raises(ValueError, match="act"):
        M.fp8_gemm(a, sa, b, sb, out, st, "relu")
    with pytest.raises(ValueError, match="status"):
        M.fp8_gemm(a, sa, b, sb, out, st.long())
    with pytest.raises(ValueError, match="out must be"):
        M.fp8_gemm(a, sa, b, sb, out.half(), st)
    with pytest.raises(ValueError, match="unit column"):
        M.fp8_gemm(a, sa, b, sb, out.t().contiguous().t(), st)
    with pytest.raises(ValueError, match="overlapping"):
        M.fp8_quant(torch.zeros(300, device="cuda").as_strided((4, 128), (10, 1)), *out8(4, 128))
    odd = torch.empty(8 * 130, dtype=torch.uint8, device="cuda").view(F8).view(8, 130)[:, :128]
    with pytest.raises(M.MtfmError) as e:    # pitch 130
        M.fp8_gemm(odd, sa, b, sb, out, st)
    assert e.value.status == 1
    x = rnd(1, 4, 64)
    with pytest.raises(M.MtfmError):         # x_out without delta
        M.add_rmsnorm_fp8(x, None, torch.ones(64, device="cuda"), x, *out8(4, 64))
    with pytest.raises(ValueError, match="x must be"):
        M.add_rmsnorm_fp8(x.double(), None, torch.ones(64, device="cuda"), None, *out8(4, 64))
    with pytest.raises(ValueError, match="weight"):
        M.add_rmsnorm_fp8(x, None, torch.ones(63, device="cuda"), None, *out8(4, 64))
    with pytest.raises(M.MtfmError) as e:
        M.rmsnorm_bwd(x, torch.ones(64, device="cuda"), torch.ones(4, device="cuda"), x, None, x.clone(),
                      torch.empty(64, device="cuda"), torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    M.fp8_check(st)
