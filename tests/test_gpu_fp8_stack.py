"""The backbone layers with 8-bit projections: against the public operators run one after
another, against the fp64 oracle, replayed from a graph and on another stream; and the
operators in the order a training step uses them."""
import numpy as np
import pytest
import torch

import fp8_ref as R
import mtfm_synth as syn
from fp8_ref import F8, groups
from gpu_cases import edge_batch
from gpu_helpers import bf16_tensor, config_for, f32_tensor, upload_batch
from oracle import mtfm_oracle as O

pytestmark = pytest.mark.gpu


def setup(batch, heads, d, kinds, seed=91):
    import hybrid_masked_attention_b200 as M
    host = syn.stack_weights(heads, d, seed, kinds=kinds, std=0.05, std_o=0.01, random_norms=True)
    layers = [M.LayerWeights(w.kind, f32_tensor(w.rms_w), bf16_tensor(w.w_in),
                             bf16_tensor(w.w_kv) if w.w_kv is not None else None, bf16_tensor(w.w_o),
                             f32_tensor(w.gamma), f32_tensor(w.beta)) for w in host]
    cfg = config_for(batch, heads)
    meta = M.alloc_meta(cfg)
    M.pack(cfg, *upload_batch(batch), meta)
    M.pack_check(meta)
    ws = torch.full((M.fp8_stack_workspace_bytes(cfg, d),), 0xFF, dtype=torch.uint8, device="cuda")
    X0 = syn.bf16_bits_to_f32(syn.stack_input(batch, d, seed)).astype(np.float32)
    return host, [M.Fp8LayerWeights.quantized(w) for w in layers], cfg, meta, ws, torch.from_numpy(X0).cuda()


def layer_by_operators(cfg, meta, w, x, status):
    """One layer as a caller of the single operators writes it."""
    import hybrid_masked_attention_b200 as M
    D, Dkv, d, N = cfg.D, cfg.Dkv, x.shape[1], cfg.total_tokens
    new = lambda r, c, t=torch.bfloat16: torch.empty(r, c, dtype=t, device="cuda")
    m = M.meta_read(cfg, meta)
    t_rows = torch.from_numpy(np.nonzero(m["row_type"] == 2)[0]).cuda()
    target = w.kind == "T"

    def normed(rows):
        q, s = new(rows.shape[0], d, F8), new(rows.shape[0], groups(d), torch.float32)
        M.add_rmsnorm_fp8(rows, None, w.rms_w, None, q, s)
        return q, s

    def product(a, wt, out, act, res=None):
        M.fp8_gemm(*a, *wt, out, status, act, res)
        return out

    xn = normed(x)
    if target:
        uq = product(normed(x[t_rows].contiguous()), w.w_in, new(len(t_rows), 2 * D), "silu")
        kv = product(xn, w.w_kv, new(N, 2 * Dkv), "silu")
        u, q = (t.contiguous() for t in uq.split(D, 1))
        k, v = (t.contiguous() for t in kv.split(Dkv, 1))
    else:
        u, q, k, v = (t.contiguous() for t in product(xn, w.w_in, new(N, 2 * D + 2 * Dkv), "silu").split([D, D, Dkv, Dkv], 1))
    rows = len(t_rows) if target else N
    a = new(rows, D, torch.float32)
    (M.attn_target if target else M.attn_full)(cfg, meta, q, k, v, a)
    y = new(rows, D, F8), new(rows, groups(D), torch.float32)
    M.gate_fwd_fp8(cfg, meta, target, a, u, w.gamma, w.beta, *y, new(rows, 2, torch.float32))
    if target:
        xt = x[t_rows].contiguous()
        x[t_rows] = product(y, w.w_o, xt, None, xt)
    else:
        product(y, w.w_o, x, None, x)


CASES = {"pair": (lambda: syn.pair_batch(4, 1002), syn.PAIR_HEADS, 512), "tiny": (syn.tiny_batch, syn.TINY_HEADS, 64),
         "d768": (lambda: syn.pair_batch(3, 1007), syn.Heads(3, 1, 256), 768), "edge": (edge_batch, syn.Heads(4, 2, 64), 320)}


@pytest.mark.parametrize("kind", ["F", "T"])
@pytest.mark.parametrize("case", sorted(CASES))
def test_layer_is_its_operators(case, kind, cuda_ok):
    import hybrid_masked_attention_b200 as M
    make, heads, d = CASES[case]
    host, (w,), cfg, meta, ws, x = setup(make(), heads, d, (kind,))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = x.clone()
    layer_by_operators(cfg, meta, w, want, status)
    x0 = x.clone()
    M.fp8_layer_fwd(cfg, meta, d, w, x, ws)
    M.pack_check(meta)
    M.fp8_check(status)
    # the same kernels on the same values; the Target attention may add its key chunks in another
    # order (fp32 reductions), which moves a rounding of Y now and then
    diff = (x - want).norm() / (want - x0).norm()
    assert diff <= 2e-3, diff
    if kind == "T":
        row_type = torch.from_numpy(M.meta_read(cfg, meta)["row_type"]).cuda()
        assert torch.equal(x[row_type != 2], x0[row_type != 2])


@pytest.mark.parametrize("kind", ["F", "T"])
@pytest.mark.parametrize("case", ["pair", "d768"])
def test_layer_against_oracle(case, kind, cuda_ok):
    """The layer's change of X against the fp64 layer on unrounded weights.  Each 8-bit operand
    is off by at most 2^-4 relative per element, of uniform distribution 2^-4 / sqrt(3) rms in
    the worst binade: a product of two such operands by sqrt(2) of that, 5.1e-2.  U and A = f(Q,
    K, V) carry it (A: three operands, sqrt(3)), Y their product, its own rounding and the
    output projection's weight two more: sqrt(1 + 3 + 1) * 5.1e-2 + bf16 roundings < 0.12."""
    import hybrid_masked_attention_b200 as M
    make, heads, d = CASES[case]
    b = make()
    host, (w,), cfg, meta, ws, x = setup(b, heads, d, (kind,))
    X0 = x.cpu().numpy().astype(np.float64)
    M.fp8_layer_fwd(cfg, meta, d, w, x, ws)
    M.pack_check(meta)
    ref = (O.full_layer if kind == "F" else O.target_layer)(b, heads, X0, host[0])
    change, want = x.cpu().numpy() - X0, ref - X0
    assert np.linalg.norm(change - want) <= 0.12 * np.linalg.norm(want)


def test_stack_layer_by_layer_graph_and_stream(cuda_ok):
    """A stack is its layers; a captured stack replays to the same X; another stream works."""
    import hybrid_masked_attention_b200 as M
    b, heads, d = syn.pair_batch(4, 1002), syn.PAIR_HEADS, 512
    _, layers, cfg, meta, ws, x = setup(b, heads, d, ("F", "T", "T", "F"))
    x0, want = x.clone(), x.clone()
    for w in layers:
        M.fp8_layer_fwd(cfg, meta, d, w, want, ws)
    M.fp8_stack_fwd(cfg, meta, d, layers, x, ws)
    M.pack_check(meta)
    near = lambda t: (t - want).norm() <= 2e-3 * (want - x0).norm()
    assert near(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x.copy_(x0)
    torch.cuda.synchronize()
    M.fp8_stack_fwd(cfg, meta, d, layers, x, ws, stream=side)
    side.synchronize()
    assert near(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.fp8_stack_fwd(cfg, meta, d, layers, x, ws)
    for _ in range(3):
        x.copy_(x0)
        g.replay()
        torch.cuda.synchronize()
        assert near(x)
    M.pack_check(meta)


def test_stack_does_nothing_on_bad_metadata(cuda_ok):
    import hybrid_masked_attention_b200 as M
    b, heads, d = syn.tiny_batch(), syn.TINY_HEADS, 64
    _, layers, cfg, meta, ws, x = setup(b, heads, d, ("F", "T"))
    lens = list(upload_batch(b))
    lens[0] = lens[0] + 1                 # lengths that do not add up
    M.pack(cfg, *lens, meta)
    x0 = x.clone()
    M.fp8_stack_fwd(cfg, meta, d, layers, x, ws)
    torch.cuda.synchronize()
    assert torch.equal(x, x0)
    with pytest.raises(M.MtfmError):
        M.pack_check(meta)


@pytest.mark.parametrize("rows", [1, 37, 700])
def test_training_step_of_a_projection(rows, cuda_ok):
    """norm + product forward; quantised gradient, product with the transposed weight, norm
    backward.  Every step against 64 bits on the step's own inputs, the chain through a graph."""
    import hybrid_masked_attention_b200 as M
    d, n = 264, 400
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, delta, wn = rnd(rows, d), rnd(rows, d).bfloat16(), 1 + 0.2 * rnd(d)
    W, dy, dres = rnd(n, d) * d ** -0.5, rnd(rows, n), rnd(rows, d)
    f8 = lambda r, c, br=1: (R.padded(r, c, F8), torch.empty(-(-r // br), groups(c), device="cuda"))
    (w8, wt8), (h8, dy8) = (f8(n, d, 128), f8(d, n, 128)), (f8(rows, d), f8(rows, n))
    y, dh = torch.empty(rows, n, device="cuda"), torch.empty(rows, d, device="cuda")
    h, rstd = torch.empty_like(x), torch.empty(rows, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty(d, device="cuda")
    ws = torch.empty(M.rmsnorm_bwd_workspace_bytes(rows, d), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Wt = W.t().contiguous()

    def step():
        M.fp8_quant(W, *w8, 128)
        M.fp8_quant(Wt, *wt8, 128)
        M.add_rmsnorm_fp8(x, delta, wn, h, *h8, rstd)
        M.fp8_gemm(*h8, *w8, y, status)
        M.fp8_quant(dy, *dy8)
        M.fp8_gemm(*dy8, *wt8, dh, status)
        M.rmsnorm_bwd(h, wn, rstd, dh, dres, dx, dw, ws)

    step()
    M.fp8_check(status)
    assert torch.equal(wt8[0].float(), w8[0].float().t())     # the same blocks, transposed
    assert torch.equal(wt8[1], w8[1].t())
    _, r, v = R.add_rmsnorm(x, delta, wn, 1e-6)
    want, S = R.gemm(*h8, *w8, None, None)
    assert ((y.double() - want).abs() <= S * 2.0 ** -16).all()
    want, S = R.gemm(*dy8, *wt8, None, None)
    assert ((dh.double() - want).abs() <= S * 2.0 ** -16).all()
    wx, ww = R.rmsnorm_bwd(h, wn, rstd, dh, dres)
    assert (dx.double() - wx).norm() <= 1e-6 * wx.norm() and (dw.double() - ww).norm() <= 1e-5 * ww.norm()
    # end to end: the 8-bit chain's gradient against the exact one (one rounded operand pair)
    exact, _ = R.rmsnorm_bwd(x.double() + delta.double(), wn, r, dy.double() @ W.double(), dres)
    assert (dx.double() - exact).norm() <= 0.06 * exact.norm()
    keep = [t.clone() for t in (y, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (y, dx, dw, h):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    for t, k in zip((y, dx, dw), keep):
        assert torch.equal(t, k)


def test_under_bounds_checked_build(cuda_ok):
    """The product's and the layers' small cases under the bounds-checked build, which tests every
    TMA coordinate: a failed test would set the error words that these cases check."""
    import os
    import subprocess
    import sys
    if os.environ.get("MTFM_LIBRARY"):
        pytest.skip("already running under another build")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "hybrid_masked_attention_b200"))
    import build
    env = dict(os.environ, MTFM_LIBRARY=build.build(debug_bounds=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_fp8.py", "tests/test_gpu_fp8_stack.py", "-q", "-x", "-m",
                        "gpu", "-k", "test_gemm or tiny or edge or training", "-p", "no:cacheprovider"],
                       cwd=root, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-3000:]
