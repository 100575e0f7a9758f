"""The bytes of the 8-bit form: q = e4m3(v * (448 (1 / m))), every operation rounded to nearest
fp32, is bit for bit what elementary fp32 torch operations give on the CPU."""
import pytest
import torch

from fp8_ref import F8, groups, padded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def formula(v, block_rows):
    """(bytes, scale) of fp32 values on the CPU."""
    R, C = v.shape
    pr, pc = -(-R // block_rows) * block_rows, groups(C) * 128
    t = torch.nn.functional.pad(v, (0, pc - C, 0, pr - R)).view(pr // block_rows, block_rows, pc // 128, 128)
    m = t.abs().amax(dim=(1, 3), keepdim=True).clamp_min(2.0 ** -100)
    q = (t * (448.0 * m.reciprocal())).view(pr, pc)[:R, :C].to(F8)
    return q.view(torch.uint8), (m / 448.0).view(pr // block_rows, pc // 128)


def check(q, s, v, block_rows=1):
    want, scale = formula(v.cpu(), block_rows)
    off = int((q.cpu().view(torch.uint8) != want).sum())
    assert off == 0, f"{off} of {want.numel()} bytes differ"
    assert torch.equal(s.cpu(), scale)


def out8(rows, cols, block_rows=1):
    return padded(rows, cols, F8), torch.empty(-(-rows // block_rows), groups(cols), device="cuda")


def rnd(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * torch.exp(torch.randn(shape[0], 1, generator=g, device="cuda"))).to(dtype)


@pytest.mark.parametrize("rows,cols", [(12345, 1000), (2000, 4097), (1, 130), (300, 128)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantiser_bytes(rows, cols, dtype, block_rows, cuda_ok):
    import hybrid_masked_attention_b200 as M
    x = rnd(101, rows, cols, dtype=dtype)
    q, s = out8(rows, cols, block_rows)
    M.fp8_quant(x, q, s, block_rows)
    check(q, s, x.float(), block_rows)


def test_quantiser_bytes_over_the_exponents(cuda_ok):
    """Group maxima from the floor to the largest finite fp32, where 1 / m is subnormal."""
    import hybrid_masked_attention_b200 as M
    e = torch.arange(-110, 128, device="cuda", dtype=torch.float64)
    x = (rnd(103, e.numel(), 256).double().clamp(-1.99, 1.99) * torch.exp2(e)[:, None]).float()
    q, s = out8(e.numel(), 256)
    M.fp8_quant(x, q, s)
    check(q, s, x)


@pytest.mark.parametrize("rows,dim", [(4000, 768), (3000, 1001), (500, 4096), (100, 9000)])
def test_norm_bytes(rows, dim, cuda_ok):
    """The norm's bytes from its own rstd: v = (x rstd) w has no sum in it."""
    import hybrid_masked_attention_b200 as M
    x, w, rstd = rnd(105, rows, dim), 1 + 0.2 * rnd(106, 1, dim)[0], torch.empty(rows, device="cuda")
    q, s = out8(rows, dim)
    M.add_rmsnorm_fp8(x, None, w, None, q, s, rstd)
    check(q, s, x.cpu() * rstd.cpu()[:, None] * w.cpu())


@pytest.mark.parametrize("target", [False, True])
def test_gate_bytes(target, cuda_ok):
    """The gate without GLN: v = a u."""
    import hybrid_masked_attention_b200 as M
    import mtfm_synth as syn
    from gpu_helpers import packed
    s = packed(syn.pair_batch(4, 1002), syn.PAIR_HEADS)
    rows, D = s.cfg.total_t if target else s.cfg.total_tokens, s.cfg.D
    a, u = rnd(107, rows, D), rnd(108, rows, D, dtype=BF16)
    q, sc = out8(rows, D)
    M.gate_fwd_fp8(s.cfg, s.meta, target, a, u, None, None, q, sc, None)
    M.pack_check(s.meta)
    check(q, sc, a.cpu() * u.cpu().float())
