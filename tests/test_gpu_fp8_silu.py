"""SiLU of the block-scaled product over the whole range of its argument, against 64 bits with
bounds relative to SiLU(x) itself.  The argument is set exactly: one element of a row of A is 1
and its scale is x, B holds powers of two."""
import pytest
import torch

from fp8_ref import F8, HALF, U, groups, padded

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
COLUMNS = [1.0, -1.0, 0.5, -0.5, 2.0, -2.0, 1.0, -1.0]


def arguments():
    a = torch.cat([torch.logspace(-30, 30, 241, dtype=torch.float64), torch.linspace(0.05, 130, 400, dtype=torch.float64),
                   torch.tensor([43.5, 43.6, 43.7, 87.2, 87.4, 88.7, 103.9], dtype=torch.float64)])
    return a.float().cuda()


def product(x, n, out_type, nan_column=None):
    import hybrid_masked_attention_b200 as M
    m, k = x.numel(), 128
    a, b = padded(m, k, F8), padded(n, k, F8)
    a.copy_(torch.zeros(m, k))
    b.copy_(torch.zeros(n, k))
    a[:, 5] = 1.0
    col = torch.tensor(COLUMNS * groups(n) * 16)[:n].cuda()
    b[:, 5] = col.to(F8)
    if nan_column is not None:
        b[nan_column, 5] = float("nan")
    out = padded(m, n, out_type)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.fp8_gemm(a, x[:, None].contiguous(), b, torch.ones(groups(n), 1, device="cuda"), out, status, "silu")
    M.fp8_check(status)
    return out, x.double()[:, None] * col.double()


def check(out, x):
    """x is exact (one product of 1, a power of two and the scale).  e = exp(-|x|): its argument is
    rounded twice, 2 |x| U, the exponential is good to 4 U; 1 + e, the products that share the
    reciprocal and the reciprocal itself 7 U, and below zero two products 2 U.  Above zero e's error
    counts e / (1 + e) times: (4 + 2 x) e / (1 + e) <= 2.1 for any x, so 11 U in all.  Results under
    2^-119 may be 0 (exp flushes below 2^-126)."""
    s = torch.where(x >= 0, x / (1 + torch.exp(-x)), x * torch.exp(x) / (1 + torch.exp(x)))
    s = torch.where(x < -700, torch.zeros_like(x), s)
    tol = torch.where(x >= 0, torch.full_like(x, 11 * U), (13 + 2 * x.abs()) * U) * s.abs()
    tol = torch.where(x < -120, torch.zeros_like(x), tol) + 2.0 ** -119
    if out.dtype != F32:
        tol = tol + HALF[out.dtype] * (s.abs() + tol)
    d = (out.double() - s).abs()
    assert torch.isfinite(out).all()
    worst = (d / tol).argmax()
    assert (d <= tol).all(), f"x = {x.flatten()[worst]}: {out.flatten()[worst]} for {s.flatten()[worst]}"


# rows of A up to 32, or CTA pairs; columns that leave by TMA, or directly
@pytest.mark.parametrize("n", [8, 7, 264])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_silu_over_the_range(n, dtype, cuda_ok):
    x = arguments()
    check(*product(x, n, dtype))
    for i in range(0, x.numel(), 32):
        check(*product(x[i:i + 32], n, dtype))


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_silu_of_nan_and_infinity(rows, dtype, cuda_ok):
    """Infinity stays, minus infinity is 0 times infinity, NaN stays in its own element."""
    x = torch.full((rows,), 1.5, device="cuda")
    x[1] = float("inf")
    out, _ = product(x, 8, dtype)
    want = [torch.tensor(c).sign().item() > 0 for c in COLUMNS]
    for j, up in enumerate(want):
        assert (out[1, j] == float("inf")) if up else torch.isnan(out[1, j])
    x[1] = 1.5
    clean, v = product(x, 8, dtype)
    check(clean, v)
    out, _ = product(x, 8, dtype, nan_column=2)
    assert torch.isnan(out[:, 2]).all()
    keep = [0, 1, 3, 4, 5, 6, 7]
    check(out[:, keep], v[:, keep])
