"""Plain 64-bit forms of the 8-bit operators and the error bounds their tests use.

Half a step of rounding is eps / 2 relative: fp32 U = 2^-24, bf16 2^-8, e4m3 2^-4 (an absolute
2^-10 below 2^-6).  Bounds count fp32 roundings along the kernels' way and add one rounding to
the output's type.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}
F8 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100


def groups(n):
    return -(-n // 128)


def padded(rows, cols, dtype, extra=0, device="cuda"):
    """[rows, cols] with rows on 16-byte boundaries, `extra` 16-byte steps between them, and a
    guard value in every byte that does not belong to it."""
    size = torch.empty((), dtype=dtype).element_size()
    step = 16 // size
    ld = (-(-cols // step) + extra) * step
    base = torch.full(((rows + 1) * ld * size,), 0x3B, dtype=torch.uint8, device=device).view(dtype).view(rows + 1, ld)
    return base[:rows, :cols]


def guards_kept(t):
    """Whether the bytes of padded()'s buffer outside t still hold their guard value."""
    rows, cols = t.shape
    base = t._base if t._base is not None else t
    ld = t.stride(0)
    b = base.view(torch.uint8).view(rows + 1, -1).cpu()
    used = cols * t.element_size()
    return bool((b[:rows, used:] == 0x3B).all() and (b[rows:] == 0x3B).all()) if ld else True


def half_step(t):
    """Half the spacing of e4m3 at |t| (64-bit tensor, |t| <= 448)."""
    e = torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6)))
    return torch.exp2(e - 4)


def group_max(v, block_rows):
    """max |v| of the group of each element, at least FLOOR (64-bit), and the scales."""
    R, C = v.shape
    m = torch.full((-(-R // block_rows), groups(C)), FLOOR, dtype=torch.float64, device=v.device)
    for i in range(m.shape[0]):
        for g in range(m.shape[1]):
            blk = v[i * block_rows:(i + 1) * block_rows, g * 128:(g + 1) * 128].abs()
            m[i, g] = torch.clamp(blk.max(), min=FLOOR)
    rows = torch.arange(R, device=v.device) // block_rows
    cols = torch.arange(C, device=v.device) // 128
    return m[rows][:, cols], m / 448.0


def group_max_rows(v):
    """group_max for 1 x 128 groups without the loops."""
    R, C = v.shape
    t = torch.nn.functional.pad(v.abs(), (0, groups(C) * 128 - C)).view(R, groups(C), 128).amax(2).clamp_min(FLOOR)
    return t.repeat_interleave(128, 1)[:, :C], t / 448.0


def check_quant(q, scale, v, err, block_rows=1):
    """(q, scale) against the 64-bit values v known to `err` absolute (same shape, or a number
    times the group's maximum): scale within the maximum's error and two roundings, q within
    half a step and the error of the scaled value (its own, the maximum's, 3 roundings)."""
    m, s = group_max_rows(v) if block_rows == 1 else group_max(v, block_rows)
    err = torch.as_tensor(err, dtype=torch.float64, device=v.device).expand_as(v)
    me, _ = group_max_rows(err) if block_rows == 1 else group_max(err, block_rows)
    srow = torch.arange(v.shape[0], device=v.device) // block_rows
    scol = torch.arange(v.shape[1], device=v.device) // 128
    got = scale.double()[srow][:, scol]
    assert torch.isfinite(scale).all()
    assert ((got - m / 448.0).abs() <= me / 448.0 + 2 * U * m / 448.0).all(), "scale"
    t = v * 448.0 / m
    tol = half_step(t.clamp(-448, 448)) + (err + t.abs() / 448.0 * me) * 448.0 / m + 4 * U * t.abs()
    d = (q.double() - t).abs()
    assert (d <= tol).all(), f"q off by {float((d - tol).max())} more than it may"


def dequant(q, scale, block_rows=1):
    R, C = q.shape
    rows = torch.arange(R, device=q.device) // block_rows
    cols = torch.arange(C, device=q.device) // 128
    return q.double() * scale.double()[rows][:, cols]


def add_rmsnorm(x, delta, w, eps):
    h = x.double() if delta is None else x.double() + delta.double()
    r = 1.0 / torch.sqrt(h.square().mean(1) + eps)
    return h, r, h * r[:, None] * w.double()


def rmsnorm_bwd(x, w, r, dy, dres):
    x, w, r, dy = x.double(), w.double(), r.double()[:, None], dy.double()
    g = dy * w
    dx = r * (g - x * r * r * (g * x).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * x * r).sum(0)


def gemm(a, sa, b, sb, act, res):
    """(out, S): the product in 64 bits and S = sum_k |A| |B|, the scale of its rounding errors."""
    A, B = dequant(a, sa), dequant(b, sb, 128)
    c = A @ B.t()
    S = A.abs() @ B.abs().t()
    if act == "silu":
        c = c / (1.0 + torch.exp(-c))
    if res is not None:
        c = c + res.double()
    return c, S
