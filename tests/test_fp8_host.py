"""Host-side argument checks of the 8-bit operators: bad calls are refused before any launch
(no GPU; the pointers are never followed)."""
import ctypes

import pytest
import torch

P = 4096   # an aligned address nothing reads


@pytest.fixture(scope="module")
def m():
    import hybrid_masked_attention_b200 as m
    return m


def norm(m, rows=4, dim=256, x=P, xt=0, ldx=256, d=P, dt=1, ldd=256, w=P, eps=1e-6, xo=P, ldo=256, q=P, ldq=256, s=P, lds=2,
         r=P):
    return m._lib.mtfm_add_rmsnorm_fp8(rows, dim, x, xt, ldx, d, dt, ldd, w, eps, xo, ldo, q, ldq, s, lds, r, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(dim=0), 1), (dict(dim=16385), 3), (dict(x=None), 1), (dict(xt=2), 1), (dict(ldx=255), 1),
    (dict(x=P + 2), 1), (dict(d=None), 1), (dict(dt=-1), 1), (dict(ldd=1), 1), (dict(d=P + 1), 1), (dict(w=None), 1),
    (dict(w=P + 2), 1), (dict(xo=P + 2), 1), (dict(ldo=0), 1), (dict(q=None), 1), (dict(ldq=255), 1), (dict(s=None), 1),
    (dict(lds=1), 1), (dict(s=P + 1), 1), (dict(r=P + 2), 1), (dict(rows=0, x=None, q=None), 0),
])
def test_norm_refusals(m, kw, status):
    assert norm(m, **kw) == status


def bwd(m, rows=4, dim=256, x=P, xt=0, ldx=256, w=P, r=P, y=P, yt=0, ldy=256, dr=P, drt=1, lddr=256, dx=P, lddx=256, dw=P,
        ws=P, wsb=None):
    wsb = m._lib.mtfm_rmsnorm_bwd_workspace_bytes(rows, dim) if wsb is None else wsb
    return m._lib.mtfm_rmsnorm_bwd(rows, dim, x, xt, ldx, w, r, y, yt, ldy, dr, drt, lddr, dx, lddx, dw, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(dim=0), 1), (dict(dim=20000), 3), (dict(x=None), 1), (dict(w=None), 1), (dict(r=None), 1),
    (dict(y=None), 1), (dict(yt=3), 1), (dict(ldy=255), 1), (dict(drt=5), 1), (dict(lddr=3), 1), (dict(dx=None), 1),
    (dict(dx=P + 2), 1), (dict(dw=None), 1), (dict(ws=None), 1), (dict(ws=P + 8), 1), (dict(wsb=64), 4),
])
def test_norm_bwd_refusals(m, kw, status):
    assert bwd(m, **kw) == status


def test_norm_bwd_workspace_query(m):
    assert m._lib.mtfm_rmsnorm_bwd_workspace_bytes(5, 0) == 0
    assert m._lib.mtfm_rmsnorm_bwd_workspace_bytes(-1, 5) == 0
    assert m._lib.mtfm_rmsnorm_bwd_workspace_bytes(5, 16385) == 0
    with pytest.raises(m.MtfmError):
        m.rmsnorm_bwd_workspace_bytes(5, 16385)
    assert m.rmsnorm_bwd_workspace_bytes(0, 1) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(br=2), 1), (dict(br=0), 1), (dict(x=None), 1), (dict(xt=7), 1), (dict(ldx=10), 1),
    (dict(q=None), 1), (dict(ldq=199), 1), (dict(s=None), 1), (dict(lds=1), 1), (dict(rows=0, x=None), 0),
    (dict(cols=0, x=None), 0),
])
def test_quant_refusals(m, kw, status):
    a = dict(rows=300, cols=200, x=P, xt=0, ldx=200, br=128, q=P, ldq=200, s=P, lds=2)
    a.update(kw)
    assert m._lib.mtfm_fp8_quant(*a.values(), None) == status


GEMM = dict(m=200, n=300, k=400, a=P, lda=400, sa=P, ldsa=4, b=P, ldb=400, sb=P, ldsb=4, act=0, res=None, ldr=0, out=P, ot=0,
            ldo=300, st=P)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(n=-1), 1), (dict(k=0), 1), (dict(m=2 ** 31 - 1), 3), (dict(k=2 ** 31 - 8), 3), (dict(act=2), 1),
    (dict(a=None), 1), (dict(a=P + 8), 1), (dict(lda=399), 1), (dict(lda=408), 1), (dict(lda=384), 1), (dict(b=None), 1),
    (dict(b=P + 4), 1), (dict(ldb=401), 1), (dict(sa=None), 1), (dict(ldsa=3), 1), (dict(sb=None), 1), (dict(ldsb=3), 1),
    (dict(sb=P + 2), 1), (dict(out=None), 1), (dict(ot=2), 1), (dict(ldo=299), 1), (dict(out=P + 2), 1), (dict(res=P, ldr=299), 1),
    (dict(res=P + 1, ldr=300), 1), (dict(res=P, ldr=304), 1), (dict(st=None), 1), (dict(st=P + 2), 1), (dict(m=0, a=None, out=None), 0),
    (dict(n=0, b=None, out=None), 0),
])
def test_gemm_refusals(m, kw, status):
    a = dict(GEMM)
    a.update(kw)
    assert m._lib.mtfm_fp8_gemm(*a.values(), None) == status


def test_check_refuses_null(m):
    assert m._lib.mtfm_fp8_check(None, None) == 1


def test_gate_refusals(m):
    c = m.Config(batch=2, total_tokens=20, total_r=4, total_t=4, hq=8, hkv=2, head_dim=64).c()
    call = lambda **kw: m._lib.mtfm_gate_fwd_fp8(ctypes.byref(c), *{**dict(meta=P, t=0, a=P, u=P, g=P, b=P, q=P, ldq=512, s=P,
                                                                        lds=4, st=P), **kw}.values(), None)
    for bad in (dict(meta=None), dict(meta=P + 16), dict(a=None), dict(a=P + 8), dict(u=None), dict(g=None), dict(b=None),
                dict(q=None), dict(q=P + 1), dict(ldq=511), dict(ldq=514), dict(s=None), dict(lds=3), dict(st=None),
                dict(st=P + 4), dict(g=P + 4)):
        assert call(**bad) == 1, bad


def test_stack_refusals(m):
    c = m.Config(batch=2, total_tokens=20, total_r=4, total_t=4, hq=8, hkv=2, head_dim=64).c()
    lib = m._lib
    ws = lib.mtfm_fp8_stack_workspace_bytes(ctypes.byref(c), 512)
    assert ws > 0
    assert lib.mtfm_fp8_stack_workspace_bytes(ctypes.byref(c), 96) == 0
    assert lib.mtfm_fp8_stack_workspace_bytes(ctypes.byref(c), 2048) == 0
    wt = lambda **kw: m.CFp8Weight(*{**dict(data=P, ld=512, scale=P, lds=4), **kw}.values())
    none = m.CFp8Weight()

    def layer(kind, w_in=None, w_kv=None, w_o=None, rms=P, g=P, b=P, x=P, wsb=ws, wsp=P, meta=P):
        lw = m.CFp8LayerWeights(rms, w_in or wt(), w_kv or (wt() if kind == "T" else none), w_o or wt(), g, b)
        return lib.mtfm_fp8_layer_fwd(ctypes.byref(c), meta, 512, int(kind == "T"), ctypes.byref(lw), x, wsp, wsb, None)

    assert layer("F", w_kv=wt()) == 1
    assert layer("T", w_kv=none) == 1
    for kind in "FT":
        for bad in (wt(data=None), wt(data=P + 8), wt(ld=500), wt(ld=520), wt(scale=None), wt(lds=3), wt(scale=P + 2)):
            assert layer(kind, w_in=bad) == 1 and layer(kind, w_o=bad) == 1
            if kind == "T":
                assert layer(kind, w_kv=bad) == 1
        assert layer(kind, rms=None) == 1 and layer(kind, g=None) == 1 and layer(kind, x=P + 4) == 1
        assert layer(kind, wsb=ws - 1) == 4 and layer(kind, wsp=P + 16) == 1 and layer(kind, meta=None) == 1
    lw = m.CFp8LayerWeights(P, wt(), none, wt(), P, P)
    assert lib.mtfm_fp8_stack_fwd(ctypes.byref(c), P, 512, 1, b"X", ctypes.byref(lw), P, P, ws, None) == 1
    assert lib.mtfm_fp8_stack_fwd(ctypes.byref(c), P, 512, 0, None, None, P, P, ws, None) == 0


def test_wrappers_refuse_host_tensors(m):
    x = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.zeros(4, 1)
    for call in (lambda: m.fp8_quant(x, q, s), lambda: m.add_rmsnorm_fp8(x, None, torch.ones(64), None, q, s),
                 lambda: m.fp8_gemm(q, s, q, s, x, torch.zeros(1, dtype=torch.int32)),
                 lambda: m.fp8_check(torch.zeros(1, dtype=torch.int32)),
                 lambda: m.rmsnorm_bwd(x, torch.ones(64), torch.ones(4), x, None, x, torch.ones(64), torch.zeros(8, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
