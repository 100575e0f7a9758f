"""Host-side refusals of the norm's calls with every matrix at an address of its own, and of
outputs in the place of an input whose rows or elements do not coincide (no GPU; the pointers are
never followed, and every call here is refused)."""
import pytest

from test_fp8_host import GEMM, P, bwd, m, norm  # noqa: F401  (m: the fixture)

NORM = dict(x=P, d=2 * P, w=3 * P, xo=4 * P, q=5 * P, s=6 * P, r=7 * P)
BWD = dict(x=P, w=2 * P, r=3 * P, y=4 * P, dr=5 * P, dx=6 * P, dw=7 * P, ws=8 * P)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(xt=2), 1), (dict(ldx=255), 1), (dict(x=P + 2), 1), (dict(d=None), 1), (dict(dt=-1), 1),
    (dict(ldd=1), 1), (dict(d=P + 1), 1), (dict(w=None), 1), (dict(xo=P + 2), 1), (dict(ldo=0), 1), (dict(q=None), 1),
    (dict(ldq=255), 1), (dict(s=None), 1), (dict(lds=1), 1), (dict(r=P + 2), 1),
    # x_out at x, or at delta, with other rows or elements
    (dict(xo=P, ldo=264), 1), (dict(xo=P, ldx=300, ldo=256), 1), (dict(xo=2 * P), 1), (dict(xo=2 * P, dt=0, ldd=260), 1),
    (dict(xo=2 * P, rows=1), 1),
])
def test_norm_refusals(m, kw, status):  # noqa: F811
    assert norm(m, **{**NORM, **kw}) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(r=None), 1), (dict(y=None), 1), (dict(yt=3), 1), (dict(ldy=255), 1),
    (dict(drt=5), 1), (dict(lddr=3), 1), (dict(dx=None), 1), (dict(dx=P + 2), 1), (dict(dw=None), 1), (dict(ws=None), 1),
    (dict(ws=P + 8), 1), (dict(wsb=64), 4),
    # dx at dy, dres or x with other rows or elements
    (dict(dx=4 * P, lddx=264), 1), (dict(dx=4 * P, ldy=264), 1), (dict(dx=4 * P, yt=1), 1), (dict(dx=5 * P), 1),
    (dict(dx=5 * P, drt=0, lddr=257), 1), (dict(dx=P, ldx=260), 1), (dict(dx=4 * P, yt=1, rows=1), 1),
])
def test_norm_bwd_refusals(m, kw, status):  # noqa: F811
    assert bwd(m, **{**BWD, **kw}) == status


def test_gemm_in_place_pitch(m):  # noqa: F811
    a = dict(GEMM, res=9 * P, ldr=304, out=9 * P)
    assert m._lib.mtfm_fp8_gemm(*a.values(), None) == 1
