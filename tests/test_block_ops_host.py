"""The calls between two FP4 linears, without a GPU: the 64-bit references
(gradients against differences, the 8-bit format against its definition),
argument refusals before anything is enqueued, size helpers."""
import ctypes as C

import numpy as np
import pytest
import torch

import block_ref as R
import fp4_fully_quantized_b200 as F

NULL, SHAPE, ALIGN, FORMAT, WORKSPACE = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from fp4_fully_quantized_b200 import build
    build.build()
    return F.load()


def _differences(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_activation_gradient_is_the_differences(kind, gated):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((3, 8)) * 2
    dy = rng.standard_normal((3, 4 if gated else 8))
    want = _differences(lambda a: (R.act_fwd(a, kind, gated) * dy).sum(), z)
    # the quotient's own error: h^2/6 of a third derivative of order one, and
    # 1e-16 / h from the subtraction
    assert np.abs(R.act_bwd(dy, z, kind, gated) - want).max() < 1e-8


def test_rmsnorm_gradient_is_the_differences():
    rng = np.random.default_rng(2)
    x, r, w = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), rng.standard_normal(8)
    dy, dres = rng.standard_normal((3, 8)), rng.standard_normal((3, 8))
    s, rstd, xhat, _ = R.rmsnorm(x, r, w, 1e-3)
    dx, dw = R.rmsnorm_bwd(dy, xhat, rstd, w, dres)

    def loss(x, r, w):
        s, _, _, y = R.rmsnorm(x, r, w, 1e-3)
        return (y * dy).sum() + (s * dres).sum()

    assert np.abs(dx - _differences(lambda a: loss(a, r, w), x)).max() < 1e-8
    assert np.abs(dx - _differences(lambda a: loss(x, a, w), r)).max() < 1e-8
    assert np.abs(dw - _differences(lambda a: loss(x, r, a), w)).max() < 1e-8


def test_block_format_by_search():
    """Scale: the least power of two that holds the block; codes: the nearest of
    all E4M3 values, ties to the even code."""
    rng = np.random.default_rng(3)
    v = rng.standard_normal((64, 32)) * np.exp2(rng.integers(-130, 100, (64, 1)).astype(float))
    v[0, 0] = 2 * np.abs(v[0]).max()
    v[1], v[2, :], v[2, 5] = 0.0, 1.0, 448.0
    v[3] = np.linspace(-448, 448, 32)
    v[4, :], v[4, 0] = 0.1, 449.0
    values, b = R.encode(v)
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fits = lambda top, e: top <= 448 * 2.0 ** e
    for r in range(64):
        top, e = np.abs(v[r]).max(), int(b[r, 0]) - 127
        assert (top == 0 and e == -127) or (fits(top, e) and (e == -127 or not fits(top, e - 1)))
        q = np.ldexp(v[r], -e)
        off = np.abs(q[:, None] - np.where(np.isnan(table), np.inf, table))
        best = off.min(1)
        assert np.array_equal(np.abs(values[r] - q), best)
        for i in range(32):
            near = {abs(int(c)) & 127 for c in np.flatnonzero(off[i] == best[i])}
            if len(near) == 2:                       # a tie: the even code
                even = [c for c in near if c % 2 == 0][0]
                assert abs(values[r, i]) == table[even]


P = lambda n: n << 20                                # fake, aligned, never dereferenced
_kept = []


def _ck(rows, cols, codes=7, scales=8):
    _kept.append(F.Ckpt8C(codes << 20 if codes else None, scales << 20 if scales else None, rows, cols))
    return C.addressof(_kept[-1])


def _fwd(lib, **o):
    ws, n = o.pop("ws", None), o.pop("n", 0)
    a = dict(x=P(1), ldx=64, res=P(2), ldr=64, out=P(3), ldo=64, w=P(4), y=P(5), ldy=64, q=0, rstd=0,
             amax=0, rows=4, cols=64, eps=1e-6, rt=0, wt=0, of=0)
    a.update(o)
    return lib.fqt_rmsnorm_fwd(F._FWD(*a.values()), ws, n, None)


@pytest.mark.parametrize("o,code", [
    (dict(x=0), NULL), (dict(w=0), NULL), (dict(y=0), NULL), (dict(res=0), NULL),
    (dict(out=0), NULL), (dict(cols=60, ldx=60), SHAPE), (dict(cols=0), SHAPE),
    (dict(cols=16392, ldx=16392), SHAPE), (dict(rows=-1), SHAPE), (dict(ldx=56), SHAPE),
    (dict(ldy=56), SHAPE), (dict(ldx=68), ALIGN), (dict(x=(1 << 20) + 2), ALIGN),
    (dict(w=(1 << 20) + 8), ALIGN), (dict(rt=2), FORMAT), (dict(wt=5), FORMAT),
    (dict(eps=0.0), FORMAT), (dict(eps=float("nan")), FORMAT), (dict(eps=float("inf")), FORMAT),
    (dict(q=_ck(4, 64), of=2), FORMAT), (dict(q=_ck(4, 96)), SHAPE), (dict(q=_ck(5, 64)), SHAPE),
    (dict(q=_ck(4, 64, codes=None)), NULL), (dict(q=_ck(4, 40), cols=40), SHAPE),
    (dict(amax=(1 << 20) + 2), ALIGN), (dict(ws=P(9), n=8), WORKSPACE)])
def test_rmsnorm_fwd_refusals(lib, o, code):
    n = lib.fp4_kernel_launches()
    assert _fwd(lib, **o) == code
    assert lib.fp4_kernel_launches() == n


def _bwd(lib, **o):
    ws, n = o.pop("ws", None), o.pop("n", 0)
    a = dict(dy=P(1), lddy=64, s=P(2), lds=64, q=0, rstd=P(3), w=P(4), dres=0, lddr=0, dx=P(5), lddx=64,
             dw=0, rows=4, cols=64, st=0, wt=0, gt=0)
    a.update(o)
    return lib.fqt_rmsnorm_bwd(F._BWD(*a.values()), ws, n, None)


@pytest.mark.parametrize("o,code", [
    (dict(dy=0), NULL), (dict(s=0), NULL), (dict(rstd=0), NULL), (dict(dx=0), NULL),
    (dict(w=0), NULL), (dict(q=_ck(4, 64)), FORMAT), (dict(s=0, q=_ck(4, 32)), SHAPE),
    (dict(st=3), FORMAT), (dict(gt=3), FORMAT), (dict(dres=P(6), lddr=60), SHAPE),
    (dict(dw=P(6)), WORKSPACE), (dict(dw=P(6), ws=P(9), n=256), WORKSPACE),
    (dict(dw=P(6), ws=P(9), n=256 + 4 * 64 * 4 - 1), WORKSPACE),
    (dict(dw=(1 << 20) + 1, ws=P(9), n=1 << 20), ALIGN)])
def test_rmsnorm_bwd_refusals(lib, o, code):
    assert _bwd(lib, **o) == code


def _afwd(lib, **o):
    ws, n = o.pop("ws", None), o.pop("n", 0)
    a = dict(z=P(1), ldz=128, zi=0, y=P(2), ldy=64, zo=0, amax=0, rows=4, cols=64, act=4, gated=1)
    a.update(o)
    return lib.fqt_act_fwd(F._ACT_FWD(*a.values()), ws, n, None)


@pytest.mark.parametrize("o,code", [
    (dict(z=0), NULL), (dict(y=0), NULL), (dict(y=0, zo=_ck(4, 128), amax=P(6)), NULL),
    (dict(act=5), FORMAT), (dict(act=-1), FORMAT), (dict(zi=_ck(4, 128)), FORMAT),
    (dict(z=0, zi=_ck(4, 64)), SHAPE), (dict(z=0, zi=_ck(4, 128), zo=_ck(4, 128)), FORMAT),
    (dict(ldz=120), SHAPE), (dict(cols=60), SHAPE), (dict(rows=-2), SHAPE),
    (dict(cols=48, ldz=96, zo=_ck(4, 96)), SHAPE),          # a block would span both halves
    (dict(z=0, cols=48, zi=_ck(4, 96)), SHAPE),
    (dict(z=(1 << 20) + 8), ALIGN), (dict(ws=P(9), n=255), WORKSPACE)])
def test_act_fwd_refusals(lib, o, code):
    assert _afwd(lib, **o) == code


def _abwd(lib, **o):
    ws, n = o.pop("ws", None), o.pop("n", 0)
    a = dict(dy=P(1), lddy=64, z=P(2), ldz=128, q=0, dz=P(3), lddz=128, db=0, amax=0, rows=4, cols=64,
             act=4, gated=1)
    a.update(o)
    return lib.fqt_act_bwd(F._ACT_BWD(*a.values()), ws, n, None)


@pytest.mark.parametrize("o,code", [
    (dict(dy=0), NULL), (dict(z=0), NULL), (dict(dz=0), NULL), (dict(lddz=64), SHAPE),
    (dict(act=9), FORMAT), (dict(q=_ck(4, 128)), FORMAT), (dict(z=0, q=_ck(3, 128)), SHAPE),
    (dict(db=P(6)), WORKSPACE), (dict(db=P(6), ws=P(9), n=256 + 4 * 128 * 4 - 1), WORKSPACE)])
def test_act_bwd_refusals(lib, o, code):
    assert _abwd(lib, **o) == code


def _q(rows, cols, fmt=0):
    return C.byref(F.QTensorC(C.c_void_p(4096), C.c_void_p(4096), C.c_void_p(4096), C.c_void_p(4096),
                              C.c_void_p(4100), rows, cols, fmt, 0))


def _epi(lib, a=(128, 128), b=(256, 128), c=P(1), ldc=256, out=0, ws=P(9), n=256, none=False, **o):
    e = dict(bias=0, residual=0, ld_residual=0, z8=0, act=0, bias_dtype=0, residual_dtype=0)
    e.update(o)
    return lib.fp4_gemm_epi(_q(*a), _q(*b), 1.0, None if none else F._EPI(*e.values()), c, ldc, out, None, ws, n,
                            None)


@pytest.mark.parametrize("o,code", [
    (dict(none=True), NULL), (dict(c=None), NULL), (dict(a=(96, 128)), SHAPE), (dict(b=(256, 64)), SHAPE),
    (dict(act=5), FORMAT), (dict(out=2), FORMAT), (dict(ws=None), WORKSPACE), (dict(ldc=200), ALIGN),
    (dict(bias=2 << 20, bias_dtype=2), FORMAT), (dict(bias=(2 << 20) + 2), ALIGN),
    (dict(residual=2 << 20, ld_residual=128), SHAPE), (dict(residual=2 << 20, ld_residual=260), ALIGN),
    (dict(residual=2 << 20, ld_residual=256, residual_dtype=-1), FORMAT),
    (dict(z8=_ck(128, 128)), SHAPE),
    (dict(z8=_ck(128, 256, codes=None)), NULL)])
def test_gemm_epi_refusals(lib, o, code):
    n = lib.fp4_kernel_launches()
    assert _epi(lib, **o) == code
    assert lib.fp4_kernel_launches() == n


def test_missing_arguments(lib):
    for f in (lib.fqt_rmsnorm_fwd, lib.fqt_rmsnorm_bwd, lib.fqt_act_fwd, lib.fqt_act_bwd):
        assert f(None, None, 0, None) == NULL


def test_size_helpers(lib):
    a, b = C.c_size_t(), C.c_size_t()
    lib.fqt_ckpt8_sizes(3, 96, C.byref(a), C.byref(b))
    assert (a.value, b.value) == (288, 9)
    assert lib.fqt_colsum_workspace_bytes(0, 4096) == 256
    assert lib.fqt_colsum_workspace_bytes(5, 4096) == 256 + 5 * 4096 * 4
    assert lib.fqt_colsum_workspace_bytes(1 << 40, 4096) == lib.fqt_colsum_workspace_bytes(1 << 20, 4096)
    q = F.Ckpt8.empty(3, 96, device="cpu")
    assert q.codes.shape == (3, 96) and q.scales.shape == (3, 3)
    for cols in (0, 40, -32):
        with pytest.raises(ValueError):
            F.Ckpt8.empty(3, cols, device="cpu")


def test_binding_checks_tensors(lib):
    """The binding refuses tensors whose shape, type, layout or device would
    make the kernels read or write elsewhere."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, y = torch.ones(64), torch.zeros(4, 64, dtype=torch.bfloat16)
    bad = [dict(x=x.float()), dict(weight=torch.ones(32)), dict(weight=torch.ones(128)[::2]),
           dict(y=y[:3]), dict(y=y.t().contiguous().t()), dict(residual=x), dict(q8=F.Ckpt8.empty(4, 32, "cpu")),
           dict(residual=x, res_out=x.float()), dict(rstd=torch.zeros(3)), dict(x=x[0]), dict()]
    for o in bad:                                   # the last: CPU tensors at all
        with pytest.raises(ValueError):
            F.fqt_rmsnorm_fwd(**{**dict(x=x, weight=w, y=y), **o})
    rstd, dx = torch.ones(4), torch.zeros(4, 64, dtype=torch.bfloat16)
    for o in [dict(s=None), dict(xhat8=F.Ckpt8.empty(4, 64, "cpu")), dict(dres=x.float()),
              dict(dweight=torch.zeros(32)), dict(dx=dx[:, :32])]:
        with pytest.raises(ValueError):
            F.fqt_rmsnorm_bwd(**{**dict(dy=x, weight=w, rstd=rstd, dx=dx, s=x), **o})
    for o in [dict(z=x[:, :63], gated=True), dict(y=y[:, :32]), dict(z=x[0]), dict(z8=F.Ckpt8.empty(3, 64, "cpu"))]:
        with pytest.raises(ValueError):
            F.fqt_act_fwd(**{**dict(z=x, y=y), **o})
    for o in [dict(dz=y[:2]), dict(z=x[:, :32]), dict(dbias=torch.zeros(32)), dict(gated=True)]:
        with pytest.raises(ValueError):
            F.fqt_act_bwd(**{**dict(dy=x, z=x, dz=y), **o})


@pytest.mark.parametrize("cols", [1 << 62, (1 << 62) + 64, (1 << 29) + 32, (1 << 63) - 64])
def test_row_lengths_past_the_limit_are_refused(lib, cols):
    """Twice a row length beyond 2^62 is not a 64-bit number."""
    wide = dict(cols=cols, ldz=(1 << 63) - 8, ldy=(1 << 63) - 8)
    assert _afwd(lib, **wide) == SHAPE and _afwd(lib, **wide, zo=_ck(4, -(1 << 63))) == SHAPE
    wide = dict(cols=cols, ldz=(1 << 63) - 8, lddy=(1 << 63) - 8, lddz=(1 << 63) - 8)
    assert _abwd(lib, **wide) == SHAPE
