"""The calls between two FP4 linears against their 64-bit references: RMS norm
forward and backward, activations with 8-bit checkpoints forward, recomputed
and backward, the GEMM with an epilogue; their layouts, streams, captures and
a block run with all of them.

Tolerances count roundings: half a step of the output's type (2^-8 BF16, 2^-24
FP32, relative), plus the FP32 arithmetic's, which each test states."""
import ctypes

import numpy as np
import pytest
import torch

import block_ref as R
from block_ref import EPS16, EPS32, f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
STEP = {BF16: EPS16, F32: EPS32}
TINY = 2.0 ** -133              # BF16's and more than FP32's smallest step


def rand(*shape, seed, std=1.0, mean=0.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def padded(t, pad=8, fill=7.0):
    """t inside a wider buffer; the padding's values are to stay."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf, buf[:, :t.shape[1]]


# --------------------------------------------------------------------------
# RMS norm
# --------------------------------------------------------------------------
NORM_SHAPES = [(1, 8), (3, 64), (5, 72), (7, 128), (2, 136), (33, 256), (9, 264), (4, 512), (17, 1000),
               (9, 1024), (6, 1032), (300, 1056), (1, 4096), (401, 4096), (2, 4104), (5, 8192), (500, 8200),
               (350, 16384), (4, 12296), (1201, 96), (5000, 2056)]


def _norm_inputs(rows, cols, residual, weight, seed=0):
    x = rand(rows, cols, seed=seed)
    x[:, : max(1, cols // 50)] *= 20
    r = rand(rows, cols, seed=seed + 1, std=3.0, dtype=TYPES[residual]) if residual else None
    w = rand(cols, seed=seed + 2, std=0.2, mean=1.0, dtype=TYPES[weight])
    return x, r, w


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("residual,weight", [(None, "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_rmsnorm_fwd(gpu_lib, rows, cols, residual, weight):
    F = gpu_lib
    eps = 1e-5
    x, r, w = _norm_inputs(rows, cols, residual, weight)
    ybuf, y = padded(torch.zeros(rows, cols, dtype=BF16, device="cuda"))
    _, xs = padded(x, 16)
    rbuf, res = padded(torch.zeros_like(r), 24) if residual else (None, None)
    rstd, amax = torch.zeros(rows, device="cuda"), torch.full((1,), 9e9, device="cuda")
    ws = F.Workspace()
    F.fqt_rmsnorm_fwd(xs, w, y, residual=padded(r)[1] if residual else None, res_out=res, rstd=rstd, y_amax=amax, eps=eps, ws=ws)
    s, rs, xhat, want = R.rmsnorm(f64(x), f64(r) if residual else None, f64(w), eps)
    if residual:                     # FP32's nearest of the exact sum, then the type's
        assert torch.equal(res, (x.float() + r.float()).to(r.dtype)) and (rbuf[:, cols:] == 7.0).all()
    # rstd: a sum of squares whose every addition is in a chain of at most 64
    # (a tree over threads on top of 32 in one), halved by the root, and two
    # units of rsqrt; y: two products more
    assert (np.abs(f64(rstd) - rs) <= 48 * EPS32 * rs).all()
    R.assert_within(f64(y), want, np.abs(want) * (EPS16 + 56 * EPS32) + TINY, "y")
    assert float(amax) == float(y.float().abs().max())
    assert (ybuf[:, cols:] == 7.0).all()
    assert ws.status() == 0


@pytest.mark.parametrize("rows,cols", [s for s in NORM_SHAPES if s[1] % 32 == 0])
@pytest.mark.parametrize("of", ["y", "xhat"])
@pytest.mark.parametrize("with_y", [False, True])
def test_rmsnorm_fwd_checkpoint(gpu_lib, rows, cols, of, with_y):
    F = gpu_lib
    x, r, w = _norm_inputs(rows, cols, "bf16", "f32", seed=5)
    q8, ws = F.Ckpt8.empty(rows, cols), F.Workspace()
    q8.codes.fill_(255)
    q8.scales.fill_(77)
    y = torch.zeros_like(x) if with_y else None
    y2, q2 = torch.zeros_like(x), torch.zeros_like(r)
    F.fqt_rmsnorm_fwd(x, w, y, residual=r, res_out=r.clone(), q8=q8,
                      q8_of=F.RMS_XHAT if of == "xhat" else F.RMS_Y, eps=1e-5, ws=ws)
    _, _, xhat, want = R.rmsnorm(f64(x), f64(r), f64(w), 1e-5)
    R.assert_checkpoint(q8.codes, q8.scales, xhat if of == "xhat" else want, rel=56 * EPS32)
    if with_y:                                   # the same y as without a checkpoint
        F.fqt_rmsnorm_fwd(x, w, y2, residual=r, res_out=q2, eps=1e-5)
        assert torch.equal(y, y2)
    assert ws.status() == 0


def test_rmsnorm_fwd_in_place_and_amax_feed(gpu_lib):
    """res_out may be residual; y_amax is the amax that the quantizer finds."""
    F = gpu_lib
    x, r, w = _norm_inputs(160, 512, "f32", "f32", seed=9)
    y, y2, out = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(r)
    amax = torch.zeros(1, device="cuda")
    F.fqt_rmsnorm_fwd(x, w, y, residual=r, res_out=out, y_amax=amax)
    inplace = r.clone()
    F.fqt_rmsnorm_fwd(x, w, y2, residual=inplace, res_out=inplace)
    assert torch.equal(inplace, out) and torch.equal(y, y2)
    a, b = F.QTensor.empty(160, 512), F.QTensor.empty(160, 512)
    F.fp4_quantize(y, a)
    F.fp4_quantize(y, b, amax_in=amax)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert torch.equal(a.amax, amax) and torch.equal(a.s_dec, b.s_dec)


def test_rmsnorm_fwd_zero_and_nonfinite_rows(gpu_lib):
    F = gpu_lib
    x = rand(5, 64, seed=1)
    x[1] = 0
    x[2, 3], x[3, 40] = float("inf"), float("nan")
    w, y, ws = torch.ones(64, device="cuda"), torch.zeros_like(x), F.Workspace()
    q8, rstd, amax = F.Ckpt8.empty(5, 64), torch.zeros(5, device="cuda"), torch.zeros(1, device="cuda")
    F.fqt_rmsnorm_fwd(x, w, y, q8=q8, rstd=rstd, y_amax=amax, eps=1e-6, ws=ws)
    assert (y[1] == 0).all() and (q8.codes[1] == 0).all() and (q8.scales[1] == 0).all()
    assert abs(float(rstd[1]) - 1000.0) < 1e-3
    assert torch.isfinite(y[[0, 1, 4]].float()).all() and torch.isnan(y[3].float()).all()
    assert (q8.scales[3] == 255).all() and (q8.scales[[0, 4]] != 255).all()
    assert not np.isfinite(float(amax)) and ws.status() == 7


def test_no_rows(gpu_lib):
    F = gpu_lib
    e = lambda c, t=BF16: torch.zeros((0, c), dtype=t, device="cuda")
    one = lambda n, v=3.0: torch.full((n,), v, device="cuda")
    amax, dw, db = one(1), one(64), one(128)
    F.fqt_rmsnorm_fwd(e(64), one(64), e(64), q8=F.Ckpt8.empty(0, 64), rstd=one(0), y_amax=amax)
    F.fqt_rmsnorm_bwd(e(64), one(64), one(0), e(64), s=e(64), dweight=dw)
    assert float(amax) == 0 and (dw == 0).all()
    F.fqt_rmsnorm_fwd(e(64), one(64), e(64))
    amax.fill_(3)
    F.fqt_act_fwd(e(128), e(64), gated=True)
    F.fqt_act_fwd(e(128), e(64), gated=True, z8=F.Ckpt8.empty(0, 128))
    F.fqt_act_bwd(e(64), F.Ckpt8.empty(0, 128), e(128), gated=True, dbias=db, dz_amax=amax)
    assert float(amax) == 0 and (db == 0).all()


@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(9000, 64), (700, 8192)])
@pytest.mark.parametrize("saved,grad,dres,weight", [("bf16", "bf16", True, "bf16"), ("f32", "f32", True, "f32"),
                                                    ("ckpt", "bf16", False, "f32"),
                                                    ("ckpt", "f32", True, "bf16")])
def test_rmsnorm_bwd(gpu_lib, rows, cols, saved, grad, dres, weight):
    F = gpu_lib
    if saved == "ckpt" and cols % 32:
        pytest.skip("no checkpoint of this row length")
    s, _, w = _norm_inputs(rows, cols, None, weight, seed=20)
    s = s.to(TYPES["f32" if saved == "f32" else "bf16"])
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-5)
    dy = rand(rows, cols, seed=23, std=0.1)
    dr = rand(rows, cols, seed=24, std=0.1, dtype=TYPES[grad]) if dres else None
    kw = {"s": padded(s)[1]}
    xhat = f64(s) * f64(rstd)[:, None]
    if saved == "ckpt":
        q8 = F.Ckpt8.empty(rows, cols)
        F.fqt_act_fwd((s.float() * rstd[:, None]).to(BF16), act=F.ACT_NONE, z8=q8)
        kw, xhat = {"xhat8": q8}, R.decode(q8.codes, q8.scales)
    dxbuf, dx = padded(torch.zeros(rows, cols, dtype=TYPES[grad], device="cuda"))
    dw = torch.full((cols,), 5.0, device="cuda")
    ws = F.Workspace.colsum(rows, cols)
    F.fqt_rmsnorm_bwd(padded(dy, 24)[1], w, rstd, dx, dres=padded(dr, 40)[1] if dres else None, dweight=dw,
                      ws=ws, **kw)
    want, want_dw = R.rmsnorm_bwd(f64(dy), xhat, f64(rstd), f64(w), f64(dr) if dres else None)
    g, rs = f64(dy) * f64(w), f64(rstd)[:, None]
    # eight roundings along each term, a dot product with chains of at most 64 + 8
    # additions and products, half a step of the output
    m, ma = np.abs((g * xhat).mean(1, keepdims=True)), np.abs(g * xhat).mean(1, keepdims=True)
    bound = EPS32 * (8 * rs * (np.abs(g) + np.abs(xhat) * m) + 72 * rs * np.abs(xhat) * ma +
                     (2 * np.abs(f64(dr)) if dres else 0)) + STEP[TYPES[grad]] * np.abs(want) * 1.01 + TINY
    R.assert_within(f64(dx), want, bound, "dx")
    # rows in one chain per CTA (rows / 148), then chains of 32, 14 and 32
    chain = rows / 148 + 2 + 32 + 14 + 32
    R.assert_within(f64(dw), want_dw, EPS32 * chain * np.abs(f64(dy) * xhat).sum(0) + TINY, "dweight")
    assert (dxbuf[:, cols:] == 7.0).all()
    again = torch.zeros_like(dw)
    if dres:                                          # dx may be dres
        F.fqt_rmsnorm_bwd(dy, w, rstd, dr, dres=dr, dweight=again, ws=ws, **kw)
        assert torch.equal(dr, dx)
    else:
        F.fqt_rmsnorm_bwd(dy, w, rstd, dx, dweight=again, **kw)
    assert torch.equal(again, dw)                     # the same additions in the same order
    plain = torch.zeros_like(dx)
    F.fqt_rmsnorm_bwd(dy, w, rstd, plain, **kw)       # without dweight and workspace
    assert dres or torch.equal(plain, dx)


# --------------------------------------------------------------------------
# Activations and checkpoints
# --------------------------------------------------------------------------
def _act_of(F, kind):
    return {"none": F.ACT_NONE, "relu": F.ACT_RELU, "gelu": F.ACT_GELU, "gelu_tanh": F.ACT_GELU_TANH,
            "silu": F.ACT_SILU}[kind]


ACT_SHAPES = [(1, 32), (3, 64), (5, 96), (7, 8), (33, 40), (260, 1000), (2, 160), (7, 256), (33, 288), (600, 2080), (1, 11008), (37, 11008)]
WIDE = [0.0, -0.0, 1e-30, -1e-30, 0.5, -1.278, -5.0, 6.0, 9.5, -9.5, 30.0, -30.0, 80.0, -87.0, -100.0, 1e4,
        -1e4, 3e18, -3e18, 1e30, -1e30, 2.0 ** -133, 3.0, -3.0]


def _z(rows, zcols, seed):
    z = rand(rows, zcols, seed=seed, std=2.0)
    n = min(len(WIDE), z.numel())
    z.view(-1)[:n] = torch.tensor(WIDE[:n], device="cuda").to(BF16)
    return z


def _exact_ckpt(codes, scales):
    """Checkpoint of values as torch sees them: E4M3 times the power of two."""
    e = torch.ldexp(torch.ones_like(scales, dtype=torch.float64), scales.int() - 127)
    return codes.view(torch.float8_e4m3fn).double() * e.repeat_interleave(32, 1)


@pytest.mark.parametrize("rows,zcols", [s for s in ACT_SHAPES if s[1] % 32 == 0])
def test_checkpoint_encoding(gpu_lib, rows, zcols):
    """Encoding alone equals the 64-bit encoding of the BF16 values."""
    F = gpu_lib
    z = rand(rows, zcols, seed=3) * torch.exp2(
        torch.randint(-126, 118, (rows, zcols // 32), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(1)).float()
    ).repeat_interleave(32, 1).to(BF16)
    z[0, :32] = torch.arange(32, device="cuda").to(BF16) * 2.0 ** -133     # subnormal block
    if zcols >= 96:
        z[-1, 32:64] = 0
        z[-1, 64:96] = 448.0
        z[-1, 65:96:2] = torch.arange(16, device="cuda").to(BF16) / 64 + 1
    q8, ws = F.Ckpt8.empty(rows, zcols), F.Workspace()
    F.fqt_act_fwd(padded(z)[1], act=F.ACT_NONE, z8=q8, ws=ws)
    values, byte = R.encode(f64(z))
    assert np.array_equal(q8.scales.cpu().numpy(), byte)
    assert np.array_equal(R.code_values(q8.codes), values)
    assert ws.status() == 0
    y = torch.zeros_like(z)
    F.fqt_act_fwd(q8, y, act=F.ACT_NONE)
    assert torch.equal(y, _exact_ckpt(q8.codes, q8.scales).float().to(BF16))


def test_checkpoint_decoding_of_every_code_and_scale(gpu_lib):
    F = gpu_lib
    q8 = F.Ckpt8.empty(256, 256)
    q8.codes.copy_(torch.arange(256, device="cuda").to(torch.uint8).expand(256, 256))
    q8.scales.copy_(torch.arange(256, device="cuda").to(torch.uint8)[:, None].expand(256, 8))
    y = torch.zeros(256, 256, dtype=BF16, device="cuda")
    F.fqt_act_fwd(q8, y, act=F.ACT_NONE)
    want = _exact_ckpt(q8.codes, q8.scales).float()
    want[255] = float("nan")
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(y[ok], want.to(BF16)[ok])


def test_checkpoint_of_nonfinite_values(gpu_lib):
    """A block with Inf or NaN decodes to NaN as a whole and sets the status;
    its neighbours stay."""
    F = gpu_lib
    z = rand(4, 128, seed=2)
    z[1, 40], z[2, 127] = float("inf"), float("nan")
    q8, ws, y = F.Ckpt8.empty(4, 128), F.Workspace(), torch.zeros(4, 128, dtype=BF16, device="cuda")
    F.fqt_act_fwd(z, act=F.ACT_NONE, z8=q8, ws=ws)
    F.fqt_act_fwd(q8, y, act=F.ACT_NONE)
    nan = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    nan[1, 32:64] = nan[2, 96:] = True
    assert torch.equal(torch.isnan(y), nan) and ws.status() == 7


@pytest.mark.parametrize("rows,zcols", ACT_SHAPES)
@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("source", ["bf16", "ckpt"])
def test_act_fwd_bwd(gpu_lib, rows, zcols, kind, gated, source):
    F = gpu_lib
    if source == "ckpt" and zcols % 32:
        pytest.skip("no checkpoint of this row length")
    if gated:
        zcols *= 2
    cols, act = zcols // 2 if gated else zcols, _act_of(F, kind)
    zt = _z(rows, zcols, seed=30)
    z, arg, ws = f64(zt), padded(zt)[1], F.Workspace.colsum(rows, zcols)
    if source == "ckpt":
        arg = F.Ckpt8.empty(rows, zcols)
        F.fqt_act_fwd(zt, act=act, gated=gated, z8=arg)
        z = R.decode(arg.codes, arg.scales)
    ybuf, y = padded(torch.zeros(rows, cols, dtype=BF16, device="cuda"))
    amax = torch.zeros(1, device="cuda")
    F.fqt_act_fwd(arg, y, act=act, gated=gated, y_amax=amax, ws=ws)
    gate, up = (z[:, :cols], np.abs(z[:, cols:])) if gated else (z, np.ones_like(z))
    # products above FP32's range are Inf on both sides, near its top either
    top = 2.0 ** 127
    with np.errstate(over="ignore"):
        want = R.act_fwd(z, kind, gated)
    keep = np.abs(want) < top
    err = R.act_value_error(gate, kind) * up
    R.assert_within(f64(y)[keep], want[keep], (np.abs(want) * (EPS16 + 2.0 ** -20) + err + TINY)[keep], "y")
    assert float(amax) == float(y.float().abs().max())
    assert (ybuf[:, cols:] == 7.0).all()

    dy = rand(rows, cols, seed=31, std=1e-3)
    dzbuf, dz = padded(torch.zeros(rows, zcols, dtype=BF16, device="cuda"), 16)
    db = torch.full((zcols,), 4.0, device="cuda")
    F.fqt_act_bwd(padded(dy)[1], arg, dz, act=act, gated=gated, dbias=db, dz_amax=amax, ws=ws)
    want = R.act_bwd(f64(dy), z, kind, gated)
    a = np.abs(f64(dy))
    err = R.act_grad_error(gate, kind) * a * up
    if gated:
        err = np.concatenate([err, R.act_value_error(gate, kind) * a], 1)
    R.assert_within(f64(dz), want, np.abs(want) * (EPS16 + 2.0 ** -20) + err + TINY, "dz")
    assert float(amax) == float(dz.float().abs().max())
    assert (dzbuf[:, zcols:] == 7.0).all()
    # chains: rows of a thread, 32 rows of the CTA, 14 and 32 slices
    chain = rows / 4 + 32 + 14 + 32
    bound = (err + np.abs(want) * EPS32 * (chain + 4)).sum(0) + TINY
    R.assert_within(f64(db), want.sum(0), bound, "dbias")
    again = torch.zeros_like(db)
    F.fqt_act_bwd(dy, arg, dz, act=act, gated=gated, dbias=again)
    assert torch.equal(again, db)
    if not gated:                                     # dz may be dy, or z
        same = dy.clone()
        F.fqt_act_bwd(same, arg, same, act=act)
        assert torch.equal(same, dz)
    if source == "bf16":
        same = zt.clone()
        F.fqt_act_bwd(dy, same, same, act=act, gated=gated)
        assert torch.equal(same, dz)


@pytest.mark.parametrize("kind", R.ACTS)
def test_activations_of_nonfinite_values(gpu_lib, kind):
    """NaN stays NaN, +Inf stays Inf, neighbours are as without them; the amax
    shows both."""
    F = gpu_lib
    act, z = _act_of(F, kind), rand(3, 256, seed=6)
    y, want, amax = torch.zeros_like(z), torch.zeros_like(z), torch.zeros(1, device="cuda")
    F.fqt_act_fwd(z, want, act=act)
    bad = z.clone()
    bad[0, 7], bad[2, 100] = float("nan"), float("inf")
    F.fqt_act_fwd(bad, y, act=act, y_amax=amax)
    assert torch.isnan(y[0, 7]) and torch.isinf(y[2, 100]) and torch.isnan(amax)
    y[0, 7], y[2, 100] = want[0, 7], want[2, 100]
    assert torch.equal(y, want)
    F.fqt_act_bwd(z, bad, y, act=act, dz_amax=amax)
    F.fqt_act_bwd(z, z, want, act=act)
    keep = torch.ones_like(z, dtype=torch.bool)
    keep[0, 7] = keep[2, 100] = False
    assert torch.equal(y[keep], want[keep])
    assert kind == "none" or torch.isnan(y[0, 7])


def test_act_fwd_with_checkpoint_gives_both(gpu_lib):
    F = gpu_lib
    z = _z(45, 1024, seed=4)
    y, y2, q, q2 = (torch.zeros(45, 512, dtype=BF16, device="cuda"),
                    torch.zeros(45, 512, dtype=BF16, device="cuda"), F.Ckpt8.empty(45, 1024), F.Ckpt8.empty(45, 1024))
    F.fqt_act_fwd(z, y, gated=True, z8=q)
    F.fqt_act_fwd(z, y2, gated=True)
    F.fqt_act_fwd(z, gated=True, z8=q2)
    assert torch.equal(y, y2) and torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)


# --------------------------------------------------------------------------
# GEMM with an epilogue
# --------------------------------------------------------------------------
def _operands(F, m, n, k, fmt, seed=0):
    qa, qb = F.QTensor.empty(m, k, fmt), F.QTensor.empty(n, k, fmt)
    F.fp4_quantize(rand(m, k, seed=seed), qa, fmt=fmt)
    F.fp4_quantize(rand(n, k, seed=seed + 1, std=k ** -0.5), qb, fmt=fmt)
    return qa, qb


@pytest.mark.parametrize("mnk", [(128, 128, 64), (256, 384, 320), (384, 640, 1856), (1280, 2176, 192)])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("kind", R.ACTS)
@pytest.mark.parametrize("out,bias,residual,ckpt", [
    ("bf16", "bf16", "bf16", True), ("f32", "f32", "f32", True), ("bf16", None, "f32", False),
    ("f32", "bf16", None, False), ("bf16", None, None, True)])
def test_gemm_epi(gpu_lib, mnk, fmt, kind, out, bias, residual, ckpt):
    """Against the 64-bit epilogue of the FP32 product that fp4_gemm stores; the
    last size has enough tiles for the wide ones."""
    F = gpu_lib
    m, n, k = mnk
    qa, qb = _operands(F, m, n, k, fmt)
    prod = torch.zeros(m, n, device="cuda")
    F.fp4_gemm(qa, qb, prod, alpha=1.5)
    b = rand(n, seed=5, std=0.5, dtype=TYPES[bias]) if bias else None
    r = rand(m, n, seed=6, dtype=TYPES[residual]) if residual else None
    z8 = F.Ckpt8.empty(m, n) if ckpt else None
    cbuf, c = padded(torch.zeros(m, n, dtype=TYPES[out], device="cuda"), 16)
    amax, ws = torch.zeros(1, device="cuda"), F.Workspace(m, n, k)
    F.fp4_gemm_epi(qa, qb, c, alpha=1.5, bias=b, act=_act_of(F, kind), residual=padded(r)[1] if residual else None,
                   z8=z8, c_amax=amax, ws=ws)
    # z as the kernel forms it: one FP32 addition to the product
    z = f64(prod + b.float()) if bias else f64(prod)
    v = R.act(z, kind)[0]
    want = v + f64(r) if residual else v
    bound = STEP[TYPES[out]] * np.abs(want) * 1.01 + R.act_value_error(z, kind) + EPS32 * (np.abs(v) + np.abs(want)) + TINY
    R.assert_within(f64(c), want, bound, "C")
    if ckpt:
        values, byte = R.encode(z)
        assert np.array_equal(z8.scales.cpu().numpy(), byte)
        assert np.array_equal(R.code_values(z8.codes), values)
    top = np.abs(want).max()
    assert abs(float(amax) - top) <= top * 2.0 ** -15
    assert (cbuf[:, n:] == 7.0).all() and ws.status() == 0


@pytest.mark.parametrize("m,n,k", [(256, 384, 512), (128, 4096, 4096), (1280, 2176, 320)])
def test_gemm_epi_without_epilogue_is_the_gemm(gpu_lib, m, n, k):
    F = gpu_lib
    qa, qb = _operands(F, m, n, k, 0)
    for t in (BF16, F32):
        a, b = torch.zeros(m, n, dtype=t, device="cuda"), torch.zeros(m, n, dtype=t, device="cuda")
        am, bm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
        F.fp4_gemm(qa, qb, a, c_amax=am)
        F.fp4_gemm_epi(qa, qb, b, c_amax=bm)
        assert torch.equal(a, b) and torch.equal(am, bm)


@pytest.mark.parametrize("m,n", [(256, 384), (1280, 2176)])
def test_gemm_epi_of_least_alignment(gpu_lib, m, n):
    """Rows and codes aligned to 16 bytes and no more give what aligned ones give."""
    F = gpu_lib
    qa, qb = _operands(F, m, n, 192, 0)
    bias = rand(n, seed=1, dtype=F32)
    for t, pad in ((BF16, 8), (F32, 4)):
        r = rand(m, n, seed=2, dtype=t)
        want, q = torch.zeros(m, n, dtype=t, device="cuda"), F.Ckpt8.empty(m, n)
        F.fp4_gemm_epi(qa, qb, want, bias=bias, act=F.ACT_SILU, residual=r, z8=q)
        buf = torch.zeros(m * n + 16, dtype=torch.uint8, device="cuda")
        codes, scales = buf[16:].view(m, n), torch.zeros_like(q.scales)
        c = F.Ckpt8C(codes.data_ptr(), scales.data_ptr(), m, n)
        q2 = F.Ckpt8(m, n, codes, scales, c, ctypes.addressof(c))
        cbuf, out = padded(torch.zeros(m, n, dtype=t, device="cuda"), pad)
        F.fp4_gemm_epi(qa, qb, out, bias=bias, act=F.ACT_SILU, residual=padded(r, pad)[1], z8=q2)
        assert torch.equal(out, want) and (cbuf[:, n:] == 7.0).all()
        assert torch.equal(codes, q.codes) and torch.equal(scales, q.scales) and (buf[:16] == 0).all()


@pytest.mark.parametrize("m,n", [(256, 256), (1280, 2176)])
def test_gemm_epi_residual_in_place(gpu_lib, m, n):
    F = gpu_lib
    qa, qb = _operands(F, m, n, 256, 1)
    for t in (BF16, F32):
        r = rand(m, n, seed=8, dtype=t)
        c = torch.zeros_like(r)
        F.fp4_gemm_epi(qa, qb, c, act=F.ACT_SILU, residual=r)
        F.fp4_gemm_epi(qa, qb, r, act=F.ACT_SILU, residual=r)
        assert torch.equal(r, c)


def test_gemm_epi_nonfinite(gpu_lib):
    F = gpu_lib
    qa, qb = _operands(F, 128, 256, 128, 0)
    bias = torch.zeros(256, device="cuda")
    bias[70] = float("inf")
    z8, ws, c = F.Ckpt8.empty(128, 256), F.Workspace(), torch.zeros(128, 256, dtype=BF16, device="cuda")
    F.fp4_gemm_epi(qa, qb, c, bias=bias, z8=z8, ws=ws)
    assert torch.isinf(c[:, 70]).all() and torch.isfinite(c[:, :70]).all()
    assert (z8.scales[:, 2] == 255).all() and (z8.scales[:, [0, 1, 3, 4, 5, 6, 7]] != 255).all()
    assert ws.status() == 7


# --------------------------------------------------------------------------
# Offsets past 32 bits, streams, captures
# --------------------------------------------------------------------------
def test_offsets_past_32_bits(gpu_lib):
    """Rows that start beyond element 2^31 (and byte 2^32), by leading
    dimension and by the number of rows."""
    F = gpu_lib
    ld = (1 << 30) + 8
    buf = torch.zeros(2 * ld + 4096, dtype=BF16, device="cuda")
    x = buf.as_strided((3, 256), (ld, 1))
    x.copy_(rand(3, 256, seed=1))
    w, y = torch.ones(256, device="cuda"), torch.zeros(3, 256, dtype=BF16, device="cuda")
    F.fqt_rmsnorm_fwd(x, w, y)
    want = torch.zeros_like(y)
    F.fqt_rmsnorm_fwd(x.contiguous(), w, want)
    assert torch.equal(y, want)
    F.fqt_act_fwd(x, y)
    F.fqt_act_fwd(x.contiguous(), want)
    assert torch.equal(y, want)
    del buf, x
    rows, cols = (1 << 31) // 16384 + 2, 16384
    q8 = F.Ckpt8.empty(rows, cols)
    q8.codes.zero_()
    q8.scales.fill_(127)
    q8.codes[-1] = 0x38                                # 1.0
    y = torch.full((rows, cols), 5.0, dtype=BF16, device="cuda")
    F.fqt_act_fwd(q8, y, act=F.ACT_NONE)
    assert (y[-1] == 1).all() and (y[-2] == 0).all() and float(y.abs().max()) == 1
    dx, rstd = y, torch.ones(rows, device="cuda")
    dy = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    dy[-1] = 2
    dw = torch.zeros(cols, device="cuda")
    F.fqt_rmsnorm_bwd(dy, torch.ones(cols, device="cuda"), rstd, dx, xhat8=q8, dweight=dw)
    assert (dw == 2).all() and (dx[-1] == 0).all() and (dx[-2] == 0).all()


def test_gemm_epi_offsets_past_32_bits(gpu_lib):
    """Output and checkpoint rows beyond element 2^32 are those of a product of
    the last rows alone."""
    F = gpu_lib
    m, n, k = (1 << 20) + 128, 4096, 64
    x, w = rand(m, k, seed=1), rand(n, k, seed=2)
    amax = x.float().abs().max().reshape(1)
    qa, qb, ql = F.QTensor.empty(m, k), F.QTensor.empty(n, k), F.QTensor.empty(128, k)
    F.fp4_quantize(x, qa, amax_in=amax)
    F.fp4_quantize(x[-128:], ql, amax_in=amax)
    F.fp4_quantize(w, qb)
    c, z8 = torch.zeros(m, n, dtype=BF16, device="cuda"), F.Ckpt8.empty(m, n)
    res, bias = c, rand(n, seed=3)                     # the residual in place: zeros
    F.fp4_gemm_epi(qa, qb, c, bias=bias, act=F.ACT_GELU, residual=res, z8=z8)
    want, z = torch.zeros(128, n, dtype=BF16, device="cuda"), F.Ckpt8.empty(128, n)
    F.fp4_gemm_epi(ql, qb, want, bias=bias, act=F.ACT_GELU, z8=z)
    assert torch.equal(c[-128:], want)
    assert torch.equal(z8.codes[-128:], z.codes) and torch.equal(z8.scales[-128:], z.scales)


def test_explicit_stream(gpu_lib):
    """stream=: ordered after that stream's earlier work, not the current one's."""
    F = gpu_lib
    s, x, y = torch.cuda.Stream(), rand(64, 4096, seed=1), torch.zeros(64, 4096, dtype=BF16, device="cuda")
    want = torch.zeros_like(y)
    F.fqt_act_fwd(x, want, act=F.ACT_GELU)
    src, big = torch.zeros_like(x), torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            big.add_(1.0)
        src.copy_(x)
    F.fqt_act_fwd(src, y, act=F.ACT_GELU, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("rows,cols", [(3, 4096), (600, 1024), (4099, 128)])
def test_calls_in_a_row_see_one_another(gpu_lib, rows, cols):
    """Launches overlap the end of the kernel before them, so: a chain in which
    every call reads what the one before wrote and writes what it read, with
    other kernels in between, gives what it gives with a wait after each."""
    F = gpu_lib
    w = rand(cols, seed=1, std=0.1, mean=1.0, dtype=F32)
    qa, qb = _operands(F, 128, 256, 128, 0)

    def chain(wait):
        x, r = rand(rows, cols, seed=2), rand(rows, cols, seed=3)
        y, dx, q8 = torch.zeros_like(x), torch.zeros_like(x), F.Ckpt8.empty(rows, cols)
        rstd, dw, db = (torch.zeros(n, device="cuda") for n in (rows, cols, cols))
        c, z8 = rand(128, 256, seed=4), F.Ckpt8.empty(128, 256)
        amax, ws = torch.zeros(1, device="cuda"), F.Workspace.colsum(rows, cols)
        total = torch.zeros(cols, device="cuda")
        steps = [
            lambda: F.fqt_rmsnorm_fwd(x, w, y, residual=r, res_out=r, q8=q8, q8_of=F.RMS_XHAT, rstd=rstd, ws=ws),
            lambda: F.fqt_act_fwd(y, x, act=F.ACT_GELU, z8=q8),
            lambda: F.fqt_act_bwd(x, q8, y, act=F.ACT_GELU, dbias=db, dz_amax=amax, ws=ws),
            lambda: F.fqt_rmsnorm_bwd(y, w, rstd, dx, s=r, dres=x, dweight=dw, ws=ws),
            lambda: total.add_(dw).add_(db),
            lambda: F.fqt_rmsnorm_bwd(dx, w, rstd, dx2, xhat8=q8, dweight=dw, ws=ws),
            lambda: F.fqt_act_fwd(dx2, x, act=F.ACT_SILU),
            lambda: F.fp4_gemm_epi(qa, qb, c, alpha=0.01, residual=c, z8=z8),
            lambda: F.fqt_act_fwd(z8, c, act=F.ACT_GELU_TANH),
            lambda: F.fp4_gemm_epi(qa, qb, c, alpha=0.01, act=F.ACT_SILU, residual=c),
            lambda: r.mul_(0.5),
        ]
        dx2 = torch.zeros_like(x)
        for _ in range(25):
            for step in steps:
                step()
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x, y, r, dx, c, total, dw, db, amax, q8.codes, z8.codes

    want = chain(True)
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))


def _block(F, st):
    """A feed-forward block of a transformer, forward and backward: norm of
    the residual stream with an 8-bit checkpoint, up projection with bias and
    GELU and its checkpoint, down projection with bias onto the stream."""
    M, H, N, ws = st["M"], st["H"], st["N"], st["ws"]
    F.fqt_rmsnorm_fwd(st["x"], st["g"], st["y"], residual=st["r"], res_out=st["s"], q8=st["xhat8"],
                      q8_of=F.RMS_XHAT, rstd=st["rstd"], y_amax=st["amax"], eps=1e-5, ws=ws)
    F.fp4_quantize(st["y"], st["yq"], st["yq_t"], amax_in=st["amax"], amax_in_t=st["amax"], ws=ws)
    F.fp4_quantize(st["w1"], st["w1q"], st["w1q_t"], block=F.BLOCK_2D, ws=ws)
    F.fp4_gemm_epi(st["yq"], st["w1q"], st["h"], bias=st["b1"], act=F.ACT_GELU, z8=st["z8"], ws=ws)
    F.fp4_quantize(st["h"], st["hq"], st["hq_t"], ws=ws)
    F.fp4_quantize(st["w2"], st["w2q"], st["w2q_t"], block=F.BLOCK_2D, ws=ws)
    F.fp4_gemm_epi(st["hq"], st["w2q"], st["o"], bias=st["b2"], residual=st["s"], ws=ws)
    # backward
    F.fp4_quantize(st["do"], st["doq"], st["doq_t"], ws=ws)
    F.fp4_gemm(st["doq"], st["w2q_t"], st["dh"], ws=ws)
    F.fp4_gemm(st["doq_t"], st["hq_t"], st["dw2"], ws=ws)
    F.fqt_act_bwd(st["dh"], st["z8"], st["dz"], act=F.ACT_GELU, dbias=st["db1"], dz_amax=st["amax2"], ws=ws)
    F.fp4_quantize(st["dz"], st["dzq"], st["dzq_t"], amax_in=st["amax2"], amax_in_t=st["amax2"], ws=ws)
    F.fp4_gemm(st["dzq"], st["w1q_t"], st["dy"], ws=ws)
    F.fp4_gemm(st["dzq_t"], st["yq_t"], st["dw1"], ws=ws)
    F.fqt_rmsnorm_bwd(st["dy"], st["g"], st["rstd"], st["dx"], xhat8=st["xhat8"], dres=st["do"],
                      dweight=st["dg"], ws=ws)


def _block_state(F, M=256, H=256, N=512, seed=50):
    t = lambda *s, k, std=1.0, dtype=BF16: rand(*s, seed=seed + k, std=std, dtype=dtype)
    e = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device="cuda")
    q = lambda a, b, blk=0: (F.QTensor.empty(a, b, 0, blk), F.QTensor.empty(b, a, 0, blk))
    st = dict(M=M, H=H, N=N, ws=F.Workspace.colsum(M, max(N, H)),
              x=t(M, H, k=1), r=t(M, H, k=2, std=2.0), g=rand(H, seed=seed + 3, std=0.1, mean=1.0, dtype=F32),
              w1=t(N, H, k=4, std=H ** -0.5), b1=t(N, k=5, std=0.2), w2=t(H, N, k=6, std=N ** -0.5),
              b2=t(H, k=7, std=0.2, dtype=F32), do=t(M, H, k=8, std=1e-2),
              y=e(M, H), s=e(M, H), rstd=e(M, dtype=F32), amax=e(1, dtype=F32), amax2=e(1, dtype=F32),
              xhat8=F.Ckpt8.empty(M, H), z8=F.Ckpt8.empty(M, N), h=e(M, N), o=e(M, H), dh=e(M, N), dz=e(M, N),
              dy=e(M, H), dx=e(M, H), dw1=e(N, H, dtype=F32), dw2=e(H, N, dtype=F32), db1=e(N, dtype=F32),
              dg=e(H, dtype=F32))
    for name, shape, blk in (("y", (M, H), 0), ("w1", (N, H), 1), ("h", (M, N), 0), ("w2", (H, N), 1),
                             ("do", (M, H), 0), ("dz", (M, N), 0)):
        st[name + "q"], st[name + "q_t"] = q(*shape, blk)
    return st


def _deq(q):
    lut = np.array([0, .5, 1, 1.5, 2, 3, 4, 6] + [-0., -.5, -1, -1.5, -2, -3, -4, -6])
    b = q.codes_2d().cpu().numpy()
    v = lut[np.stack([b & 15, b >> 4], -1).reshape(q.rows, q.cols)]
    sc = q.scales_2d().cpu().view(torch.float8_e4m3fn).double().numpy()
    sc = np.repeat(np.repeat(sc, 16, 1), 16, 0) if q.block else np.repeat(sc, 16, 1)
    return v * sc * float(q.s_dec)


OUTPUTS = ("s", "o", "dx", "dw1", "dw2", "db1", "dg", "dz")


def test_block_run(gpu_lib):
    """Each step of the block in 64 bits, from the operands as the run left
    them (its quantized tensors and checkpoints), within its own roundings."""
    F = gpu_lib
    st = _block_state(F)
    _block(F, st)
    assert st["ws"].status() == 0
    s, rstd, xhat, y = R.rmsnorm(f64(st["x"]), f64(st["r"]), f64(st["g"]), 1e-5)
    R.assert_within(f64(st["y"]), y, np.abs(y) * (EPS16 + 56 * EPS32) + TINY, "y")
    P = _deq(st["yq"]) @ _deq(st["w1q"]).T
    # the tensor cores' FP32 sums: 1e-6 of the sum of magnitudes is four units
    # of FP32 for each of the 16 accumulations of a K of 256
    acc = 1e-6 * (np.abs(_deq(st["yq"])) @ np.abs(_deq(st["w1q"])).T)
    z = P + f64(st["b1"])
    h = R.act(z, "gelu")[0]
    R.assert_within(f64(st["h"]), h, np.abs(h) * EPS16 + 1.2 * acc + R.act_value_error(z, "gelu") + TINY, "h")
    o = _deq(st["hq"]) @ _deq(st["w2q"]).T + f64(st["b2"]) + f64(st["s"])
    acc2 = 1e-6 * (np.abs(_deq(st["hq"])) @ np.abs(_deq(st["w2q"])).T + np.abs(f64(st["s"])) + 1)
    R.assert_within(f64(st["o"]), o, np.abs(o) * EPS16 + acc2, "o")
    z8 = R.decode(st["z8"].codes, st["z8"].scales)
    assert np.linalg.norm(z8 - z) < 2.0 ** -4 * np.linalg.norm(z)
    dz = R.act_bwd(f64(st["dh"]), z8, "gelu", False)
    R.assert_within(f64(st["dz"]), dz, np.abs(dz) * EPS16 + np.abs(f64(st["dh"])) * R.act_grad_error(z8, "gelu") + TINY, "dz")
    assert np.abs(f64(st["db1"]) - dz.sum(0)).max() <= 1e-5 * np.abs(dz).sum(0).max()
    xh = R.decode(st["xhat8"].codes, st["xhat8"].scales)
    assert np.linalg.norm(xh - xhat) < 2.0 ** -4 * np.linalg.norm(xhat)
    dx, dg = R.rmsnorm_bwd(f64(st["dy"]), xh, f64(st["rstd"]), f64(st["g"]), f64(st["do"]))
    assert np.abs(f64(st["dx"]) - dx).max() <= EPS16 * 1.02 * np.abs(dx).max()
    assert np.abs(f64(st["dg"]) - dg).max() <= 1e-5 * np.abs(f64(st["dy"]) * xh).sum(0).max()
    # against the unquantized block: operands of 4 bits are off by 10 to 15 %
    # each, the products by their root sum of squares, two products deep; a
    # wrong or missing gradient is off by about 1
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)
    H1 = R.act(y @ f64(st["w1"]).T + f64(st["b1"]), "gelu")
    DZ = (f64(st["do"]) @ f64(st["w2"])) * H1[1]
    DY = DZ @ f64(st["w1"])
    DX, DG = R.rmsnorm_bwd(DY, xhat, rstd, f64(st["g"]), f64(st["do"]))
    assert rel(f64(st["dx"]), DX) < 0.35 and rel(f64(st["dw1"]), DZ.T @ y) < 0.45
    assert rel(f64(st["dg"]), DG) < 0.45 and rel(f64(st["db1"]), DZ.sum(0)) < 0.45


def test_block_on_other_streams_and_captured(gpu_lib):
    """The block on a stream of its own, two blocks on two streams at once with
    workspaces of their own, and a captured block replayed on new inputs."""
    F = gpu_lib
    want, other = _block_state(F), _block_state(F, seed=90)
    _block(F, want)
    _block(F, other)
    torch.cuda.synchronize()
    a, b = _block_state(F), _block_state(F, seed=90)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for s, st in ((s1, a), (s2, b)):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                _block(F, st)
    torch.cuda.synchronize()
    for k in OUTPUTS:
        assert torch.equal(a[k], want[k]) and torch.equal(b[k], other[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _block(F, a)
    for k in ("x", "r", "g", "w1", "b1", "w2", "b2", "do"):
        a[k].copy_(other[k])
    for k in OUTPUTS:
        a[k].zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in OUTPUTS:
        assert torch.equal(a[k], other[k]), k


def test_refuses_other_devices_streams_and_aliases(gpu_lib):
    F = gpu_lib
    x, y = rand(4, 64, seed=1), torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    for o in (dict(weight=torch.ones(64)), dict(y=y.cpu()), dict(q8=F.Ckpt8.empty(4, 64, "cpu")),
              dict(rstd=torch.zeros(4))):
        with pytest.raises(ValueError):
            F.fqt_rmsnorm_fwd(**{**dict(x=x, weight=w, y=y), **o})
    with pytest.raises(F.Fp4Error):                    # rows on top of one another
        F.fqt_rmsnorm_fwd(x, w, y[:1].expand(4, 64))
    with pytest.raises(F.Fp4Error):                    # too small a workspace
        F.fqt_act_bwd(x, x, y, dbias=torch.zeros(64, device="cuda"), ws=F.Workspace())


@pytest.mark.parametrize("chained", [False, True])
def test_swiglu_stack_with_checkpoints(gpu_lib, chained):
    """The MLP stack of the bench with its glue by the activation calls, gate
    and up kept in 8 bits: every linear within its operands' noise, as without;
    dgu off by what E4M3 loses of gate and up.  Rounding to four significant
    bits is off by a relative root mean square of 2^-4 / sqrt(3) at most (3.6 %,
    uniform in half a step of 2^-4 of the value); du carries f(g)'s and dg the
    root sum of squares of u's and f'(g)'s, of which each is at most about
    g's: below 2 * 3.6 %."""
    import bench
    from test_gpu_swiglu import _check
    res = bench.run_swiglu(torch.device("cuda", 0), layers=3, hidden=256, ffn=512, tokens=1024, chained=chained,
                           ckpt8=True)
    _check(res)
    c = res["ckpt8"]
    assert c["bytes_kept"] * 64 == c["bytes_bf16"] * 33
    assert all(0 < e < 0.072 for e in c["dgu_rel_err"])
