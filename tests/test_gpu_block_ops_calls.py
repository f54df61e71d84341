"""Calls around the FP4 linear that their documentation allows and that
tests/test_gpu_block_ops.py does not make."""
import numpy as np
import pytest
import torch

import block_ref as R
from block_ref import EPS16, EPS32, f64
from test_gpu_block_ops import BF16, F32, STEP, TINY, TYPES, _act_of, _norm_inputs, _operands, padded, rand

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# A workspace that the call makes itself, on a stream that is not the current one
# --------------------------------------------------------------------------
def _behind_work(stream, call):
    """Runs call(stream) behind a few milliseconds of that stream's work; until
    they are over, the current stream allocates and writes as much as the
    allocator has free."""
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for _ in range(16):
            big.add_(1.0)
    call(stream)
    kept = []
    for n in (256, 1 << 14, 1 << 18, 1 << 20, 1 << 22):
        kept += [torch.full((n,), 3.0e9, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all((t == 3.0e9).all() for t in kept)         # nor did the call write there


@pytest.mark.parametrize("call", ["norm", "act", "gated"])
def test_row_sums_on_another_stream_without_workspace(gpu_lib, call):
    F = gpu_lib
    rows, cols = 2049, 2048
    dy, x, w = rand(rows, cols, seed=1), rand(rows, 2 * cols, seed=2), torch.ones(cols, device="cuda")
    dx, rstd = torch.zeros(rows, 2 * cols, dtype=BF16, device="cuda"), torch.ones(rows, device="cuda")
    sums, want = (torch.zeros(2 * cols if call == "gated" else cols, device="cuda") for _ in range(2))

    def run(out, **k):
        if call == "norm":
            F.fqt_rmsnorm_bwd(dy, w, rstd, dx[:, :cols], s=x[:, :cols], dweight=out, **k)
        else:
            zc = 2 * cols if call == "gated" else cols
            F.fqt_act_bwd(dy, x[:, :zc], dx[:, :zc], act=F.ACT_SILU, gated=call == "gated", dbias=out, **k)

    run(want, ws=F.Workspace.colsum(rows, 2 * cols))
    s = torch.cuda.Stream()
    for _ in range(3):
        sums.zero_()
        _behind_work(s, lambda stream: run(sums, stream=stream))
        assert torch.equal(sums, want)


def test_gemm_epi_on_another_stream_without_workspace(gpu_lib):
    """A block with Inf is recorded in the call's own workspace, not in memory
    that the allocator gave away since."""
    F = gpu_lib
    qa, qb = _operands(F, 128, 256, 128, 0)
    bias = torch.full((256,), float("inf"), device="cuda")
    z8, c = F.Ckpt8.empty(128, 256), torch.zeros(128, 256, dtype=BF16, device="cuda")
    s = torch.cuda.Stream()
    for _ in range(3):
        c.zero_()
        _behind_work(s, lambda stream: F.fp4_gemm_epi(qa, qb, c, bias=bias, z8=z8, stream=stream))
        assert torch.isinf(c).all() and (z8.scales == 255).all()


# --------------------------------------------------------------------------
# Checkpoints whose tensors are not those they were made with
# --------------------------------------------------------------------------
def test_checkpoint_brought_back(gpu_lib):
    """Codes and scales moved off the device and back, into an object of their
    own or the old one, decode to what they held."""
    F = gpu_lib
    z = rand(33, 256, seed=1)
    q, y, want = F.Ckpt8.empty(33, 256), torch.zeros_like(z), torch.zeros_like(z)
    F.fqt_act_fwd(z, act=F.ACT_NONE, z8=q)
    F.fqt_act_fwd(q, want, act=F.ACT_NONE)
    codes, scales = q.codes.cpu(), q.scales.cpu()
    again = F.Ckpt8(33, 256, codes.cuda(), scales.cuda())
    F.fqt_act_fwd(again, y, act=F.ACT_NONE)
    assert torch.equal(y, want)
    q.codes.zero_()
    q.codes, q.scales = codes.cuda(), scales.cuda()
    y.zero_()
    F.fqt_act_fwd(q, y, act=F.ACT_NONE)
    assert torch.equal(y, want)
    # written through the constructor's object: both tensors, by each call that writes one
    for made in (lambda c: F.fqt_act_fwd(z, y, z8=c, act=F.ACT_NONE),
                 lambda c: F.fqt_rmsnorm_fwd(z, torch.ones(256, device="cuda"), y, q8=c)):
        old = F.Ckpt8.empty(33, 256)
        made(old)
        new = F.Ckpt8(33, 256, torch.zeros_like(old.codes), torch.zeros_like(old.scales))
        made(new)
        assert torch.equal(new.codes, old.codes) and torch.equal(new.scales, old.scales)


def test_checkpoint_on_the_host_is_refused(gpu_lib):
    F = gpu_lib
    z = rand(33, 256, seed=1)
    for part in ("codes", "scales"):
        q = F.Ckpt8.empty(33, 256)
        setattr(q, part, getattr(q, part).cpu())
        with pytest.raises(ValueError):
            F.fqt_act_fwd(z, act=F.ACT_NONE, z8=q)


# --------------------------------------------------------------------------
# The GEMM's amax of values that are not finite
# --------------------------------------------------------------------------
@pytest.mark.parametrize("m,n", [(128, 256), (1280, 2176)])       # narrow tiles, wide ones
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu"])
def test_gemm_epi_amax_of_nonfinite_values(gpu_lib, m, n, out, kind):
    """A NaN or Inf of the bias or the residual is in C and in c_amax, without a
    checkpoint too; a NaN outweighs Inf."""
    F = gpu_lib
    qa, qb = _operands(F, m, n, 128, 0)
    c, amax = torch.zeros(m, n, dtype=TYPES[out], device="cuda"), torch.zeros(1, device="cuda")
    act = _act_of(F, kind)
    bias, res = torch.zeros(n, device="cuda"), torch.zeros(m, n, dtype=BF16, device="cuda")
    F.fp4_gemm_epi(qa, qb, c, bias=bias, act=act, residual=res, c_amax=amax)
    finite = float(amax)
    assert finite == float(c.abs().max()) or out == "bf16"        # the FP32 values' maximum
    for value in (float("nan"), float("inf")):
        for col in (0, n - 1, 70):
            bias.zero_()
            bias[col] = value
            F.fp4_gemm_epi(qa, qb, c, bias=bias, act=act, c_amax=amax)
            bad = torch.isnan(c) if value != value else torch.isinf(c)
            assert bad[:, col].all() and int(bad.sum()) == m
            assert np.isnan(float(amax)) if value != value else float(amax) == value
    for row, col in ((0, 0), (m - 1, n - 1), (77, 33)):
        res.zero_()
        res[row, col] = float("nan")
        F.fp4_gemm_epi(qa, qb, c, act=act, residual=res, c_amax=amax)
        assert int(torch.isnan(c).sum()) == 1 and torch.isnan(c[row, col]) and np.isnan(float(amax))
        res[row, col] = -float("inf")
        F.fp4_gemm_epi(qa, qb, c, act=act, residual=res, c_amax=amax)
        assert float(amax) == float("inf")
    bias.fill_(float("inf"))
    res[5, 5] = float("nan")
    F.fp4_gemm_epi(qa, qb, c, bias=bias, act=act, residual=res, c_amax=amax)
    assert np.isnan(float(amax))
    F.fp4_gemm_epi(qa, qb, c, act=act, c_amax=amax)                # and the next call's is its own
    assert float(amax) == finite


# --------------------------------------------------------------------------
# Launches that start early, and another stream
# --------------------------------------------------------------------------
def test_early_launches_leave_room_for_another_stream(gpu_lib):
    """A product of 32 narrow tiles with another one queued behind it leaves 116
    SMs to a second stream: 110 tiles there run at once, as they do alone.  If
    the queued product already held 32 SMs while it waits, they would take two
    turns, twice the time."""
    F = gpu_lib
    k = 32768

    def product(f, m, n):
        qa, qb = _operands(F, m, n, k, 0)
        c, ws = torch.zeros(m, n, device="cuda"), F.Workspace()
        return lambda: f(qa, qb, c, ws=ws)

    chain, other = product(F.fp4_gemm_epi, 128, 4096), product(F.fp4_gemm, 1280, 2816)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def time_other(beside):
        times = []
        for _ in range(5):
            e0, e1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            torch.cuda.synchronize()
            with torch.cuda.stream(a):
                for _ in range(24 if beside else 0):
                    chain()
            with torch.cuda.stream(b):
                other()                                   # the first, while the chain begins
                e0.record()
                for _ in range(8):
                    other()
                e1.record()
            torch.cuda.synchronize()
            times.append(e0.elapsed_time(e1))
        return sorted(times)[2]

    time_other(True)
    alone, beside = time_other(False), time_other(True)
    assert beside < 1.4 * alone, (beside, alone)


# --------------------------------------------------------------------------
# RMS norm: every pair of stored and gradient type, without the residual's
# gradient; rings that go round
# --------------------------------------------------------------------------
def _within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[0].tolist(), float(off[bad].max()))


def _bwd_case(F, rows, cols, saved, grad, dres, seed):
    """One backward against the formulas in 64 bits; the bounds are those of
    test_gpu_block_ops.test_rmsnorm_bwd."""
    s = rand(rows, cols, seed=seed, dtype=TYPES["f32" if saved == "f32" else "bf16"])
    s[:, : max(1, cols // 50)] *= 20
    rstd = torch.rsqrt(s.float().square().mean(1) + 1e-5)
    w = rand(cols, seed=seed + 1, std=0.2, mean=1.0, dtype=F32)
    dy = rand(rows, cols, seed=seed + 2, std=0.1)
    dr = rand(rows, cols, seed=seed + 3, std=0.1, dtype=TYPES[grad]) if dres else None
    if saved == "ckpt":
        q8 = F.Ckpt8.empty(rows, cols)
        F.fqt_act_fwd((s.float() * rstd[:, None]).to(BF16), act=F.ACT_NONE, z8=q8)
        e = torch.ldexp(torch.ones_like(q8.scales, dtype=torch.float64), q8.scales.int() - 127)
        kw, xhat = {"xhat8": q8}, q8.codes.view(torch.float8_e4m3fn).double() * e.repeat_interleave(32, 1)
    else:
        kw, xhat = {"s": s}, s.double() * rstd.double()[:, None]
    dx, dw = torch.full((rows, cols), 7.0, dtype=TYPES[grad], device="cuda"), torch.full((cols,), 5.0, device="cuda")
    F.fqt_rmsnorm_bwd(dy, w, rstd, dx, dres=dr, dweight=dw, **kw)
    r, d = rstd.double()[:, None], dy.double()
    t, g = d * xhat, d * w.double()
    gx = g * xhat
    m, ma = gx.mean(1, keepdim=True), gx.abs().mean(1, keepdim=True)
    want = r * (g - xhat * m) + (dr.double() if dres else 0)
    bound = EPS32 * (8 * r * (g.abs() + xhat.abs() * m.abs()) + 72 * r * xhat.abs() * ma +
                     (2 * dr.double().abs() if dres else 0)) + STEP[TYPES[grad]] * want.abs() * 1.01 + TINY
    _within(dx, want, bound, "dx")
    chain = rows / 148 + 2 + 32 + 14 + 32
    _within(dw, t.sum(0), EPS32 * chain * t.abs().sum(0) + TINY, "dweight")
    alone = torch.zeros_like(dx)
    F.fqt_rmsnorm_bwd(dy, w, rstd, alone, dres=dr, **kw)              # without dweight
    assert torch.equal(alone, dx)


NORM_SHAPES = [(1, 8), (3, 64), (5, 72), (33, 256), (9, 264), (17, 1000), (9, 1024), (300, 1056), (401, 4096),
               (2, 4104), (500, 8200), (350, 16384), (1201, 96), (5000, 2056), (9000, 64)]


@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
@pytest.mark.parametrize("saved", ["bf16", "f32"])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("dres", [False, True])
def test_rmsnorm_bwd_from_the_stored_sum(gpu_lib, rows, cols, saved, grad, dres):
    _bwd_case(gpu_lib, rows, cols, saved, grad, dres, seed=60)


def _rows_round(cols, bytes_per_value):
    """Rows of more than twice all the shared memory of 148 SMs, so that every
    group of threads goes round its ring more than twice; rings of short rows
    have at most 8 stages of 32 rows in each of 444 CTAs."""
    return min(int(2.2 * 148 * 228 * 1024 / (cols * bytes_per_value)), int(2.2 * 444 * 8 * 32)) + 13


# one width for each of the layouts: 8 and 16 threads to a row with one to four
# chunks, 32, and more, some a multiple of the threads' columns and some not
RING_COLS = [64, 128, 192, 256, 352, 512, 544, 768, 1024, 1440, 2080, 2336, 2784, 4096, 4128, 5344, 6880, 8192,
             8224, 9696, 12288, 14496, 16384]


@pytest.mark.parametrize("cols", RING_COLS)
@pytest.mark.parametrize("saved,grad,dres,value_bytes", [
    ("bf16", "bf16", False, 4), ("bf16", "bf16", True, 6), ("f32", "bf16", True, 8), ("f32", "f32", True, 10),
    ("ckpt", "bf16", False, 3), ("ckpt", "bf16", True, 5), ("ckpt", "f32", True, 7)])
def test_rmsnorm_bwd_rings_go_round(gpu_lib, cols, saved, grad, dres, value_bytes):
    _bwd_case(gpu_lib, _rows_round(cols, value_bytes), cols, saved, grad, dres, seed=70)


@pytest.mark.parametrize("cols", RING_COLS)
@pytest.mark.parametrize("residual,q8,value_bytes", [(None, False, 2), (None, True, 2), ("bf16", False, 4),
                                                     ("bf16", True, 4), ("f32", True, 6)])
def test_rmsnorm_fwd_rings_go_round(gpu_lib, cols, residual, q8, value_bytes):
    """The bounds are those of test_gpu_block_ops.test_rmsnorm_fwd."""
    F, rows = gpu_lib, _rows_round(cols, value_bytes)
    x, r, w = _norm_inputs(rows, cols, residual, "f32", seed=80)
    y, rstd = torch.zeros_like(x), torch.zeros(rows, device="cuda")
    res = torch.zeros_like(r) if residual else None
    q = F.Ckpt8.empty(rows, cols) if q8 else None
    F.fqt_rmsnorm_fwd(x, w, y, residual=r, res_out=res, q8=q, q8_of=F.RMS_XHAT, rstd=rstd, eps=1e-5)
    s = x.double() + r.double() if residual else x.double()
    rs = (s.square().mean(1) + 1e-5).rsqrt()
    _within(rstd, rs, 48 * EPS32 * rs, "rstd")
    if residual:
        assert torch.equal(res, (x.float() + r.float()).to(r.dtype))
    xhat = s * rs[:, None]
    want = xhat * w.double()
    _within(y, want, want.abs() * (EPS16 + 56 * EPS32) + TINY, "y")
    if q8:
        e = torch.ldexp(torch.ones_like(q.scales, dtype=torch.float64), q.scales.int() - 127).repeat_interleave(32, 1)
        top = xhat.abs().view(rows, -1, 32).amax(2)
        assert bool((top * (1 - 56 * EPS32) <= 448 * e[:, ::32]).all())
        assert bool((top * (1 + 56 * EPS32) > 224 * e[:, ::32]).all())       # the least such power
        values = q.codes.view(torch.float8_e4m3fn).double() * e
        _within(values, xhat, torch.maximum(xhat.abs() * 2.0 ** -4, e * 2.0 ** -10) * (1 + 2.0 ** -10) +
                xhat.abs() * 56 * EPS32, "checkpoint")


# --------------------------------------------------------------------------
# GELU's left tail, where the value is small against z
# --------------------------------------------------------------------------
def _all_bf16(lo, hi):
    """Every BF16 value in [lo, hi], a row of them."""
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF16).float()
    v = v[(v >= lo) & (v <= hi)]
    return v[: v.numel() // 32 * 32].to(BF16).cuda().view(1, -1)


def _upper_tail(a):
    """1 - Phi(a); torch's ndtr is a sum with 1, which leaves 2^-53 of error."""
    return torch.special.erfc(a * 0.5 ** 0.5) / 2


def test_gelu_tail(gpu_lib):
    """Relative to the value itself, for z < 0.  The tail function Q is within
    2^-10 (a fit within 0.85 * 2^-10, act_device.cuh; the exponent, up to 141,
    has three roundings of 2^-24, 1.7e-5, and the rest is below that), the
    result is rounded once; where exp(-z^2 / 2) is below FP32's normal range it
    may be flushed to zero: |z| 2^-126.  The derivative is Q - |z| phi, phi
    within 2^-15 by the same exponent."""
    F = gpu_lib
    z = _all_bf16(-40.0, -2.0 ** -20)
    y, dz, one = torch.zeros_like(z), torch.zeros_like(z), torch.ones_like(z)
    F.fqt_act_fwd(z, y, act=F.ACT_GELU)
    F.fqt_act_bwd(one, z, dz, act=F.ACT_GELU)
    a = -z.double()
    q, pdf = _upper_tail(a), torch.exp(-a * a / 2) / (2 * np.pi) ** 0.5
    flush = (1 + a) * 2.0 ** -126
    _within(y, -a * q, a * q * (EPS16 + 2.0 ** -10) + flush, "gelu")
    _within(dz, q - a * pdf, (q - a * pdf).abs() * EPS16 + q * 2.0 ** -10 + a * pdf * 2.0 ** -15 + flush, "derivative")


def test_gemm_epi_gelu_tail(gpu_lib):
    """The same of an FP32 output: z is what the product and bias give exactly."""
    F = gpu_lib
    qa, qb = _operands(F, 128, 256, 64, 0)
    zero = torch.zeros(128, 256, device="cuda")
    bias = -torch.linspace(0.01, 12.5, 256, device="cuda")
    F.fp4_gemm_epi(qa, qb, zero, alpha=0.0, bias=bias, act=F.ACT_GELU)
    a = -bias.double()
    q = _upper_tail(a)
    _within(zero, (-a * q).expand(128, 256), (a * q * 2.0 ** -10).expand(128, 256), "gelu")


# --------------------------------------------------------------------------
# The gradient of a bias that no activation follows
# --------------------------------------------------------------------------
@pytest.mark.parametrize("rows,cols", [(1, 8), (33, 72), (260, 4096), (4099, 264)])
def test_bias_gradient_without_activation(gpu_lib, rows, cols):
    """ACT_NONE with dy as z and dz: the sums of dy over the rows, dy as it was,
    the padding of its rows too."""
    F = gpu_lib
    dy = rand(rows, cols, seed=1, std=0.1)
    buf, a = padded(dy, 24)
    db = torch.full((cols,), 5.0, device="cuda")
    F.fqt_act_bwd(a, a, a, act=F.ACT_NONE, dbias=db, ws=F.Workspace.colsum(rows, cols))
    assert torch.equal(a, dy) and (buf[:, cols:] == 7.0).all()
    d = dy.double()
    # chains: rows of a thread, 32 rows of the CTA, 14 and 32 slices
    _within(db, d.sum(0), EPS32 * (rows / 4 + 32 + 14 + 32) * d.abs().sum(0) + TINY, "dbias")
