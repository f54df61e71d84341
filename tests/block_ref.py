"""64-bit references of the calls between two FP4 linears (numpy, float64),
written from the formulas in include/fp4.h; no code of the library."""
from __future__ import annotations

import numpy as np
import torch
from scipy import special

EPS32 = 2.0 ** -24            # half a step, relative: FP32, BF16, E4M3
EPS16 = 2.0 ** -8
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().to("cpu").double().numpy()


def block_scale_bytes(v: np.ndarray) -> np.ndarray:
    """E8M0 byte of each 32-block of the rows of v: the least 2^e >= max / 448."""
    top = np.abs(v).reshape(v.shape[0], -1, 32).max(-1)
    frac, e = np.frexp(np.where(np.isfinite(top), top, 1.0) / 448.0)
    e = np.where(frac == 0.5, e - 1, e)
    e = np.where(top == 0, -127, np.maximum(e, -127))
    return np.where(np.isfinite(top), e + 127, 255).astype(np.int64)


def e4m3_round(q: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value, ties to even, for |q| <= 448."""
    k = np.maximum(np.frexp(q)[1] - 1, -6)
    unit = np.ldexp(1.0, k - 3)
    return np.round(q / unit) * unit


def encode(v: np.ndarray):
    """(E4M3 values, scale bytes) of finite v."""
    b = block_scale_bytes(v)
    e = np.repeat(b - 127, 32, axis=1)
    return e4m3_round(np.ldexp(v, -e)), b


def code_values(codes: torch.Tensor) -> np.ndarray:
    return codes.cpu().view(torch.float8_e4m3fn).double().numpy()


def decode(codes: torch.Tensor, scales: torch.Tensor) -> np.ndarray:
    b = scales.cpu().numpy().astype(np.int64)
    e = np.where(b == 255, np.nan, np.ldexp(1.0, np.minimum(b, 254) - 127))
    return code_values(codes) * np.repeat(e, 32, axis=1)


def act(z: np.ndarray, kind: str):
    """The activation, its derivative and the size of the terms that the
    derivative is a sum of (what an FP32 evaluation's error is relative to)."""
    if kind == "none":
        return z, np.ones_like(z), np.ones_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(z.dtype), (z > 0).astype(z.dtype)
    if kind == "silu":
        p = special.expit(z)
        return z * p, p + z * p * special.expit(-z), p + np.abs(z * p)
    if kind == "gelu":
        cdf, pdf = special.ndtr(z), np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
        # an FP32 CDF (1 + erf) / 2 is good to its last places near 1, not near 0
        return z * cdf, cdf + z * pdf, 1 + np.abs(z) * pdf
    c = 2 * np.sqrt(2 / np.pi)
    z2 = np.minimum(z * z, 1e6)            # p is 0 or 1 there
    p, m = special.expit(c * z * (1 + 0.044715 * z2)), special.expit(-c * z * (1 + 0.044715 * z2))
    t = z * p * m * c * (1 + 0.134145 * z2)
    return z * p, p + t, p + np.abs(t)


def act_value_error(z: np.ndarray, kind: str) -> np.ndarray:
    """Bound on the error of an FP32 evaluation of the activation.

    silu, gelu_tanh: z p with p from exp(-t): the argument t has at most eight
    roundings (relative 2^-21), so exp is off by |t| 2^-21 relative, the fast
    exponential itself by 2 + 1.173 |t| units (2^-23 each), the quotient by two:
    below (|t| + 4) 2^-20.  Where |t| > 88 the value is below 2^-126 |z| or
    equal to z.

    gelu: |z| times the CDF's error.  The tail is q(t) e, q = (a1 t + ... + a5 t^5) / 2
    (A&S 7.1.26, off by 0.75e-7).  t comes from a reciprocal (a sum rounded, the
    reciprocal within 2^-23; 6 units of 2^-24 leave room for a product of two) and
    enters with dq/dln t <= (a1 + 2 a2 + 3 a3 + 4 a4 + 5 a5)/2 = 1.73; Horner's five
    steps stay below 0.54, rounded to 2.2 units in all; e is within 4 units and the
    tail below 1/2: 0.75e-7 + (1.73 * 6 + 2.2 + 2) 2^-24
    = 9.4e-7 < 2^-20."""
    v = np.abs(act(z, kind)[0])
    if kind in ("none", "relu"):
        return np.zeros_like(v)
    if kind == "gelu":
        return np.abs(z) * 2.0 ** -20
    t = np.abs(z) if kind == "silu" else 1.6 * np.abs(z) * (1 + 0.045 * np.minimum(z * z, 1e6))
    return v * (np.minimum(t, 88) + 4) * 2.0 ** -20 + np.where(t > 80, np.abs(z) * 2.0 ** -115, 0)


def act_grad_error(z: np.ndarray, kind: str) -> np.ndarray:
    """The same for the derivative: each of its terms within (|t| + 8) 2^-19."""
    if kind in ("none", "relu"):
        return np.zeros_like(z)
    size = act(z, kind)[2]
    if kind == "gelu":
        return size * 2.0 ** -19
    t = np.abs(z) if kind == "silu" else 1.6 * np.abs(z) * (1 + 0.045 * np.minimum(z * z, 1e6))
    return size * (np.minimum(t, 88) + 8) * 2.0 ** -19 + np.where(t > 80, (1 + np.abs(z)) * 2.0 ** -115, 0)


def assert_within(got, want, bound, what=""):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    off = np.abs(got - want) - bound
    bad = ~(off <= 0)
    if bad.any():
        i = np.unravel_index(np.nanargmax(np.where(bad, np.where(np.isnan(off), np.inf, off), -np.inf)),
                             off.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {off.size} out of bounds, e.g. at {i}: got "
                             f"{got[i]!r}, want {want[i]!r} within {np.broadcast_to(bound, off.shape)[i]!r}")


def assert_checkpoint(codes, scales, want, rel=0.0):
    """The checkpoint holds `want`, known up to a relative error `rel`: every
    scale byte is the one of some block maximum within rel, every decoded value
    is within half an E4M3 step (2^-4 of the value, 2^-10 of the scale below
    E4M3's normal range) and that error."""
    b = scales.cpu().numpy().astype(np.int64)
    lo, hi = block_scale_bytes(want * (1 - rel)), block_scale_bytes(want * (1 + rel))
    assert ((b >= lo) & (b <= hi)).all(), "scale bytes"
    e = np.repeat(np.ldexp(1.0, b - 127), 32, axis=1)
    size = np.abs(want) * (1 + rel)
    assert_within(decode(codes, scales), want, np.maximum(size * 2.0 ** -4, e * 2.0 ** -10) +
                  np.abs(want) * rel, "checkpoint values")


def rmsnorm(x, residual, weight, eps):
    s = x if residual is None else x + residual
    rstd = 1 / np.sqrt((s * s).mean(1) + eps)
    xhat = s * rstd[:, None]
    return s, rstd, xhat, xhat * weight


def rmsnorm_bwd(dy, xhat, rstd, weight, dres):
    g = dy * weight
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdims=True))
    return dx if dres is None else dx + dres, (dy * xhat).sum(0)


def act_fwd(z, kind, gated):
    w = z.shape[1] // 2
    return act(z[:, :w], kind)[0] * z[:, w:] if gated else act(z, kind)[0]


def act_bwd(dy, z, kind, gated):
    if not gated:
        return dy * act(z, kind)[1]
    w = z.shape[1] // 2
    f, df, _ = act(z[:, :w], kind)
    return np.concatenate([dy * z[:, w:] * df, dy * f], 1)
