"""Measured cases of the operators around the FP4 linear layer: RMS norm with
the residual's addition and 8-bit output (forward, backward), activations with
8-bit checkpoints (forward, recomputation, backward), and the FP4 matrix
product with bias, activation, residual and checkpoint in its epilogue.

Each case has a plain form (torch, 32 bits, rounded once at the end), the
library's own call (`own` true) and a 64-bit form (`exact`).

The 8-bit format: blocks of 32 consecutive values of a row share the power of
two 2^e, e the least with block max <= 448 * 2^e (e >= -127); each value is
stored as E4M3, rounded to nearest even, of value / 2^e.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
EPS = 1e-5


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _norm_fwd(rows, cols, residual="none", weight="bf16", q8="none", amax=False, pad=0, **name):
    return dict(name, op="norm_fwd", rows=rows, cols=cols, residual=residual, weight=weight, q8=q8,
                amax=amax, pad=pad)


def _norm_bwd(rows, cols, saved, grad="bf16", dres=True, weight="bf16", **name):
    return dict(name, op="norm_bwd", rows=rows, cols=cols, saved=saved, grad=grad, dres=dres,
                weight=weight)


def _act_fwd(rows, cols, act, gated, source="bf16", z8=False, amax=False, pad=0, **name):
    return dict(name, op="act_fwd", rows=rows, cols=cols, act=act, gated=gated, source=source,
                z8=z8, amax=amax, pad=pad)


def _act_bwd(rows, cols, act, gated, source, dbias=False, amax=False, **name):
    return dict(name, op="act_bwd", rows=rows, cols=cols, act=act, gated=gated, source=source,
                dbias=dbias, amax=amax)


def _gemm(m, n, k, fmt, act, bias, residual, out="bf16", z8=False, **name):
    return dict(name, op="gemm", m=m, n=n, k=k, fmt=fmt, act=act, bias=bias, residual=residual,
                out=out, z8=z8)


def listed():
    return [
        # one new token of a 4096-wide model: latency alone
        _norm_fwd(1, 4096, "bf16", name="norm fwd 1x4096 decode"),
        # per-head norms of queries, an odd number of short rows
        _norm_fwd(40001, 128, q8="y", name="norm fwd 40001x128 heads"),
        # a training step's norm: residual stream kept in 32 bits, the
        # normalized rows checkpointed in 8 bits, amax for the next quantizer
        _norm_fwd(32768, 4096, "f32", "f32", q8="xhat", amax=True, name="norm fwd 32768x4096 ckpt"),
        # its backward from the checkpoint, and a smaller one from the stored sum
        _norm_bwd(32768, 4096, "xhat8", "f32", weight="f32", name="norm bwd 32768x4096 ckpt"),
        _norm_bwd(2049, 2048, "s_bf16", name="norm bwd 2049x2048 stored"),
        # SwiGLU of a few tokens being served
        _act_fwd(7, 11008, "silu", True, name="swiglu fwd 7x11008 serving"),
        # SwiGLU of a training step, gate and up checkpointed in 8 bits
        _act_fwd(16384, 8192, "silu", True, z8=True, amax=True, name="swiglu fwd 16384x8192 ckpt"),
        # its backward from the checkpoint
        _act_bwd(16384, 8192, "silu", True, "ckpt8", amax=True, name="swiglu bwd 16384x8192 ckpt"),
        # backward of a biased GELU layer on a ragged batch, with the bias gradient
        _act_bwd(1531, 11008, "gelu", False, "ckpt8", dbias=True, name="gelu bwd 1531x11008 dbias"),
        # a small batch through a biased GELU layer, 32-bit output
        _gemm(128, 4096, 4096, "nvfp4", "gelu_tanh", "f32", "none", "f32",
              name="gemm 128x4096x4096 gelu"),
        # the up projection of a training step with its checkpoint
        _gemm(32768, 11008, 4096, "nvfp4", "gelu", "bf16", "none", z8=True,
              name="gemm 32768x11008x4096 gelu ckpt"),
        # the down projection onto the residual stream
        _gemm(32768, 4096, 11008, "mxfp4", "none", "bf16", "bf16",
              name="gemm 32768x4096x11008 residual"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "act_fwd", "act_bwd", "gemm"])
    if op == "gemm":
        m, n, k = (128 * _spread(rng, 1, 256), 128 * _spread(rng, 1, 86), 64 * _spread(rng, 1, 172))
        m = min(m, max(128, (32768 * 11008 * 4096 // (n * k)) // 128 * 128))
        fmt = rng.choice(["nvfp4", "mxfp4"])
        return _gemm(m, n, k, fmt, rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                     rng.choice(["none", "bf16", "f32"]), rng.choice(["none", "bf16", "f32"]),
                     rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5)
    rows = _spread(rng, 1, 65536)
    step = 32 if op != "norm_fwd" or rng.random() < 0.5 else 8
    cols = step * _spread(rng, max(1, 64 // step), (16384 if "norm" in op else 11008) // step)
    pad = rng.choice([0, 0, 8, 24])
    if op == "norm_fwd":
        rows = min(rows, 32768 * 4096 // cols)
        return _norm_fwd(rows, cols, rng.choice(["none", "bf16", "f32"]), rng.choice(["bf16", "f32"]),
                         rng.choice(["none", "y", "xhat"]) if step == 32 else "none",
                         rng.random() < 0.3, pad)
    if op == "norm_bwd":
        rows = min(rows, 32768 * 4096 // cols)
        return _norm_bwd(rows, cols, rng.choice(["s_bf16", "s_f32", "xhat8"]),
                         rng.choice(["bf16", "f32"]), rng.random() < 0.7, rng.choice(["bf16", "f32"]))
    gated = rng.random() < 0.5
    rows = min(rows, 16384 * 8192 // cols)
    source = rng.choice(["bf16", "ckpt8"])
    act = rng.choice(["relu", "gelu", "gelu_tanh", "silu", "silu"])
    if op == "act_fwd":
        return _act_fwd(rows, cols, act, gated, source, source == "bf16" and rng.random() < 0.5,
                        rng.random() < 0.3, pad if source == "bf16" else 0)
    return _act_bwd(rows, cols, act, gated, source, rng.random() < 0.5, rng.random() < 0.3)


def work(c):
    size = lambda t: 4 if t == "f32" else 2 if t == "bf16" else 0
    ck = 1 + 1 / 32                                    # bytes of a checkpointed value
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        per = 0.5 + (1 / 16 if c["fmt"] == "nvfp4" else 1 / 32)
        b = (m + n) * k * per + m * n * (size(c["out"]) + size(c["residual"]) + (ck if c["z8"] else 0))
        return {"bytes": b + n * size(c["bias"]), "flops": 2 * m * n * k}
    r, w = c["rows"], c["cols"]
    if c["op"] == "norm_fwd":
        b = r * w * (2 + 2 * size(c["residual"]) + 2 + (ck if c["q8"] != "none" else 0)) + 4 * r
        return {"bytes": b + w * size(c["weight"]), "flops": 5 * r * w}
    if c["op"] == "norm_bwd":
        s = {"s_bf16": 2, "s_f32": 4, "xhat8": ck}[c["saved"]]
        b = r * w * (2 + s + size(c["grad"]) * (2 if c["dres"] else 1)) + 4 * r
        return {"bytes": b + w * (size(c["weight"]) + 4), "flops": 9 * r * w}
    zw = w * (2 if c["gated"] else 1)
    zin = r * zw * (ck if c["source"] == "ckpt8" else 2)
    if c["op"] == "act_fwd":
        return {"bytes": zin + r * w * 2 + (r * zw * ck if c["z8"] else 0), "flops": 6 * r * zw}
    return {"bytes": zin + r * w * 2 + r * zw * 2 + (4 * zw if c["dbias"] else 0),
            "flops": 10 * r * zw}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)

    def normal(self, rows, cols, std=1.0, outliers=False, pad=0, dtype=BF16):
        a = torch.randn((rows, cols + pad), generator=self.g, device="cuda")
        if outliers:                                   # a few channels carry most of the size
            hot = torch.randint(0, cols, (max(1, cols // 100),), generator=self.g, device="cuda")
            a[:, hot] *= 8.0
        return a.mul_(std).to(dtype)[:, :cols]

    def vector(self, n, mean, std, dtype):
        return (torch.randn(n, generator=self.g, device="cuda") * std + mean).to(dtype)


def _empty(*shape, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _fp4_operand(d, rows, k, fmt):
    """A Gaussian operand in FP4: packed codes and one scale byte per block."""
    nv = fmt == "nvfp4"
    bs = 16 if nv else 32
    x = torch.randn((rows, k), generator=d.g, device="cuda").view(rows, k // bs, bs)
    top = x.abs().amax(-1)
    if nv:
        byte = (top * (448.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
        scale = byte.float() / 448.0
        byte = byte.view(torch.uint8)
    else:
        e = torch.floor(torch.log2(top)).int() - 2
        byte = (e + 127).to(torch.uint8)
        scale = ((e + 127) << 23).view(F32)
    mag = (x / scale.unsqueeze(-1)).abs().clamp(max=6.0)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    code = torch.bucketize(mag, edges, out_int32=True).to(torch.uint8) + (x < 0).to(torch.uint8) * 8
    code = code.view(rows, k // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), byte.contiguous()


def _mma_layout(byte):
    """Scale bytes [rows, blocks] in the tensor-core layout of the library."""
    rows, s = byte.shape
    s4 = -(-s // 4) * 4
    full = torch.zeros((rows, s4), dtype=torch.uint8, device="cuda")
    full[:, :s] = byte
    return full.view(rows // 128, 4, 32, s4 // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def prepare(c, seed):
    d, st = _Draws(seed), {"case": c}
    if c["op"] == "gemm":
        m, n, k = c["m"], c["n"], c["k"]
        for side, rows in (("a", m), ("b", n)):
            codes, byte = _fp4_operand(d, rows, k, c["fmt"])
            st[side] = {"codes": codes, "scales": byte, "scales_mma": _mma_layout(byte),
                        "s_dec": torch.full((1,), 0.04 if side == "a" else 0.05, device="cuda")}
        if c["bias"] != "none":
            st["bias"] = d.vector(n, 0.0, 0.3, TYPES[c["bias"]])
        if c["residual"] != "none":
            st["residual"] = d.normal(m, n, dtype=TYPES[c["residual"]])
        # brings the product to unit size: the NVFP4 operands hold 448 times the Gaussian values
        st["alpha"] = (448.0 ** -2 if c["fmt"] == "nvfp4" else 1.0) / (0.04 * 0.05 * math.sqrt(k))
        st["out"] = _empty(m, n, dtype=TYPES[c["out"]])
        if own:
            import fp4_fully_quantized_b200 as F
            fmt = F.NVFP4 if c["fmt"] == "nvfp4" else F.MXFP4
            for side, rows in (("a", m), ("b", n)):
                q, src = F.QTensor.empty(rows, k, fmt, logical_scales=False), st[side]
                q.codes.copy_(src["codes"].view(-1))
                q.scales_mma.copy_(src["scales_mma"])
                q.s_dec.copy_(src["s_dec"])
                st["q" + side] = q
            st["z8"] = F.Ckpt8.empty(m, n) if c["z8"] else None
            st["ws"] = F.Workspace(m, n, k)
        return st
    r, w, pad = c["rows"], c["cols"], c.get("pad", 0)
    if c["op"] == "norm_fwd":
        st["x"] = d.normal(r, w, outliers=True, pad=pad)
        st["weight"] = d.vector(w, 1.0, 0.1, TYPES[c["weight"]])
        st["y"], st["rstd"] = _empty(r, w), _empty(r, dtype=F32)
        if c["residual"] != "none":
            st["residual"] = d.normal(r, w, 3.0, outliers=True, dtype=TYPES[c["residual"]])
            st["res"] = _empty(r, w, dtype=TYPES[c["residual"]])
        st["amax"] = _empty(1, dtype=F32)
        if own:
            import fp4_fully_quantized_b200 as F
            st["q8"] = F.Ckpt8.empty(r, w) if c["q8"] != "none" else None
            st["ws"] = F.Workspace()
        return st
    if c["op"] == "norm_bwd":
        s = d.normal(r, w, 3.0, outliers=True, dtype=F32 if c["saved"] == "s_f32" else BF16)
        st["rstd"] = torch.rsqrt(s.float().square().mean(-1) + EPS)
        if c["saved"] == "xhat8":
            st["codes"], st["scales"] = _encode(s.float() * st["rstd"].unsqueeze(-1))
        else:
            st["s"] = s
        st["weight"] = d.vector(w, 1.0, 0.1, TYPES[c["weight"]])
        st["dy"] = d.normal(r, w, 1e-3)
        if c["dres"]:
            st["dres"] = d.normal(r, w, 1e-3, dtype=TYPES[c["grad"]])
        st["dx"], st["dweight"] = _empty(r, w, dtype=TYPES[c["grad"]]), _empty(w, dtype=F32)
        if own:
            import fp4_fully_quantized_b200 as F
            st["q8"] = _own_ckpt(F, st, r, w) if "codes" in st else None
            st["ws"] = F.Workspace.colsum(r, w)
        return st
    zw = w * (2 if c["gated"] else 1)
    z = d.normal(r, zw, 1.5, outliers=True, pad=pad)
    if c["source"] == "ckpt8":
        st["codes"], st["scales"] = _encode(z.float())
    else:
        st["z"] = z
    st["amax"] = _empty(1, dtype=F32)
    if c["op"] == "act_fwd":
        st["y"] = _empty(r, w)
    else:
        st["dy"] = d.normal(r, w, 1e-3)
        st["dz"], st["dbias"] = _empty(r, zw), _empty(zw, dtype=F32)
    if own:
        import fp4_fully_quantized_b200 as F
        st["q8"] = _own_ckpt(F, st, r, zw) if "codes" in st else \
            F.Ckpt8.empty(r, zw) if c.get("z8") else None
        st["ws"] = F.Workspace.colsum(r, zw)
    return st


def _own_ckpt(F, st, rows, cols):
    q = F.Ckpt8.empty(rows, cols)
    q.codes.copy_(st["codes"].view(torch.uint8))
    q.scales.copy_(st["scales"].view(torch.uint8))
    return q


# --------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------
def _encode(v):
    """32-bit values [rows, cols] -> E4M3 codes and E8M0 block scales."""
    rows, cols = v.shape
    top = v.view(rows, cols // 32, 32).abs().amax(-1)
    bits = top.view(torch.int32)
    e = (bits >> 23) - 135 + ((bits & 0x7FFFFF) > 0x600000).int()
    e = torch.where(top == 0, torch.full_like(e, -127), e.clamp(min=-127))
    inv = ((127 - e).clamp(max=254) << 23).view(F32)
    codes = (v.view(rows, cols // 32, 32) * inv.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.view(rows, cols), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _decode(codes, scales):
    rows, cols = codes.shape
    two_e = (scales.view(torch.uint8).int() << 23).view(F32)
    return (codes.float().view(rows, cols // 32, 32) * two_e.unsqueeze(-1)).view(rows, cols)


def _act(z, kind):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_grad(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def _dequantize(q, k, fmt):
    rows, bs = q["codes"].shape[0], 16 if fmt == "nvfp4" else 32
    lut = torch.tensor(LEVELS + tuple(-v for v in LEVELS), device="cuda")
    code = torch.stack((q["codes"] & 15, q["codes"] >> 4), -1).view(rows, k // bs, bs).int()
    scale = q["scales"].view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else \
        (q["scales"].int() << 23).view(F32)
    return (lut[code] * scale.unsqueeze(-1)).view(rows, k)


def run(st):
    c = st["case"]
    if own:
        return _own_run(c, st)
    if c["op"] == "gemm":
        z = _dequantize(st["a"], c["k"], c["fmt"]) @ _dequantize(st["b"], c["k"], c["fmt"]).t()
        z = z * (st["alpha"] * st["a"]["s_dec"] * st["b"]["s_dec"])
        if c["bias"] != "none":
            z = z + st["bias"].float()
        y = _act(z, c["act"])
        if c["residual"] != "none":
            y = y + st["residual"].float()
        out = {"out": y.to(TYPES[c["out"]])}
        if c["z8"]:
            out["codes"], out["scales"] = _encode(z)
        return out
    if c["op"] == "norm_fwd":
        s, out = st["x"].float(), {}
        if c["residual"] != "none":
            s = s + st["residual"].float()
            out["res"] = s.to(TYPES[c["residual"]])
        out["rstd"] = torch.rsqrt((s * s).mean(-1) + EPS)
        xhat = s * out["rstd"].unsqueeze(-1)
        y = xhat * st["weight"].float()
        out["y"] = y.to(BF16)
        if c["q8"] != "none":
            out["codes"], out["scales"] = _encode(y if c["q8"] == "y" else xhat)
        if c["amax"]:
            out["amax"] = out["y"].abs().max().float()
        return out
    if c["op"] == "norm_bwd":
        if c["saved"] == "xhat8":
            xhat = _decode(st["codes"], st["scales"])
        else:
            xhat = st["s"].float() * st["rstd"].unsqueeze(-1)
        dy = st["dy"].float()
        g = dy * st["weight"].float()
        dx = st["rstd"].unsqueeze(-1) * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        if c["dres"]:
            dx = dx + st["dres"].float()
        return {"dx": dx.to(TYPES[c["grad"]]), "dweight": (dy * xhat).sum(0)}
    z = _decode(st["codes"], st["scales"]) if c["source"] == "ckpt8" else st["z"].float()
    w = c["cols"]
    if c["op"] == "act_fwd":
        y = _act(z[:, :w], c["act"])
        if c["gated"]:
            y = y * z[:, w:]
        out = {"y": y.to(BF16)}
        if c["z8"]:
            out["codes"], out["scales"] = _encode(z)
    else:
        dy = st["dy"].float()
        if c["gated"]:
            dz = torch.cat((dy * z[:, w:] * _act_grad(z[:, :w], c["act"]), dy * _act(z[:, :w], c["act"])), 1)
        else:
            dz = dy * _act_grad(z, c["act"])
        out = {"dz": dz.to(BF16)}
        if c["dbias"]:
            out["dbias"] = dz.sum(0)
    if c["amax"]:
        out["amax"] = out["y" if "y" in out else "dz"].abs().max().float()
    return out


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------
def _own_run(c, st):
    import fp4_fully_quantized_b200 as F
    act = {"none": F.ACT_NONE, "relu": F.ACT_RELU, "gelu": F.ACT_GELU, "gelu_tanh": F.ACT_GELU_TANH,
           "silu": F.ACT_SILU}[c.get("act", "none")]
    out, ws = {}, st["ws"]
    amax = st["amax"] if c.get("amax") else None
    if c["op"] == "gemm":
        F.fp4_gemm_epi(st["qa"], st["qb"], st["out"], alpha=st["alpha"], bias=st.get("bias"), act=act,
                       residual=st.get("residual"), z8=st["z8"], ws=ws)
        out["out"], q8 = st["out"], st["z8"]
    elif c["op"] == "norm_fwd":
        q8 = st["q8"]
        F.fqt_rmsnorm_fwd(st["x"], st["weight"], st["y"], residual=st.get("residual"),
                          res_out=st.get("res"), q8=q8, q8_of=F.RMS_XHAT if c["q8"] == "xhat" else F.RMS_Y,
                          rstd=st["rstd"], y_amax=amax, eps=EPS, ws=ws)
        out.update(y=st["y"], rstd=st["rstd"])
        if "res" in st:
            out["res"] = st["res"]
    elif c["op"] == "norm_bwd":
        q8 = None
        F.fqt_rmsnorm_bwd(st["dy"], st["weight"], st["rstd"], st["dx"], s=st.get("s"), xhat8=st["q8"],
                          dres=st.get("dres"), dweight=st["dweight"], ws=ws)
        out.update(dx=st["dx"], dweight=st["dweight"])
    elif c["op"] == "act_fwd":
        ckpt = c["source"] == "ckpt8"
        q8 = None if ckpt else st["q8"]
        F.fqt_act_fwd(st["q8"] if ckpt else st["z"], st["y"], act=act, gated=c["gated"], z8=q8,
                      y_amax=amax, ws=ws)
        out["y"] = st["y"]
    else:
        q8 = None
        F.fqt_act_bwd(st["dy"], st["q8"] if c["source"] == "ckpt8" else st["z"], st["dz"], act=act,
                      gated=c["gated"], dbias=st["dbias"] if c["dbias"] else None, dz_amax=amax, ws=ws)
        out["dz"] = st["dz"]
        if c["dbias"]:
            out["dbias"] = st["dbias"]
    if q8 is not None:
        out["codes"] = q8.codes.view(torch.float8_e4m3fn)
        out["scales"] = q8.scales.view(torch.float8_e8m0fnu)
    if amax is not None:
        out["amax"] = amax[0]
    return out


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------
def _exact_encode(v):
    """The block format from its definition: the least power of two that
    brings the block under 448, then the nearest E4M3 value (spacing 2^(k-3)
    from 2^k on, 2^-9 below 2^-6), ties to the even multiple."""
    blocks = v.reshape(v.shape[0], -1, 32)
    frac, e = torch.frexp(blocks.abs().amax(-1) / 448.0)       # top/448 = frac * 2^e, 1/2 <= frac < 1
    e = torch.where(frac == 0.5, e - 1, e)
    e = torch.where(frac == 0, torch.full_like(e, -127), e).clamp(min=-127)
    q = torch.ldexp(blocks, -e.unsqueeze(-1))
    k = (torch.frexp(q)[1] - 1).clamp(min=-6)
    unit = torch.ldexp(torch.ones_like(q), k - 3)
    return (torch.round(q / unit) * unit).reshape(v.shape), torch.ldexp(torch.ones_like(frac), e)


def _exact_values(st):
    return st["codes"].double() * st["scales"].double().repeat_interleave(32, 1)


def _exact_act(z, kind):
    """The activation and its derivative."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if kind == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    if kind == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    # z * logistic(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    p = torch.special.expit(u2)
    return z * p, p + z * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z.square())


def _exact_operand(q, fmt):
    byte = q["codes"].long()
    nibble = torch.stack((byte % 16, byte // 16), -1).reshape(byte.shape[0], -1)
    m = nibble % 8
    mag = torch.where(m < 2, m / 2, torch.ldexp(1 + (m % 2).double() / 2, m // 2 - 1))
    if fmt == "nvfp4":
        s = q["scales"].view(torch.float8_e4m3fn).double()
    else:
        s = torch.ldexp(torch.ones(q["scales"].shape, dtype=torch.float64, device="cuda"),
                        q["scales"].int() - 127)
    s = s.repeat_interleave(16 if fmt == "nvfp4" else 32, 1)
    return torch.where(nibble >= 8, -mag, mag) * s


def exact(c, seed):
    st = prepare(c, seed)
    if c["op"] == "gemm":
        z = _exact_operand(st["a"], c["fmt"]) @ _exact_operand(st["b"], c["fmt"]).t()
        z *= st["alpha"] * st["a"]["s_dec"].double() * st["b"]["s_dec"].double()
        if "bias" in st:
            z += st["bias"].double()
        out = {"out": _exact_act(z, c["act"])[0]}
        if "residual" in st:
            out["out"] = out["out"] + st["residual"].double()
        if c["z8"]:
            out["codes"], out["scales"] = _exact_encode(z)
        return out
    if c["op"] == "norm_fwd":
        s = st["x"].double()
        out = {}
        if "residual" in st:
            s = out["res"] = s + st["residual"].double()
        r = (s.square().sum(1) / c["cols"] + EPS) ** -0.5
        n = r[:, None] * s
        y = n * st["weight"].double()
        out.update(rstd=r, y=y)
        if c["q8"] != "none":
            out["codes"], out["scales"] = _exact_encode(n if c["q8"] == "xhat" else y)
        if c["amax"]:
            out["amax"] = None                 # the largest value as rounded to 16 bits
        return out
    if c["op"] == "norm_bwd":
        r = st["rstd"].double()[:, None]
        n = _exact_values(st) if c["saved"] == "xhat8" else st["s"].double() * r
        dy = st["dy"].double()
        g = dy * st["weight"].double()
        dx = (g - n * (n * g).sum(1, keepdim=True) / c["cols"]) * r
        if "dres" in st:
            dx += st["dres"].double()
        return {"dx": dx, "dweight": (n * dy).sum(0)}
    z = _exact_values(st) if c["source"] == "ckpt8" else st["z"].double()
    gate, up = (z[:, :c["cols"]], z[:, c["cols"]:]) if c["gated"] else (z, None)
    f, df = _exact_act(gate, c["act"])
    if c["op"] == "act_fwd":
        out = {"y": f * up if c["gated"] else f}
        if c["z8"]:
            out["codes"], out["scales"] = _exact_encode(z)
    else:
        dy = st["dy"].double()
        dz = torch.cat((dy * up * df, dy * f), 1) if c["gated"] else dy * df
        out = {"dz": dz}
        if c["dbias"]:
            out["dbias"] = dz.sum(0)
    if c["amax"]:
        out["amax"] = None
    return out
