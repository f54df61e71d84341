"""What the binding of the calls around the FP4 linear passes to the library, without a
GPU: the library's entry points are stood in for by recorders, so nothing is
launched."""
import contextlib
import ctypes as C

import pytest
import torch

import fp4_fully_quantized_b200 as F

BF16, F32 = torch.bfloat16, torch.float32


class _Recorder:
    """The library with its compute calls replaced: each records its arguments
    and returns FP4_OK."""
    CALLS = ("fqt_rmsnorm_fwd", "fqt_rmsnorm_bwd", "fqt_act_fwd", "fqt_act_bwd", "fp4_gemm_epi", "fp4_gemm",
             "fp4_gemm_quant", "fp4_gemm_quant_ex")

    def __init__(self, lib):
        self._lib, self.calls = lib, []

    def __getattr__(self, name):
        if name in _Recorder.CALLS:
            return lambda *a: self.calls.append((name, a)) or 0
        return getattr(self._lib, name)


class _FakeStream:
    cuda_stream, device = 1234, torch.device("cpu")


@pytest.fixture
def recorder(monkeypatch):
    from fp4_fully_quantized_b200 import build
    build.build()
    r = _Recorder(F.load())
    monkeypatch.setattr(F, "_lib", r)
    monkeypatch.setattr(F, "_on_device", lambda where, dev, stream: 1234)
    monkeypatch.setattr(F, "_stream", lambda stream=None: C.c_void_p(1234))
    return r


class _Cuda:
    """A tensor that says it is on a CUDA device."""
    is_cuda = True

    def __init__(self, t):
        self._t = t

    def __getattr__(self, name):
        return getattr(self._t, name)


def _without_workspace(name, stream):
    """The call `name` on `stream`, with all its arguments but a workspace."""
    m = lambda r, c, t=BF16: torch.zeros(r, c, dtype=t)
    v = lambda n: torch.zeros(n)
    f = getattr(F, name)
    if name == "fqt_rmsnorm_bwd":
        a, k = (m(4, 64), v(64), v(4), m(4, 64)), dict(s=m(4, 64), dweight=v(64))
    elif name == "fqt_act_bwd":
        a, k = (m(4, 64), m(4, 64), m(4, 64)), dict(dbias=v(64))
    else:
        q = lambda rows, cols: F.QTensor.empty(rows, cols, device="cpu")
        out = {"fp4_gemm_epi": lambda: (m(128, 256),), "fp4_gemm": lambda: (_Cuda(m(128, 256)),)}
        a, k = (q(128, 64), q(256, 64), *out.get(name, lambda: (q(128, 256), v(1)))()), {}
    return lambda: f(*a, **k, stream=stream)


@pytest.mark.parametrize("name", ["fqt_rmsnorm_bwd", "fqt_act_bwd", "fp4_gemm_epi", "fp4_gemm", "fp4_gemm_quant",
                                  "fp4_gemm_quant_ex"])
def test_own_workspace_belongs_to_the_stream(recorder, monkeypatch, name):
    """A workspace that a call makes itself is allocated and zeroed on the stream
    that its kernels run on: on another one the allocator would hand the memory
    out again while they still use it, and the zeroing would be unordered."""
    current, made = [None], []
    stream = _FakeStream()
    call = _without_workspace(name, stream)

    @contextlib.contextmanager
    def on(s):
        before, current[0] = current[0], s
        try:
            yield
        finally:
            current[0] = before

    def noted(make):
        return lambda *a, **k: made.append(current[0]) or make(*a, **k)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "zeros", noted(torch.zeros))
    monkeypatch.setattr(torch, "empty", noted(torch.empty))
    call()
    assert [c[0] for c in recorder.calls] == [name]
    assert made and all(s is stream for s in made)
