"""What the binding of the calls around the FP4 linear passes to the library, without a
GPU: the library's entry points are stood in for by recorders, so nothing is
launched."""
import contextlib
import copy
import ctypes as C
import dataclasses
import pickle

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


# --------------------------------------------------------------------------
# Checkpoints: the library gets the addresses of the tensors that are in the
# object at the call
# --------------------------------------------------------------------------
def _passed(recorder, name, field):
    """What the structure at address argument `field` of the last call holds."""
    layout = {"fqt_rmsnorm_fwd": F._FWD, "fqt_rmsnorm_bwd": F._BWD, "fqt_act_fwd": F._ACT_FWD,
              "fqt_act_bwd": F._ACT_BWD, "fp4_gemm_epi": F._EPI}[name].__self__
    called, args = recorder.calls[-1]
    assert called == name
    address = layout.unpack(args[3 if name == "fp4_gemm_epi" else 0])[field]
    assert address
    c = F.Ckpt8C.from_address(address)
    return c.codes, c.scales, c.rows, c.cols


def _uses(q):
    """Each call that reads or writes the checkpoint q of [128, 256], with the
    place of its address among the call's packed arguments."""
    x, v = torch.zeros(128, 256, dtype=BF16), torch.ones(256)
    a, b = F.QTensor.empty(128, 64, device="cpu"), F.QTensor.empty(256, 64, device="cpu")
    ws = F.Workspace(device="cpu")
    return [("fqt_rmsnorm_fwd", 9, lambda: F.fqt_rmsnorm_fwd(x, v, x, q8=q)),
            ("fqt_rmsnorm_bwd", 4, lambda: F.fqt_rmsnorm_bwd(x, v, torch.ones(128), x, xhat8=q)),
            ("fqt_act_fwd", 2, lambda: F.fqt_act_fwd(q, x)),
            ("fqt_act_fwd", 5, lambda: F.fqt_act_fwd(x, x, z8=q)),
            ("fqt_act_bwd", 4, lambda: F.fqt_act_bwd(x, q, x)),
            ("fp4_gemm_epi", 3, lambda: F.fp4_gemm_epi(a, b, x, z8=q, ws=ws))]


def _new(rows=128, cols=256):
    return torch.zeros(rows, cols, dtype=torch.uint8), torch.zeros(rows, cols // 32, dtype=torch.uint8)


def _check_uses(recorder, q):
    for name, field, call in _uses(q):
        call()
        assert _passed(recorder, name, field) == (q.codes.data_ptr(), q.scales.data_ptr(), 128, 256)


def test_checkpoint_made_by_its_constructor(recorder):
    codes, scales = _new()
    _check_uses(recorder, F.Ckpt8(128, 256, codes, scales))
    _check_uses(recorder, F.Ckpt8(128, 256, codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)))


def test_checkpoint_with_other_tensors(recorder):
    """Codes brought back from elsewhere, a copy with other scales, storage that
    moved: always the memory that the fields have at the call."""
    q = F.Ckpt8.empty(128, 256, "cpu")
    _check_uses(recorder, q)
    q.codes = q.codes.clone()
    _check_uses(recorder, q)
    other = dataclasses.replace(q, scales=q.scales.clone())
    _check_uses(recorder, other)
    _check_uses(recorder, q)
    for again in (copy.copy(q), copy.deepcopy(q), pickle.loads(pickle.dumps(q))):
        _check_uses(recorder, again)
        again.scales = q.scales.clone()
        _check_uses(recorder, again)
        _check_uses(recorder, q)
    q.codes.set_(torch.zeros(128, 256, dtype=torch.uint8))
    _check_uses(recorder, q)


@pytest.mark.parametrize("field,value", [
    ("codes", lambda q: q.codes[:64]), ("codes", lambda q: q.codes.t().contiguous().t()),
    ("codes", lambda q: q.codes.float()), ("codes", lambda q: q.codes.view(-1)), ("codes", lambda q: None),
    ("scales", lambda q: q.scales[:, :4]), ("scales", lambda q: q.scales.expand(2, 128, 8)[0].t().contiguous().t()),
    ("scales", lambda q: q.scales.to(torch.int8)), ("scales", lambda q: q.scales.repeat(1, 2)[:, ::2]),
    ("scales", lambda q: None), ("rows", lambda q: 64), ("cols", lambda q: 512)])
def test_checkpoint_with_unfit_tensors_is_refused(recorder, field, value):
    for i in range(6):
        q = F.Ckpt8.empty(128, 256, "cpu")
        call = _uses(q)[i][2]
        setattr(q, field, value(q))
        with pytest.raises(ValueError):
            call()
    assert not recorder.calls
