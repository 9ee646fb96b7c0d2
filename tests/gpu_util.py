"""Helpers shared by the GPU parity tests (device moves, oracle inputs)."""
import numpy as np
import pytest
import torch

TOL = {"f16": 2e-3, "bf16": 2e-3, "fp8": 2e-2, "int8": 2e-2}

requires_cuda = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")


def np_exact(t):
    """CPU numpy copy of a tensor with every value exact (bf16 -> float32)."""
    t = t.detach().cpu()
    if t.dtype == torch.bfloat16:
        return t.float().numpy()
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8).numpy()
    return t.numpy()


def half_ulp(x, dtype):
    """Half a unit in the last place of |x| in a 16-bit float dtype."""
    mant = 10 if dtype == torch.float16 else 7
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -14)))
    return 0.5 * 2.0 ** (e - mant)


class PointerSpy:
    """The library, with every address that a call passes kept in `seen`."""

    def __init__(self, lib):
        self._lib, self.seen = lib, set()

    def __getattr__(self, name):
        f = getattr(self._lib, name)

        def call(*args):
            self.seen |= {getattr(a, "value", a) for a in args if isinstance(getattr(a, "value", a), int)}
            return f(*args)
        return call


def held_by_a_call_on_another_stream(monkeypatch, ops, call):
    """call(stream) returns its result, as a copy on the host.  While a call on a
    stream that is still busy has yet to run, with its result dropped, memory that
    the current stream allocates is none that the call was given.  (Nothing is
    written to it: a call that let go of its scratch would fail here, not go astray.)
    Returns the results on the current stream and on the other."""
    plain = [x.cpu() for x in call(None)]
    torch.cuda.synchronize()  # (scratch and results of that call are free, and would be taken again)
    spy = PointerSpy(ops.lib())
    monkeypatch.setattr(ops, "_lib", spy)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    call(s)
    assert not s.query(), "the stream was not busy"
    again = [torch.empty(1 << b, dtype=torch.uint8, device="cuda") for b in range(6, 26) for _ in range(3)]
    again += [torch.empty_like(x, device="cuda") for x in plain for _ in range(3)]
    assert not {x.data_ptr() for x in again if x.numel()} & spy.seen
    s.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000)
    other = call(s)
    s.synchronize()
    return plain, [x.cpu() for x in other]


def assert_close(got, want, tol, what=""):
    got = np.asarray(got, dtype=np.float64)
    err = np.abs(got - want)
    worst = float(err.max()) if err.size else 0.0
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    assert worst <= tol, f"{what}: max abs err {worst:.3e} > {tol:.1e}"
    return worst
