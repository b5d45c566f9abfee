"""Packed sequences without a GPU: the oracle against a plain statement, and the refusals."""

import ctypes
import math
import os

import numpy as np
import pytest

import exact_attention_92_gb300 as fa
from exact_attention_92_gb300 import _binding, build
from oracle import packed as oracle


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load()


def test_oracle_forward():
    """Row by row over the keys that each row sees, in Python sums."""
    r = np.random.default_rng(0)
    cu_q, cu_k, used = [1, 4, 4, 6], [0, 5, 7, 10], [4, 2, 1]
    q, k, v = r.standard_normal((7, 4, 3)), r.standard_normal((10, 2, 3)), r.standard_normal((10, 2, 3))
    pre = (r.standard_normal((2, 2, 3)), r.standard_normal((2, 2, 3)))
    for causal in ("none", "top_left", "bottom_right"):
        for prefix in (None, pre):
            got = oracle.forward(q, k, v, cu_q, cu_k, 0.7, causal, used, prefix)
            assert not got["o"][[0, 6]].any() and np.isneginf(got["lse"][:, [0, 6]]).all()
            for b in range(3):
                nq, nk = cu_q[b + 1] - cu_q[b], used[b]
                for i in range(nq):
                    for h in range(4):
                        keys = [(pre[0][j, h // 2], pre[1][j, h // 2]) for j in range(2)] if prefix else []
                        last = {"none": nk - 1, "top_left": i, "bottom_right": i + nk - nq}[causal]
                        keys += [(k[cu_k[b] + j, h // 2], v[cu_k[b] + j, h // 2]) for j in range(min(nk, last + 1))]
                        row = q[cu_q[b] + i, h]
                        w = [math.exp(0.7 * float(row @ x)) for x, _ in keys]
                        if not w:
                            assert np.isneginf(got["lse"][h, cu_q[b] + i]) and not got["o"][cu_q[b] + i, h].any()
                            continue
                        assert math.isclose(got["lse"][h, cu_q[b] + i], math.log(sum(w)), rel_tol=1e-12, abs_tol=1e-12)
                        want = sum(a * y for a, (_, y) in zip(w, keys)) / sum(w)
                        assert np.allclose(got["o"][cu_q[b] + i, h], want, atol=1e-13)


def test_oracle_gradients_against_differences():
    """Central differences of sum(dO * O)."""
    r = np.random.default_rng(0)
    q, k, v, do = (r.standard_normal((7, h, 5)) for h in (4, 2, 2, 4))
    cu_q, cu_k = [0, 3, 7], [0, 2, 7]
    for causal in ("none", "top_left", "bottom_right"):
        want = oracle.backward(q, k, v, do, cu_q, cu_k, 0.4, causal)
        for name, x in (("dq", q), ("dk", k), ("dv", v)):
            for at in ((0, 0, 0), (2, 1, 3), (6, 1, 4), (4, 0, 2)):
                keep, vals = x[at], []
                for h in (1e-5, -1e-5):
                    x[at] = keep + h
                    vals.append((do * oracle.forward(q, k, v, cu_q, cu_k, 0.4, causal)["o"]).sum())
                x[at] = keep
                assert abs((vals[0] - vals[1]) / 2e-5 - want[name][at]) <= 1e-7 * (1 + abs(want[name][at]))


def _rows(ptr, row=256, head=64):
    return ctypes.byref(_binding.Rows(ptr, 0, row, head))


def _fwd(lib, **kw):
    a = dict(q=_rows(0x10000), k=_rows(0x20000), v=_rows(0x30000), o=_rows(0x40000), lse=0x50000, cu_q=0x60000,
             cu_k=0x70000, used=None, B=2, Tq=10, Tk=12, H=4, Hkv=4, d=64, causal=0, scale=0.125)
    a.update(kw)
    return lib.fa_packed_fwd(*a.values(), None)


def _prefix(lib, **kw):
    a = dict(q=_rows(0x10000), kp=_rows(0x80000), vp=_rows(0x90000), k=_rows(0x20000), v=_rows(0x30000), o=_rows(0x40000),
             lse=0x50000, cu_q=0x60000, cu_k=0x70000, used=None, B=2, P=5, Tq=10, Tk=12, H=4, Hkv=4, d=64, causal=0,
             scale=0.125)
    a.update(kw)
    return lib.fa_prefix_fwd(*a.values(), None)


def test_argument_errors_without_a_device(lib):
    inv, uns = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    bad = [dict(q=None), dict(k=None), dict(v=_rows(0)), dict(o=_rows(0x40008)), dict(lse=0), dict(lse=0x50004),
           dict(cu_q=None), dict(cu_k=0x70002), dict(used=0x1001), dict(B=0), dict(B=-1), dict(Tq=0), dict(Tk=-1), dict(H=0),
           dict(Hkv=0), dict(Hkv=3), dict(causal=3), dict(causal=-1), dict(scale=0.0), dict(scale=math.nan),
           dict(scale=math.inf), dict(q=_rows(0x10000, row=0)), dict(k=_rows(0x20000, head=-64)),
           dict(v=_rows(0x30000, row=260)), dict(k=_rows(0x20000, row=1 << 40)), dict(o=_rows(0x40000, row=64)),
           dict(o=_rows(0x40000, row=128, head=128)), dict(Tq=(1 << 30) + 1), dict(Tk=(1 << 30) + 1),
           dict(Tq=1 << 30, H=1 << 12, Hkv=1 << 12, q=_rows(0x10000, 1 << 20, 64), o=_rows(0x40000, 1 << 20, 64))]
    for kw in bad:
        got = _fwd(lib, **kw)
        assert got == inv or (got in (fa.FA_ERR_CUDA, uns) and kw.get("H") == 1 << 12), (kw, got)
        assert _prefix(lib, **kw) == got, kw
    for kw in (dict(P=0), dict(P=-3), dict(kp=None), dict(vp=_rows(0x90008)), dict(kp=_rows(0x80000, row=0))):
        assert _prefix(lib, **kw) == inv, kw
    for d in (32, 80, 192, 256, 0):
        assert _fwd(lib, d=d) == uns and _prefix(lib, d=d) == uns
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        # Well-formed calls get as far as the device.
        for kw in ({}, dict(Tk=0, k=None, v=None), dict(o=_rows(0x40000, row=64, head=640)),
                   dict(H=1, Hkv=1, q=_rows(0x10000, 64, 0), o=_rows(0x40000, 64, 1)), dict(Tq=1, q=_rows(0x10000, 0, 64))):
            assert _fwd(lib, **kw) in (fa.FA_ERR_CUDA, uns), kw


def _bwd(lib, **kw):
    a = dict(q=_rows(0x10000), k=_rows(0x20000), v=_rows(0x30000), o=_rows(0x40000), lse=0x50000, dout=_rows(0x80000),
             dq=_rows(0x90000), dk=_rows(0xa0000), dv=_rows(0xb0000), cu_q=0x60000, cu_k=0x70000, B=2, Tq=10, Tk=12, H=4,
             Hkv=4, d=64, causal=0, scale=0.125)
    a.update(kw)
    return lib.fa_packed_bwd(*a.values(), None)


def test_backward_argument_errors_without_a_device(lib):
    inv, uns = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for kw in (dict(q=None), dict(k=_rows(0)), dict(v=None), dict(o=None), dict(lse=0), dict(dout=_rows(0x80001)),
               dict(dq=None), dict(dk=_rows(0xa0008)), dict(dv=None), dict(cu_q=0), dict(cu_k=0x70001), dict(B=0), dict(Tq=0),
               dict(Tk=0), dict(H=0), dict(Hkv=3), dict(H=65536, Hkv=65536), dict(causal=4), dict(scale=-1.0),
               dict(dq=_rows(0x90000, row=128)), dict(dk=_rows(0xa0000, row=64)), dict(dv=_rows(0xb0000, row=0)),
               dict(dout=_rows(0x80000, head=12)), dict(Tk=(1 << 30) + 1)):
        assert _bwd(lib, **kw) == inv, kw
    for d in (32, 256):
        assert _bwd(lib, d=d) == uns
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        assert _bwd(lib) in (fa.FA_ERR_CUDA, uns)


def test_binding_refuses_what_is_no_tensor(lib):
    pytest.importorskip("torch")
    for bad in (None, 3, [1.0]):
        with pytest.raises(TypeError):
            fa.fa_packed_fwd(bad, bad, bad, bad, bad, bad, bad)
        with pytest.raises(TypeError):
            fa.fa_prefix_fwd(bad, bad, bad, bad, bad, bad, bad, bad, bad)


def _native():
    torch = pytest.importorskip("torch")
    native = _binding._native_caller(torch.__version__, "._packed_call", "the calls on packed sequences")
    assert native is not None, "the native caller is built where torch is installed"
    return native


def test_native_caller_checks_its_numbers(lib):
    native = _native()
    for call in (native.bind, native.rope, native.forward, native.backward):
        for args in ((), (1, 2), (None,) * 30):
            with pytest.raises(TypeError):
                call(*args)


@pytest.mark.parametrize("native", [True, False])
def test_binding_refuses_host_tensors(lib, native, monkeypatch):
    torch = pytest.importorskip("torch")
    if not native:
        monkeypatch.setattr(_binding, "_packed", False)
    q = torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    cu, lse = torch.tensor([0, 2, 6], dtype=torch.int32), torch.zeros(2, 6)
    for call in (lambda: fa.fa_packed_fwd(q, q, q, q, lse, cu, cu), lambda: fa.fa_prefix_fwd(q, q, q, q, q, q, lse, cu, cu),
                 lambda: fa.fa_packed_bwd(q, q, q, q, lse, q, q, q, q, cu, cu),
                 lambda: fa.fa_rope(q, q, q, q, torch.zeros(32, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()


def test_build_does_without_a_native_caller(lib, monkeypatch, tmp_path):
    """A compiler that is not there costs the native caller only; one of an older source is not left behind."""
    pytest.importorskip("torch")
    cxx = tmp_path / "cxx"
    cxx.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\necho made > "$2"\n')
    cxx.chmod(0o755)
    monkeypatch.setenv("CXX", str(cxx))
    monkeypatch.setattr(build, "PACKED_CALL", str(tmp_path / "_packed_call.so"))
    assert build.build_packed_call() == build.PACKED_CALL
    os.utime(build.PACKED_CALL, (1, 1))
    monkeypatch.setenv("CXX", "/nonexistent/c++")
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build_packed_call() is None
    assert not os.path.exists(build.PACKED_CALL)
