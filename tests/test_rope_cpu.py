"""Rotary positions without a GPU: the phases, the frequencies and the refusals."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import exact_attention_92_gb300 as fa
from exact_attention_92_gb300 import _binding
from oracle import rope as oracle

TURN = oracle._TURN


@pytest.fixture(scope="module")
def lib():
    from exact_attention_92_gb300 import build

    build.build()
    return fa.load()


def test_phases_are_fractions_of_a_turn(lib):
    """2^64 f / (2 pi) modulo 2^64, off by the rounding of one division in 64
    bits (2^-53 of the quotient) and half a unit."""
    freq = [1.0, 0.5, 10000.0 ** -0.5, 1e-4, 7.25, 6.283185307179586, 0.0, -0.3, 1e-12, 123456.789]
    for f, p in zip(freq, fa.fa_rope_phases(freq)):
        want = Fraction(f) * TURN
        got = Fraction(p, 1 << 64)
        off = got - want
        off -= round(off)
        # The quotient's rounding, that of 2 pi in 64 bits, and the last place.
        assert abs(off) <= abs(want) * Fraction(2, 1 << 53) + Fraction(1, 1 << 64), f
        assert 0 <= p < 1 << 64


def test_phases_refusals(lib):
    for bad in ([], [math.inf], [1.0, math.nan]):
        with pytest.raises(fa.FaError) as e:
            fa.fa_rope_phases(bad)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    out = (ctypes.c_uint64 * 1)()
    one = (ctypes.c_double * 1)(1.0)
    assert lib.fa_rope_phases(None, 1, out) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_rope_phases(one, 1, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_rope_phases(one, -1, out) == fa.FA_ERR_INVALID_ARG


def test_frequencies():
    plain = fa.rope_frequencies(64, base=10000.0)
    assert len(plain) == 32 and plain[0] == 1.0 and math.isclose(plain[16], 0.01)
    assert fa.rope_frequencies(64, scaling="linear", factor=4) == [f / 4 for f in plain]
    stretched = fa.rope_frequencies(64, scaling="base", factor=4)
    assert stretched[0] == 1.0 and math.isclose(stretched[-1], plain[-1] / 4, rel_tol=1e-12)
    parts = fa.rope_frequencies(64, scaling="by_parts", factor=8, original=4096)
    for f, g in zip(plain, parts):
        turns = 4096 * f / (2 * math.pi)
        if turns >= 32:
            assert g == f
        elif turns <= 1:
            assert g == f / 8
        else:
            assert f / 8 < g < f
    for kw in ({"rot": 7}, {"rot": 0}, {"rot": 8, "base": 0.0}, {"rot": 8, "factor": -1}, {"rot": 8, "scaling": "x"},
               {"rot": 8, "scaling": "by_parts"}, {"rot": 2, "scaling": "base"},
               {"rot": 8, "scaling": "by_parts", "original": 100, "slow": 2, "fast": 2}):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**kw)


def _rows(ptr=0x1000, batch=512, row=64, head=256):
    return ctypes.byref(_binding.Rows(ptr, batch, row, head))


def _call(lib, **kw):
    a = dict(q=_rows(), k=_rows(0x2000), q_out=_rows(0x3000), k_out=_rows(0x4000), phases=0x5000, positions=0x6000,
             start=None, B=1, N=8, H=4, Hkv=2, d=64, rot=64, interleaved=0, mscale=1.0, inverse=0)
    a.update(kw)
    return lib.fa_rope(*a.values(), None)


def test_argument_errors_without_a_device(lib):
    inv, uns = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
    for bad in (dict(q=None), dict(q_out=None), dict(k_out=None), dict(phases=None), dict(phases=0x5004),
                dict(positions=0x6002), dict(positions=None, start=0x6001), dict(start=0x6000),
                dict(q=_rows(0)), dict(q=_rows(0x1008)), dict(q=_rows(row=12)), dict(q_out=_rows(head=4)),
                dict(k=_rows(batch=1)), dict(k_out=_rows(0x4004)), dict(B=0), dict(N=0), dict(H=0), dict(Hkv=0),
                dict(B=1 << 16, N=1 << 16), dict(H=1 << 21), dict(rot=0), dict(rot=63), dict(rot=66), dict(rot=-2),
                dict(mscale=math.inf), dict(mscale=math.nan)):
        assert _call(lib, **bad) == inv, bad
    for d in (32, 48, 192, 0, -64):
        assert _call(lib, d=d, rot=16) == uns
    # Well-formed arguments get as far as the device (none here, or null pointers to it are not followed).
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        assert _call(lib) in (fa.FA_ERR_CUDA, uns)
        assert _call(lib, k=None, k_out=None, Hkv=0, positions=None) in (fa.FA_ERR_CUDA, uns)


def test_binding_refuses_what_is_no_tensor(lib):
    pytest.importorskip("torch")
    for bad in (None, 3, [1.0]):
        with pytest.raises(TypeError):
            fa.fa_rope(bad, bad, bad, bad, bad)


def test_oracle_turns_by_whole_positions():
    """The oracle against complex powers at small positions, and a whole number
    of turns far out."""
    freq = [1.0, 0.25]
    th = oracle.angles(np.array([0, 1, 5]), freq)
    assert np.allclose(np.exp(1j * th), np.exp(1j * np.array([[0, 0], [1, 0.25], [5, 1.25]])), atol=1e-15)
    x = np.random.default_rng(0).standard_normal((3, 6))
    for inter in (False, True):
        y = oracle.rotate(x, th, 4, inter, 2.0)
        z = oracle.rotate(y, th, 4, inter, 0.5, inverse=True)
        assert np.allclose(z, x, atol=1e-14) and np.array_equal(y[:, 4:], x[:, 4:])
        lo, hi = ((0, 1) if inter else (0, 2))
        assert np.isclose(y[1, lo], 2 * (x[1, lo] * math.cos(1) - x[1, hi] * math.sin(1)))
        assert np.isclose(y[1, hi], 2 * (x[1, hi] * math.cos(1) + x[1, lo] * math.sin(1)))
