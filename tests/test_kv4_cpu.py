"""The 4-bit key/value cache without a GPU: pins of its oracle, and the
refusals that the host makes before any device work."""

import ctypes
import itertools
import os

import numpy as np
import pytest

import exact_attention_92_gb300 as fa
from exact_attention_92_gb300 import _binding, build
from oracle import kv4

P = ctypes.c_void_p
DIMS = (64, 96, 128, 256)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fa.load()


# ------------------------------------------------------------------ oracle

@pytest.mark.parametrize("d", DIMS)
def test_a_block_has_a_place_for_everything(d):
    """Every nibble and every scale byte of a block belongs to exactly one
    channel of one token."""
    seen = set()
    for p, c in itertools.product(range(16), range(d)):
        for place in (kv4.key_place(d, p, c), kv4.value_place(d, p, c)):
            assert place not in seen
            seen.add(place)
    assert seen == {(b, s) for b in range(16 * d) for s in (0, 4)}
    scales = {kv4.scale_place(d, p, w, g) for p in range(16) for w in range(2) for g in range(d // 32)}
    assert scales == set(range(16 * d, 18 * d, 2))


def test_levels_round_to_nearest_with_ties_to_even():
    """With a largest value of 6 the scale is 1, so the codes are those of
    e2m1 itself: each border between two levels goes to the even code."""
    x = np.zeros(32)
    x[:15] = [6, 0.25, 0.26, 0.75, 0.74, 1.25, 1.26, 1.75, 2.5, 2.52, 3.5, 3.48, 5.0, 5.03, -0.75]
    code, bits = kv4.quantise(x)
    assert kv4.bits_value(bits).tolist() == [1.0]
    assert code[:15].tolist() == [7, 0, 1, 2, 1, 2, 3, 4, 4, 5, 6, 5, 6, 7, 8 | 2]
    assert (code[15:] == 0).all()
    assert kv4.values(code, bits)[:8].tolist() == [6, 0, 0.5, 1, 0.5, 1, 1.5, 2]


def test_scale_is_the_rounded_sixth_of_the_largest():
    x = np.zeros((3, 32))
    x[0, 3], x[1, 4], x[2, 5] = -7.0, 1.0, 2.0 ** -125
    code, bits = kv4.quantise(x)
    s = kv4.bits_value(bits)[:, 0]
    assert abs(s[0] - 7 / 6) <= 2.0 ** -8 and abs(s[1] - 1 / 6) <= 2.0 ** -11
    assert s[2] == 0.0 and (code[2] == 0).all()  # a scale below 2^-126
    assert code[0, 3] == 15 and code[1, 4] == 7


def test_a_group_with_a_non_finite_value_reads_as_nan():
    x = np.ones((2, 64))
    x[0, 5], x[1, 40] = np.inf, np.nan
    v = kv4.held(x)
    assert np.isnan(v[0, :32]).all() and np.isfinite(v[0, 32:]).all()
    assert np.isfinite(v[1, :32]).all() and np.isnan(v[1, 32:]).all()


def test_error_of_a_held_value():
    """A value below the largest level is off by at most half the widest gap
    (one scale), and the scale by half a step of bf16."""
    x = kv4.to_bf16(np.random.default_rng(0).standard_normal((200, 128)) * 3)
    top = np.abs(x.reshape(200, 4, 32)).max(-1)
    err = np.abs(kv4.held(x) - x).reshape(200, 4, 32).max(-1)
    # Half the gap from 4 to 6 is one scale, a sixth of the largest value;
    # the scale's rounding moves the largest level by at most 2^-8 of itself.
    assert (err <= top / 6 * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("d", DIMS)
def test_write_then_read(d):
    rng = np.random.default_rng(d)
    page, Hkv = 32, 2
    cache = np.full((5, Hkv, page * 9 * d // 8), 0xAB, np.uint8)
    before = cache.copy()
    table = [[3, 1], [4, 0]]
    k, v = (kv4.to_bf16(rng.standard_normal((2, Hkv, 20, d))) for _ in range(2))
    kv4.write(cache, table, [25, 0], [20, 7], k, v, page)
    for b, first, n in ((0, 25, 20), (1, 0, 7)):
        rk, rv = kv4.read(cache, table[b], n, page, d, first)
        assert np.array_equal(rk, kv4.held(k[b, :, :n])) and np.array_equal(rv, kv4.held(v[b, :, :n]))
    assert np.array_equal(cache[2], before[2])
    # 27 tokens of 2 heads, 9 d / 8 bytes each, may have changed.
    assert (cache != before).sum() <= 27 * Hkv * 9 * d // 8
    assert (cache != before).any(axis=(1, 2)).tolist() == [False, True, False, True, True]


def test_bf16_rounding_of_the_oracle():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).standard_normal(4000).astype(np.float32) * np.float32(2.0) ** np.arange(-100, 100).repeat(20)
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(kv4.to_bf16(x.astype(np.float64)), want)


def test_planted_mistakes_in_the_oracle_show():
    """Two places exchanged, or a level changed, do not survive the pins."""
    assert kv4.value_place(128, 2, 0) != kv4.value_place(128, 4, 0)
    wrong = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 5.0])
    x = np.zeros(32)
    x[0] = 6
    code, bits = kv4.quantise(x)
    keep = kv4.LEVELS
    try:
        kv4.LEVELS = wrong
        assert kv4.values(code, bits)[0] != 6
    finally:
        kv4.LEVELS = keep


# ---------------------------------------------------------------- refusals

def test_cache_bytes(lib):
    for d in DIMS:
        assert fa.fa_kv4_cache_bytes(10, 8, 64, d) == 10 * 8 * 64 * 9 * d // 8
    assert fa.fa_kv4_cache_bytes(2 ** 31 - 1, 64, 1024, 256) == (2 ** 31 - 1) * 64 * 1024 * 288
    n = ctypes.c_uint64()
    for args, want in (((0, 8, 64, 128), fa.FA_ERR_INVALID_ARG), ((1, 0, 64, 128), fa.FA_ERR_INVALID_ARG),
                       ((1, 1, 8, 128), fa.FA_ERR_INVALID_ARG), ((1, 1, 48, 128), fa.FA_ERR_INVALID_ARG),
                       ((1, 1, 2048, 128), fa.FA_ERR_INVALID_ARG), ((1, 1, -16, 128), fa.FA_ERR_INVALID_ARG),
                       ((1, 1, 64, 80), fa.FA_ERR_UNSUPPORTED), ((1, 1, 64, 0), fa.FA_ERR_UNSUPPORTED)):
        assert lib.fa_kv4_cache_bytes(*args, ctypes.byref(n)) == want
    assert lib.fa_kv4_cache_bytes(1, 1, 64, 128, None) == fa.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FaError):
        fa.fa_kv4_cache_bytes(1, 1, 64, 80)


SIZES = dict(B=2, Hkv=4, N=8, d=128, num_pages=100, page_size=64, max_pages=10)


def _bad_sizes():
    for name in ("B", "Hkv", "N", "num_pages", "max_pages"):
        for x in (0, -1):
            yield {name: x}, "FA_ERR_INVALID_ARG"
    for x in (0, 8, 17, 96, 2048, -64):
        yield {"page_size": x}, "FA_ERR_INVALID_ARG"
    for x in (0, 32, 80, 512, -128):
        yield {"d": x}, "FA_ERR_UNSUPPORTED"
    yield {"max_pages": 1 << 26, "page_size": 32}, "FA_ERR_INVALID_ARG"   # 2^31 positions
    yield {"max_pages": (1 << 25) + 1, "page_size": 32}, "FA_ERR_INVALID_ARG"
    yield {"B": 1, "Hkv": 1, "N": (1 << 30) + 1}, "FA_ERR_INVALID_ARG"
    yield {"B": 1 << 16, "Hkv": 1 << 10, "N": 1 << 10}, "FA_ERR_INVALID_ARG"  # 2^36 rows


@pytest.mark.parametrize("change,want", list(_bad_sizes()))
def test_write_and_read_refuse_sizes(lib, change, want):
    s = list({**SIZES, **change}.values())
    ptrs = [P(0x1000 * (i + 1)) for i in range(6)]
    assert lib.fa_kv4_write(*ptrs, *s, None) == getattr(fa, want)
    assert lib.fa_kv4_read(*ptrs, *s, None) == getattr(fa, want)


def test_write_and_read_refuse_pointers(lib):
    s = list(SIZES.values())
    good = [P(0x1000 * (i + 1)) for i in range(6)]
    # Order: k, v, cache, table, start, count / cache, table, start, count, k, v.
    for call, wide, optional in ((lib.fa_kv4_write, {0, 1, 2}, 5), (lib.fa_kv4_read, {0, 4, 5}, 3)):
        for i in range(6):
            bad = list(good)
            bad[i] = P(0x1000 * (i + 1) + (8 if i in wide else 2))
            assert call(*bad, *s, None) == fa.FA_ERR_INVALID_ARG, i
            if i != optional:
                bad[i] = P(0)
                assert call(*bad, *s, None) == fa.FA_ERR_INVALID_ARG, i


FWD = dict(B=2, H=32, Hkv=4, Nq=2, d=128, num_pages=100, page_size=64, max_pages=10, causal=2)


def _fwd(lib, ptrs=None, scale=0.1, **change):
    s = list({**FWD, **change}.values())
    return lib.fa_kv4_fwd(*(ptrs or [P(0x1000 * (i + 1)) for i in range(6)]), *s, scale, None)


def test_fwd_refusals(lib):
    for name in ("B", "H", "Hkv", "Nq", "num_pages", "max_pages"):
        assert _fwd(lib, **{name: 0}) == fa.FA_ERR_INVALID_ARG, name
        assert _fwd(lib, **{name: -4}) == fa.FA_ERR_INVALID_ARG, name
    assert _fwd(lib, Hkv=3) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, page_size=24) == fa.FA_ERR_INVALID_ARG
    for causal in (-1, 3):
        assert _fwd(lib, causal=causal) == fa.FA_ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _fwd(lib, scale=scale) == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, d=80) == fa.FA_ERR_UNSUPPORTED
    assert _fwd(lib, Nq=17) == fa.FA_ERR_UNSUPPORTED       # 8 * 17 rows > 128
    assert _fwd(lib, B=1 << 20, H=1 << 10, Hkv=1 << 10, Nq=4) == fa.FA_ERR_INVALID_ARG  # 2^32 rows
    for i in range(6):
        ptrs = [P(0x1000 * (j + 1)) for j in range(6)]
        ptrs[i] = P(0)
        assert _fwd(lib, ptrs) == fa.FA_ERR_INVALID_ARG
        ptrs[i] = P(0x1000 * (i + 1) + (2 if i in (2, 3) else 8))
        assert _fwd(lib, ptrs) == fa.FA_ERR_INVALID_ARG


def test_selftest_refuses_what_the_call_refuses(lib):
    ptrs = [P(0x1000 * (i + 1)) for i in range(6)]
    s = [FWD[n] for n in ("B", "H", "Hkv", "Nq", "d", "num_pages", "page_size", "max_pages")]
    assert lib.fa_selftest_kv4_timeout(*ptrs, *s, 2_000_000_001, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_selftest_kv4_timeout(*ptrs, 0, *s[1:], 1000, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_selftest_kv4_timeout(*ptrs[:5], P(0), *s, 1000, None) == fa.FA_ERR_INVALID_ARG
    assert lib.fa_selftest_kv4_timeout(*ptrs, *s[:3], 17, *s[4:], 1000, None) == fa.FA_ERR_UNSUPPORTED


PLANS = [
    # B, H, Hkv, Nq, d, page_size, max_pages
    (1, 1, 1, 1, 64, 16, 1), (1, 32, 8, 1, 128, 16, 3), (8, 32, 8, 1, 128, 64, 128), (64, 32, 8, 1, 128, 64, 256),
    (9, 12, 4, 5, 96, 32, 188), (16, 64, 4, 1, 256, 64, 128), (3, 8, 1, 16, 128, 1024, 7), (1500, 2, 1, 1, 64, 16, 3),
    (16, 64, 8, 2, 128, 64, 125), (16, 64, 8, 2, 64, 64, 62), (2, 5, 1, 1, 128, 16, 17), (2, 4, 1, 1, 256, 16, 16), (1, 16, 2, 1, 256, 256, 4096),
    (16, 24, 1, 1, 64, 64, 500), (16, 20, 1, 1, 96, 64, 500), (16, 24, 1, 1, 128, 64, 500),
]


@pytest.mark.parametrize("sizes", PLANS)
@pytest.mark.parametrize("sm_count", (1, 152))
def test_plan(lib, sizes, sm_count):
    B, H, Hkv, Nq, d, page, pages = sizes
    pl = fa.fa_kv4_fwd_plan(*sizes, sm_count)
    assert pl["rows"] == H // Hkv * Nq
    steps = B * Hkv * -(-pl["rows"] // 8) * pl["max_steps"] // sm_count
    many, least = (24, 280 if d == 64 else 160) if 16 < pl["rows"] <= 24 and d <= 96 else (16, 160)
    assert pl["unit_rows"] == (4 if pl["rows"] <= 4 else many if pl["rows"] > 8 and d < 256 and steps >= least else 8)
    assert pl["row_blocks"] * pl["unit_rows"] >= pl["rows"] > (pl["row_blocks"] - 1) * pl["unit_rows"]
    assert pl["units"] == B * Hkv * pl["row_blocks"]
    assert pl["max_steps"] * pl["step_keys"] >= page * pages > (pl["max_steps"] - 1) * pl["step_keys"]
    assert 1 <= pl["grid"] <= sm_count
    assert pl["grid"] == min(sm_count, pl["units"] * (1 if pl["whole"] else pl["max_steps"]))
    assert pl["launches"] == (1 if pl["whole"] else 2)
    part = pl["unit_rows"] * (4 * d + 8)
    if pl["whole"]:
        assert pl["workspace_bytes"] == 0
    else:
        assert 2 * pl["grid"] * part < pl["workspace_bytes"] <= pl["grid"] * (2 * part + 64)


def test_plan_refusals(lib):
    good = (2, 32, 4, 2, 128, 64, 10, 152)
    fa.fa_kv4_fwd_plan(*good)
    for i, bad, want in ((0, 0, 1), (1, 0, 1), (2, 3, 1), (3, 0, 1), (3, 17, 2), (4, 80, 2), (5, 20, 1), (6, 0, 1), (7, 0, 1)):
        args = list(good)
        args[i] = bad
        with pytest.raises(fa.FaError) as e:
            fa.fa_kv4_fwd_plan(*args)
        assert e.value.status == want, (i, bad)
    # Units times steps beyond 31 bits.
    with pytest.raises(fa.FaError) as e:
        fa.fa_kv4_fwd_plan(1 << 12, 32, 32, 1, 128, 1024, 1 << 10, 152)
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    assert _fwd(lib, B=1 << 12, H=32, Hkv=32, Nq=1, page_size=1024, max_pages=1 << 10) == fa.FA_ERR_INVALID_ARG
    args = [*good, None]
    assert lib.fa_kv4_fwd_plan(*args) == fa.FA_ERR_INVALID_ARG


def test_launch_count_and_status_name(lib):
    assert fa.fa_strerror(fa.FA_ERR_BAD_INDEX).startswith("FA_ERR_BAD_INDEX")
    n = ctypes.c_uint64(7)
    for kid in (fa.FA_KERNEL_KV4_WRITE, fa.FA_KERNEL_KV4_READ, fa.FA_KERNEL_KV4_FWD, fa.FA_KERNEL_KV4_MERGE):
        assert lib.fa_launch_count(kid, ctypes.byref(n)) == fa.FA_OK
    for kid in (5, 6, 7, 12):
        assert lib.fa_launch_count(kid, ctypes.byref(n)) == fa.FA_ERR_INVALID_ARG


@pytest.fixture(params=["native", "ctypes"])
def caller(lib, request, monkeypatch):
    """The binding with its native caller, and with the one that does without."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(_binding, "_torch", torch)
    made = _binding._kv4_caller()
    if request.param == "native":
        assert made.__name__.endswith("_kv4_call"), "the native caller is built where torch is installed"
    else:
        made = _binding._Kv4Ctypes(lib)
    monkeypatch.setattr(_binding, "_kv4", made)
    return made


def test_callers_refuse_what_is_no_tensor(caller):
    for bad in (None, 3, "x", [1]):
        assert caller.move(True, bad, bad, bad, bad, bad, None, 0) == -1
        assert caller.fwd(bad, bad, bad, bad, bad, bad, 0, None, 0) == -1
        with pytest.raises(TypeError):
            fa.fa_kv4_write(bad, bad, bad, bad, bad)
        with pytest.raises(TypeError):
            fa.fa_kv4_fwd(bad, bad, bad, bad, bad, bad)
    with pytest.raises(ValueError):
        fa.fa_kv4_fwd(None, None, None, None, None, None, causal="sideways")


def _cuda():
    import torch

    return torch.cuda.is_available()


def test_native_caller_checks_its_numbers(lib):
    pytest.importorskip("torch")
    native = _binding._kv4_caller()
    for args in ((), (1, 2), (None,) * 10):
        with pytest.raises(TypeError):
            native.fwd(*args)
        with pytest.raises(TypeError):
            native.move(*args)
        with pytest.raises(TypeError):
            native.bind(*args)
    for causal, scale, stream in (("x", None, None), (0, "x", None), (0, None, "x")):
        if causal == 0 and scale is None and not _cuda():
            continue  # without a device the stream is not looked at
        with pytest.raises(TypeError):
            native.fwd(*(None,) * 6, causal, scale, stream)


def test_binding_refuses_host_tensors(caller):
    torch = pytest.importorskip("torch")
    k = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(3, 2, 16 * 72, dtype=torch.uint8)
    table = torch.zeros(1, 1, dtype=torch.int32)
    lens = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.fa_kv4_write(k, k, cache, table, lens)
    with pytest.raises(ValueError):
        fa.fa_kv4_read(cache, table, lens, k, k)
    with pytest.raises(ValueError):
        fa.kv4_forward(k, cache, table, lens)
    assert fa.kv4_cache(3, 2, 16, 64, device="cpu").shape == cache.shape
    with pytest.raises(fa.FaError):
        fa.kv4_cache(3, 2, 24, 64, device="cpu")


# ------------------------------------------------------------ native caller

@pytest.fixture
def caller_build(lib, monkeypatch, tmp_path):
    """The build of the native caller with a compiler that only notes that it
    ran, and its product elsewhere."""
    pytest.importorskip("torch")
    runs = tmp_path / "runs"
    cxx = tmp_path / "cxx"
    cxx.write_text("#!/bin/sh\n"
                   f"echo run >> {runs}\n"
                   'while [ "$1" != -o ]; do shift; done\n'
                   'echo made > "$2"\n')
    cxx.chmod(0o755)
    monkeypatch.setenv("CXX", str(cxx))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_kv4_call.so"))
    return lambda: len(runs.read_text().split()) if runs.exists() else 0


@pytest.mark.parametrize("cxx", ("/bin/false", "/nonexistent/c++"))
def test_build_does_without_a_native_caller(caller_build, monkeypatch, cxx):
    """A compiler that fails, or is not there, costs the native caller only; one
    of an older source is not left behind."""
    assert build.build_call() == build.CALL
    os.utime(build.CALL, (1, 1))
    monkeypatch.setenv("CXX", cxx)
    for _ in range(2):
        with pytest.warns(UserWarning, match="ctypes"):
            assert build.build() == build.LIB
        assert not os.path.exists(build.CALL)


def test_native_caller_is_compiled_again_for_another_torch(caller_build, monkeypatch):
    import importlib.metadata

    assert build.build_call() == build.CALL and caller_build() == 1
    assert build.build_call() == build.CALL and caller_build() == 1
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "1.0")
    assert build.build_call() == build.CALL and caller_build() == 2
    assert build.build_call() == build.CALL and caller_build() == 2
    os.remove(build.CALL + ".key")
    assert build.build_call() == build.CALL and caller_build() == 3


def test_native_caller_is_this_pythons(lib):
    import sysconfig

    assert build.CALL.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_native_caller_of_another_torch_is_not_used(lib, monkeypatch):
    torch = pytest.importorskip("torch")
    native = _binding._native_caller(torch.__version__)
    assert native is not None
    with pytest.warns(UserWarning, match="1.0.0"):
        assert _binding._native_caller("1.0.0+cu1") is None
    monkeypatch.setattr(_binding, "_kv4", None)
    monkeypatch.setattr(native, "torch_version", "1.0.0")
    with pytest.warns(UserWarning, match="1.0.0"):
        assert isinstance(_binding._kv4_caller(), _binding._Kv4Ctypes)


# ------------------------------------------------------- sizes beyond an int

@pytest.mark.parametrize("i", range(4))
def test_cache_bytes_refuses_sizes_beyond_an_int(lib, i):
    args = [10, 8, 64, 128]
    for off in (2 ** 32, -2 ** 32):
        args[i] += off
        with pytest.raises(fa.FaError) as e:
            fa.fa_kv4_cache_bytes(*args)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
        args[i] -= off


@pytest.mark.parametrize("i", range(8))
def test_plan_refuses_sizes_beyond_an_int(lib, i):
    args = [2, 32, 4, 2, 128, 64, 10, 152]
    args[i] += 2 ** 32
    with pytest.raises(fa.FaError) as e:
        fa.fa_kv4_fwd_plan(*args)
    assert e.value.status == fa.FA_ERR_INVALID_ARG


def test_ctypes_caller_refuses_sizes_beyond_an_int(lib, monkeypatch):
    """A block table of more than 2^31 columns (tensors without memory stand in
    for it) is refused like the native caller does, not cut to its low bits."""
    torch = pytest.importorskip("torch")

    class Lib:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    class Meta(torch.Tensor):  # a tensor without memory that says it is on the device
        is_cuda = True

        def get_device(self):
            return 0

    def meta(*shape, dtype=torch.int32):
        return torch.empty(shape, dtype=dtype, device="meta").as_subclass(Meta)

    monkeypatch.setattr(_binding, "_torch", torch)
    monkeypatch.setattr(_binding, "_device_and_stream", lambda stream: (0, 0))
    made = _binding._Kv4Ctypes(Lib())
    k = meta(1, 2, 4, 64, dtype=torch.bfloat16)
    cache, table, one = meta(3, 2, 16 * 72, dtype=torch.uint8), meta(1, 2 ** 32 + 5), meta(1)
    with pytest.raises(AssertionError):  # the stand-ins are good tensors otherwise
        made.move(True, k, k, cache, meta(1, 5), one, None, 0)
    assert made.move(True, k, k, cache, table, one, None, 0) == -1
    assert made.move(False, k, k, cache, table, one, None, 0) == -1
    q, lse = meta(1, 4, 1, 64, dtype=torch.bfloat16), meta(1, 4, 1, dtype=torch.float32)
    assert made.fwd(q, cache, table, one, q, lse, 0, None, 0) == -1
    with pytest.raises(ValueError, match="block_table has a size"):
        _binding._kv4_refuse_fwd("fa_kv4_fwd", -1, q, cache, table, one, q, lse)


def test_cache_bytes_beyond_64_bits_are_refused(lib):
    n = ctypes.c_uint64(5)
    big = 2 ** 31 - 1
    for args in ((big, big, 1024, 256), (big, big, 16, 64), (big, 2 ** 14, 1024, 256)):
        exact = args[0] * args[1] * args[2] * 9 * args[3] // 8
        want = fa.FA_OK if exact < 2 ** 63 else fa.FA_ERR_INVALID_ARG
        assert lib.fa_kv4_cache_bytes(*args, ctypes.byref(n)) == want
        assert n.value == (exact if want == fa.FA_OK else 5)
        n.value = 5


# -------------------------------------------- planted mistakes in the oracle

def _pin_of_places(d):
    """Where include/fa.h puts channels, taken apart from the other end: the
    channel and token of each nibble of a block, read in the order of bytes."""
    ng = d // 32
    for byte in range(16 * d):
        section, at = divmod(byte, 8 * d)
        row, col = divmod(at, d // 2)
        if section == 0:
            p = row
            col ^= 64 * (p & 1) if d == 256 else 0
            word, byte_in = divmod(col, 4)
            high, rest = divmod(word, 16)
            t, low = divmod(rest, min(ng, 4))
            c = 32 * (4 * high + low) + 8 * t + 2 * byte_in
        else:
            col ^= {128: 32 * ((row >> 1) & 1), 256: 32 * (row & 3)}.get(d, 0)
            p = 2 * (row & 3) + ((row >> 2) & 1) + 8 * (row >> 3)
            unit, byte_in = divmod(col, 2)
            u, g = divmod(unit, ng)
            c = 32 * g + 4 * u + 2 * byte_in
        place = kv4.key_place if section == 0 else kv4.value_place
        assert place(d, p, c) == (byte, 0) and place(d, p, c + 1) == (byte, 4)
    at = 16 * d
    for p, w, g in itertools.product(range(16), range(2), range(ng)):
        assert kv4.scale_place(d, p, w, g) == at
        at += 2


@pytest.mark.parametrize("d", DIMS)
def test_places_are_the_headers(d):
    _pin_of_places(d)


def _pins():
    for d in DIMS:
        _pin_of_places(d)
        test_a_block_has_a_place_for_everything(d)
    test_levels_round_to_nearest_with_ties_to_even()
    test_scale_is_the_rounded_sixth_of_the_largest()
    test_a_group_with_a_non_finite_value_reads_as_nan()
    test_error_of_a_held_value()
    test_bf16_rounding_of_the_oracle()
    for d in DIMS:
        test_write_then_read(d)


def test_pins_hold_without_a_mistake():
    _pins()


_KEY, _VALUE, _SCALE, _QUANTISE, _ROUND = (kv4.key_place, kv4.value_place, kv4.scale_place, kv4.quantise, kv4.to_bf16)


def _coarse(x):
    code, bits = _QUANTISE(x)
    return code & 14, bits


def _no_nan(x):
    code, bits = _QUANTISE(x)
    return code, np.where(bits == kv4.NAN_BITS, 0, bits).astype(np.uint16)


MISTAKES = {
    "the largest level is 5": ("LEVELS", np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 5.0])),
    "two levels exchanged": ("LEVELS", np.array([0.0, 0.5, 1.5, 1.0, 2.0, 3.0, 4.0, 6.0])),
    "tokens 2 and 4 of the values exchanged": ("value_place", lambda d, p, c: _VALUE(d, {2: 4, 4: 2}.get(p, p), c)),
    "nibbles exchanged": ("key_place", lambda d, p, c: _KEY(d, p, c ^ 1)),
    "no exchange of halves at d = 256": ("key_place", lambda d, p, c: _KEY(d, p, c) if d != 256 else (
        p * 128 + _KEY(d, 0, c)[0], _KEY(d, 0, c)[1])),
    "scales of keys and values exchanged": ("scale_place", lambda d, p, w, g: _SCALE(d, p, 1 - w, g)),
    "scales of two groups exchanged": ("scale_place", lambda d, p, w, g: _SCALE(d, p, w, g ^ 1 if g < 2 else g)),
    "three bits of code": ("quantise", _coarse),
    "non-finite groups held as zeros": ("quantise", _no_nan),
    "scales cut and not rounded": ("to_bf16", lambda x: _ROUND(np.asarray(x, dtype=np.float64) * (1 - 2.0 ** -9))),
}


@pytest.mark.parametrize("mistake", MISTAKES)
def test_pins_catch_a_planted_mistake(mistake, monkeypatch):
    name, wrong = MISTAKES[mistake]
    monkeypatch.setattr(kv4, name, wrong)
    with pytest.raises(AssertionError):
        _pins()
