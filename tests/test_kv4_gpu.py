"""The 4-bit key/value cache on a GB300: writing, reading back and attention
over it, against the float64 oracle of the format.

Tolerances, derived from the arithmetic:
  write   : the codes and scales are a function of the bf16 inputs; the bytes
            must be the oracle's (but for the sign of a zero code).
  read    : code * scale rounded once to bf16: equal to the rounded oracle.
  attend  : with A = scale * sum_c |q_c k_c| the magnitude a score is summed
            from, a score in fp32 is off by at most e = 2^-19 max A (32
            products a group through the tensor cores, whose partial sums may
            be truncated, then at most 8 groups), and a weight P by a factor
            of at most 1 + 2 e + 2^-20 (the exponential, the sum).  The
            weights enter the P V product in 16 bits with at least 11
            significant ones (2^-11), its sums are fp32 (2^-13 covers 2^10
            steps), O is rounded once to bf16 (2^-8):
              |dO| <= 2^-8 |O| + (2^-11 + 2^-13 + 2^-20 + 2 e) sum_j P_j |v_j|
                      + n 2^-29 max_j P_j max_c |v_jc|
              |dL| <= e + 2^-20 max(1, |L|).
            The last term of |dO|: the 16 bits are fp16's, whose step is
            2^-24 below 2^-14, so a weight times its value's scale s is off by
            at most 2^-25 there, times a code of at most 6.  The reference is
            such that the largest P s of the row stands at 2^4 at least, and
            6 s_j is the largest |v_jc| of the group: n keys give at most
            n 6 2^-25 / 2^4 max_j P_j s_j = n 2^-29 max_j P_j max_c |v_jc|.
"""

import numpy as np
import pytest

from oracle import attention as att
from oracle import kv4

from exact_attention_92_gb300 import inputs

from gpu_util import dev, ensure_built, host, torch_cuda

pytestmark = pytest.mark.gpu

DIMS = (64, 96, 128, 256)


@pytest.fixture(scope="module")
def fa():
    torch_cuda()
    return ensure_built()


@pytest.fixture(params=["native", "ctypes"])
def caller(fa, request, monkeypatch):
    """The binding with its native caller, and with the one that does without."""
    from exact_attention_92_gb300 import _binding

    made = _binding._kv4_caller()
    assert made.__name__.endswith("_kv4_call")
    if request.param == "ctypes":
        monkeypatch.setattr(_binding, "_kv4", _binding._Kv4Ctypes(fa.load()))
    return request.param


def ints(x):
    return torch_cuda().tensor(x, dtype=torch_cuda().int32, device="cuda")


def normal(rng, shape, std=1.0):
    """bf16 normals: (device tensor, float64 values)."""
    bits = inputs.normal_bits(rng, shape, std)
    return dev(bits), inputs.bits_to_f64(bits)


def given(x):
    """A float64 array of bf16 values on the device."""
    return dev(kv4.bf16_bits(x))


def make_table(rng, B, pages_each, spare=3):
    """Scattered pages; entries that no position uses come last."""
    n = B * pages_each + spare
    return rng.permutation(n)[:B * pages_each].reshape(B, pages_each).astype(np.int32), n


# ------------------------------------------------------------ write and read

MOVES = [
    # B, Hkv, N, page, start, count
    (1, 1, 1, 16, [0], None),
    (2, 3, 1, 16, [15, 16], None),
    (3, 2, 40, 16, [0, 5, 31], [40, 0, 17]),
    (2, 1, 37, 32, [30, 1], [37, 36]),
    (1, 4, 70, 64, [63], None),
    (2, 2, 33, 256, [200, 255], [33, 1]),
    (5, 1, 3, 128, [0, 1, 2, 126, 127], [3, 2, 1, 3, 0]),
    # Enough tokens that a CTA takes four blocks.
    (16, 8, 200, 32, list(range(0, 80, 5)), [200, 0, 1, 15, 16, 17, 63, 64, 65, 128, 150, 191, 192, 193, 199, 200]),
    (8, 13, 223, 64, [0, 1, 15, 16, 17, 48, 63, 64], None),
]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("B,Hkv,N,page,start,count", MOVES)
def test_write_and_read(fa, d, B, Hkv, N, page, start, count):
    """The cache's bytes are the oracle's, those of other tokens stay as they
    were, and reading back gives the held values rounded once."""
    torch = torch_cuda()
    rng = np.random.default_rng(1000 * d + N + page)
    kd, k = normal(rng, (B, Hkv, N, d))
    vd, v = normal(rng, (B, Hkv, N, d), 0.01)
    table, n = make_table(rng, B, -(-(max(start) + N) // page))
    before = rng.integers(0, 256, (n, Hkv, page * 9 * d // 8), dtype=np.uint8)
    want = before.copy()
    kv4.write(want, table, start, count, k, v, page)
    cache = torch.from_numpy(before).cuda()
    cnt = None if count is None else ints(count)
    fa.fa_kv4_write(kd, vd, cache, ints(table), ints(start), cnt)
    assert fa.fa_poll_status() == fa.FA_OK
    got = cache.cpu().numpy()
    # Bytes of tokens that were not written: bit for bit.
    touched = np.zeros_like(before)
    ones = np.ones_like(k)
    other = np.full_like(before, 0xFF)
    kv4.write(touched, table, start, count, ones, ones, page)
    kv4.write(other, table, start, count, ones, ones, page)
    free = touched != other
    assert np.array_equal(got[free], before[free])
    assert np.array_equal(kv4.canonical(got, d), kv4.canonical(want, d))
    ko, vo = (torch.full_like(kd, 7.0) for _ in range(2))
    fa.fa_kv4_read(cache, ints(table), ints(start), ko, vo, cnt)
    assert fa.fa_poll_status() == fa.FA_OK
    for out, x in ((host(ko), k), (host(vo), v)):
        for b in range(B):
            m = N if count is None else count[b]
            assert np.array_equal(out[b, :, :m], kv4.to_bf16(kv4.held(x[b, :, :m])))
            assert (out[b, :, m:] == 7.0).all()


def _hard_values(d):
    """Rows whose groups hold borders between levels, under even and odd
    scales, zeros, the smallest and largest values, infinities and NaN."""
    rows = []
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rng = np.random.default_rng(5)
    for step in range(128, 256, 3):  # scales of every significand, tops of 6 s
        s = step / 128 * 2.0 ** int(rng.integers(-60, 60))
        top = kv4.to_bf16(np.array(6 * s))
        held_s = float(kv4.to_bf16(np.array(top / 6)))
        near = kv4.to_bf16(borders * held_s)
        ulp = np.abs(near) * 2.0 ** -7
        vals = np.concatenate([[top], near, -near, kv4.to_bf16(near + ulp), kv4.to_bf16(near - ulp)])
        rows.append(np.concatenate([vals, np.zeros(32)])[:32])
    rows.append(np.zeros(32))
    rows.append(np.full(32, 2.0 ** -133))
    rows.append(np.r_[2.0 ** -126 * 6, np.full(31, 2.0 ** -126)])   # the smallest scale that is held
    rows.append(np.r_[2.0 ** -126 * 5, np.full(31, 2.0 ** -126)])   # a scale below it
    rows.append(np.r_[3.3895313892515355e38, np.full(31, -3.3895313892515355e38)])
    rows.append(np.r_[np.inf, np.ones(31)])
    rows.append(np.r_[np.ones(31), -np.inf])
    rows.append(np.r_[1.0, np.nan, np.ones(30)])
    g = np.stack(rows)
    per = d // 32
    g = np.concatenate([g, np.ones(((-len(g)) % per, 32))])
    return g.reshape(-1, d)


@pytest.mark.parametrize("d", DIMS)
def test_values_at_the_borders(fa, d):
    torch = torch_cuda()
    x = _hard_values(d)
    N = len(x)
    k, v = x[None, None], x[None, None, ::-1].copy()
    page = 64
    table = np.arange(-(-N // page), dtype=np.int32)[None]
    cache = fa.kv4_cache(table.shape[1], 1, page, d)
    want = np.zeros(tuple(cache.shape), np.uint8)
    with np.errstate(invalid="ignore"):
        kv4.write(want, table, [0], None, k, v, page)
    kd, vd = given(k), given(v)
    fa.fa_kv4_write(kd, vd, cache, ints(table), ints([0]))
    got = kv4.canonical(cache.cpu().numpy(), d)
    assert np.array_equal(got, kv4.canonical(want, d)), np.argwhere(got != kv4.canonical(want, d))[:5]
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    fa.fa_kv4_read(cache, ints(table), ints([0]), ko, vo)
    assert fa.fa_poll_status() == fa.FA_OK
    assert np.array_equal(host(ko), kv4.to_bf16(kv4.held(k)), equal_nan=True)
    assert np.array_equal(host(vo), kv4.to_bf16(kv4.held(v)), equal_nan=True)


# ----------------------------------------------------------------- attention

class Filled:
    """A cache of given lengths, its bytes behind the tokens all ones (NaN
    scales), and the held values in float64."""

    def __init__(self, fa, rng, lens, Hkv, d, page, k_std=1.0, v_std=1.0, room=0, keys=None, vals=None):
        torch = torch_cuda()
        self.lens, self.page, B, N = lens, page, len(lens), max(1, max(lens))
        need = -(-(N + room) // page)
        self.table, n = make_table(rng, B, need + 1)
        for b in range(B):
            self.table[b, -(-(lens[b] + room) // page):] = -1  # not in use: may be anything
        kd, k = normal(rng, (B, Hkv, N, d), k_std)
        vd, v = normal(rng, (B, Hkv, N, d), v_std)
        if keys is not None:
            kd, k = given(keys), keys
        if vals is not None:
            vd, v = given(vals), vals
        self.cache = torch.full((n, Hkv, page * 9 * d // 8), 0xFF, dtype=torch.uint8, device="cuda")
        self.td, self.ld = ints(self.table), ints(lens)
        fa.fa_kv4_write(kd, vd, self.cache, self.td, ints([0] * B), self.ld)
        self.k, self.v = kv4.held(k), kv4.held(v)


def check_attend(o, lse, q, k, v, lens, scale, causal, what=""):
    """o, lse against the oracle on q [B, H, Nq, d] and held k, v."""
    o, lse = host(o), lse.double().cpu().numpy()
    B, H, Nq, d = q.shape
    group = H // k.shape[1]
    for b, n in enumerate(lens):
        O, L = kv4.attend(q[b], k[b], v[b], n, scale, causal)
        for h in range(H):
            empty = np.isneginf(L[h])
            assert np.array_equal(np.isneginf(lse[b, h]), empty), f"{what} b={b} h={h}: L {lse[b, h]} for {L[h]}"
            assert (o[b, h][empty] == 0).all(), f"{what} b={b} h={h}: O of an empty row"
            if n == 0:
                continue
            kk, vv = k[b, h // group, :n], v[b, h // group, :n]
            off = 0 if causal == "none" else att.causal_offset(Nq, n, causal)
            P = att.probabilities_head(q[b, h], kk, scale, causal != "none", offset=off)
            A = scale * np.abs(q[b, h]) @ np.abs(kk).T
            e = 2.0 ** -19 * A.max(1)
            bound = 2.0 ** -8 * np.abs(O[h]) + (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -20 + 2 * e)[:, None] * (P @ np.abs(vv))
            bound += n * 2.0 ** -29 * (P * np.abs(vv).max(1)).max(1)[:, None]
            err = np.abs(o[b, h] - O[h])
            assert (err <= bound + 1e-38).all(), (
                f"{what} b={b} h={h}: O off by {np.nanmax(err / (bound + 1e-38)):.3g} of the bound, {err.max():.3g}")
            lb = e + 2.0 ** -20 * np.maximum(1, np.abs(np.where(empty, 0, L[h])))
            dl = np.abs(np.where(empty, 0, lse[b, h]) - np.where(empty, 0, L[h]))
            assert (dl <= lb).all(), f"{what} b={b} h={h}: L off by {dl.max():.3g}, bound {lb.min():.3g}"


ATTENDS = [
    # H, Hkv, Nq, page, lens, causal
    (1, 1, 1, 16, [1], "none"),
    (8, 8, 1, 16, [16, 17, 0, 1], "none"),
    (4, 1, 1, 32, [31, 32, 33], "bottom_right"),
    (8, 1, 1, 64, [500], "bottom_right"),
    (6, 2, 1, 64, [129, 0, 64, 7, 300], "none"),
    (7, 1, 1, 256, [257, 255], "bottom_right"),
    (16, 2, 2, 16, [100, 1, 2], "bottom_right"),
    (3, 1, 5, 32, [3, 0, 4, 5, 200], "bottom_right"),
    (4, 2, 9, 128, [9, 130, 8], "top_left"),
    (2, 2, 40, 16, [70, 39, 40, 41], "bottom_right"),
    (8, 1, 16, 64, [333, 5], "bottom_right"),
    (16, 1, 8, 32, [65], "none"),
    (5, 1, 3, 1024, [1030, 2], "top_left"),
]


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("H,Hkv,Nq,page,lens,causal", ATTENDS)
def test_attend(fa, d, H, Hkv, Nq, page, lens, causal):
    rng = np.random.default_rng(d + 7 * H + Nq)
    f = Filled(fa, rng, lens, Hkv, d, page)
    qd, q = normal(rng, (len(lens), H, Nq, d))
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld, causal=causal)
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, causal, f"d={d}")


@pytest.mark.parametrize("d,H,Hkv,Nq,page,lens", [
    (128, 8, 2, 1, 64, [9000, 12, 4097]),
    (64, 2, 2, 1, 16, [5001]),
    (96, 3, 1, 5, 32, [6001, 0, 33]),
    (256, 4, 1, 1, 128, [2500, 2500]),
    (128, 16, 1, 1, 16, [20000]),
])
def test_attend_long(fa, d, H, Hkv, Nq, page, lens):
    rng = np.random.default_rng(d + sum(lens))
    f = Filled(fa, rng, lens, Hkv, d, page)
    qd, q = normal(rng, (len(lens), H, Nq, d))
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld, causal="bottom_right")
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, "bottom_right")


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("q_std,k_std,v_std", [(20.0, 2.0, 1.0), (1.0, 1.0, 1e-20), (1.0, 1.0, 1e25), (1e-10, 1e9, 1.0),
                                               (1e20, 1e-20, 1.0), (1e-30, 1.0, 1e-3)])
def test_attend_magnitudes(fa, d, q_std, k_std, v_std):
    """Sharp softmaxes, and inputs far from 1 that cancel or do not matter."""
    rng = np.random.default_rng(d)
    lens = [300, 41]
    f = Filled(fa, rng, lens, 2, d, 32, k_std, v_std)
    qd, q = normal(rng, (2, 4, 1, d), q_std)
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, "none", f"{q_std} {k_std} {v_std}")


@pytest.mark.parametrize("d", DIMS)
def test_attend_uneven_values(fa, d):
    """Keys whose scores rise along the sequence (every stretch raises the
    running maximum), values whose size changes by 2^40 along it, a stretch of
    zero values, zero query rows, and one channel far above the others."""
    rng = np.random.default_rng(11)
    N = 700
    base = np.abs(kv4.to_bf16(rng.standard_normal((1, 1, N, d))))
    keys = kv4.to_bf16(base * (np.arange(N)[None, None, :, None] / 40 + 0.1))
    keys[..., 3] = kv4.to_bf16(keys[..., 3] * 100)
    vals = kv4.to_bf16(rng.standard_normal((1, 1, N, d)) * 2.0 ** (20 - 40 * np.arange(N)[None, None, :, None] / N))
    vals[:, :, 300:400] = 0
    for flip in (False, True):
        kk, vv = (np.ascontiguousarray(x[:, :, ::-1]) if flip else x for x in (keys, vals))
        f = Filled(fa, rng, [N], 1, d, 16, keys=kk, vals=vv)
        q = np.abs(kv4.to_bf16(rng.standard_normal((1, 3, 1, d))))
        q[0, 1] = 0
        q[0, 2] = -q[0, 2]
        wide = np.full((1, 4000), -1, np.int32)  # room for so many steps that CTAs share a sequence
        wide[:, :f.table.shape[1]] = f.table
        for table in (f.td, ints(wide)):
            o, lse = fa.kv4_forward(given(q), f.cache, table, f.ld, scale=0.01)
            assert fa.fa_poll_status() == fa.FA_OK
            check_attend(o, lse, q, f.k, f.v, [N], 0.01, "none", f"flip={flip} {tuple(table.shape)}")


def two_parts(N, d, big, small):
    """Keys of one head whose channel 0 holds `big` [N] and whose channel 32
    holds `small` [N], other channels 0."""
    keys = np.zeros((1, 1, N, d))
    keys[..., 0], keys[..., 32] = kv4.to_bf16(big), kv4.to_bf16(small)
    return keys


@pytest.mark.parametrize("sign", (1, -1))
@pytest.mark.parametrize("power", (24, 25, 26, 27, 28, 31, 60))
@pytest.mark.parametrize("d,H,v_std", [(64, 4, 1.0), (64, 20, 1.0), (96, 6, 1e-3), (96, 20, 1.0), (128, 4, 1e3),
                                       (128, 16, 1.0), (256, 8, 1.0)])
def test_attend_scores_beyond_fp32_units(fa, d, H, v_std, power, sign):
    """Scores of 2^power, where fp32's step is 1 or more, that rise every 32
    keys by one such step or two: O stays finite and, its weights being at least
    0, within the values' range.  (O = sum_j w_j v_j / sum_j w_j; the 16-bit
    weights are off by 2^-11 of themselves, the sums and exponentials by less
    than another, O by 2^-8.)  Many sequences over the same pages, so that a
    warp has several steps of each."""
    rng = np.random.default_rng(power + d)
    N, B = 2000, 100
    step = 2.0 ** (power - 23)
    keys = two_parts(N, d, np.full(N, sign * 2.0 ** (power - 8) * 6), np.arange(N) // 32 * step / 32)
    f = Filled(fa, rng, [N], 1, d, 16, keys=keys, v_std=v_std)
    q = np.zeros((1, H, 1, d))
    q[..., 0] = 2.0 ** 8 / 6
    q[0, :, 0, 32] = 32 * (1 + np.arange(H) / H)  # base-2 scores of 2^power, and j / 32 steps and more
    q = kv4.to_bf16(q)
    scale = float(np.log(2.0))
    wide = np.full((1, 600), -1, np.int32)  # room for more steps: the unit's rows by the steps of an SM
    wide[:, :f.table.shape[1]] = f.table
    top = np.abs(f.v[0, 0]).max(0)
    for table in (f.table, wide):
        o, lse = fa.kv4_forward(given(np.repeat(q, B, 0)), f.cache, ints(np.repeat(table, B, 0)), ints([N] * B), scale=scale)
        assert fa.fa_poll_status() == fa.FA_OK
        O = host(o)[:, :, 0]
        assert np.isfinite(O).all() and np.isfinite(lse.cpu().numpy()).all()
        assert (np.abs(O) <= top * (1 + 2.0 ** -8 + 2.0 ** -10)).all()
        for b in (0, B - 1):
            check_attend(o[b:b + 1], lse[b:b + 1], q, f.k, f.v, [N], scale, "none", f"2^{power}")


@pytest.mark.parametrize("sign", (1, -1))
@pytest.mark.parametrize("power", (24, 26, 28, 32, 64, 110))
@pytest.mark.parametrize("d,H,v_std", [(64, 9, 1.0), (96, 3, 1.0), (128, 1, 1e10), (256, 5, 1e-10)])
def test_attend_one_key_far_above_the_others(fa, d, H, v_std, power, sign):
    """Scores of 2^power, each key's 2^-7 of that or more from the next: a
    score is off by e = 2^-19 of its size at most, so the largest one's key
    has all the weight (2^(2 e - 2^(power - 7)) of it, nothing, goes to
    others).  The weight is off by 2^-11 in the product and not in the sum,
    with less than 2^-12 from the exponentials; O is rounded once."""
    rng = np.random.default_rng(power + d)
    N = 60
    order = rng.permutation(N)
    keys = two_parts(N, d, sign * 2.0 ** (power // 2) * (1 + order / 32), np.zeros(N))
    f = Filled(fa, rng, [N], 1, d, 16, keys=keys, v_std=v_std)
    q = np.zeros((1, H, 1, d))
    q[..., 0] = 2.0 ** (power - power // 2)
    best = int(np.argmax(f.k[0, 0, :, 0]))
    gap = np.sort(f.k[0, 0, :, 0])[-1] - np.sort(f.k[0, 0, :, 0])[-2]
    assert gap >= 2.0 ** (power // 2 - 7)
    o, lse = fa.kv4_forward(given(q), f.cache, f.td, f.ld, scale=1.0)
    assert fa.fa_poll_status() == fa.FA_OK
    want = f.v[0, 0, best]
    assert (np.abs(host(o)[0, :, 0] - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12) * np.abs(want)).all()
    L = q[0, 0, 0, 0] * f.k[0, 0, best, 0]
    assert (np.abs(lse.cpu().numpy()[0] - L) <= 2.0 ** -19 * abs(L)).all()


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("q_std,k_std", [(1e-30, 1e31), (1e-33, 1e33), (1e-35, 3e35), (3e-37, 5e36)])
def test_attend_small_queries_over_large_keys(fa, d, q_std, k_std):
    """Query rows so small, and keys so large, that neither can be brought to
    the other's size in fp32: the scores are ordinary ones."""
    rng = np.random.default_rng(d)
    lens = [300, 41]
    f = Filled(fa, rng, lens, 2, d, 32, k_std)
    for H in (4, 12):
        qd, q = normal(rng, (2, H, 1, d), q_std)
        o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
        assert fa.fa_poll_status() == fa.FA_OK
        check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, "none", f"{q_std} {k_std}")


@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("q_std,k_std,scale", [(1e19, 1e19, 1e-39), (1e10, 1e30, 1e-41), (1e-19, 1e-19, 1e37),
                                               (1e-30, 1e-8, 3e37), (1e-3, 1e-36, 3e38), (1e-30, 1e31, 0.05)])
def test_attend_scales_far_from_one(fa, d, q_std, k_std, scale):
    """Scores that only the softmax's scale brings to an ordinary size: q k
    overflows, or is subnormal, in fp32."""
    rng = np.random.default_rng(d)
    scale = float(np.float32(scale))
    lens = [300, 41]
    f = Filled(fa, rng, lens, 2, d, 32, k_std)
    for H in (4, 12):
        qd, q = normal(rng, (2, H, 1, d), q_std)
        o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld, scale=scale)
        assert fa.fa_poll_status() == fa.FA_OK
        check_attend(o, lse, q, f.k, f.v, lens, scale, "none", f"{q_std} {k_std} {scale}")


def test_attend_all_values_zero(fa):
    rng = np.random.default_rng(3)
    f = Filled(fa, rng, [77], 1, 128, 16, vals=np.zeros((1, 1, 77, 128)))
    qd, q = normal(rng, (1, 4, 1, 128))
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
    check_attend(o, lse, q, f.k, f.v, [77], 128 ** -0.5, "none")


@pytest.mark.parametrize("d", DIMS)
def test_held_nan_reaches_the_rows_that_see_it(fa, d):
    """A token written with an infinity reads as NaN: rows that see it give
    NaN, rows that do not are untouched by it."""
    rng = np.random.default_rng(2)
    N = 50
    vals = kv4.to_bf16(rng.standard_normal((1, 1, N, d)))
    vals[0, 0, N - 1, 0] = np.inf
    f = Filled(fa, rng, [N], 1, d, 16, vals=vals)
    qd, q = normal(rng, (1, 1, 2, d))
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld, causal="bottom_right")
    O = host(o)[0, 0]
    assert np.isfinite(O[0]).all() and np.isnan(O[1, :32]).all() and np.isfinite(O[1, 32:]).all()
    clean = f.v.copy()
    clean[0, 0, N - 1] = 0
    want, _ = kv4.attend(q[0, :, :1], f.k[0], clean[0], N - 1, d ** -0.5, "none")
    assert np.abs(O[0] - want[0, 0]).max() < 0.02


def test_held_nan_of_a_key_reaches_all_channels(fa):
    rng = np.random.default_rng(3)
    N, d = 300, 128
    keys = kv4.to_bf16(rng.standard_normal((1, 1, N, d)))
    keys[0, 0, N - 1, 5] = np.nan
    f = Filled(fa, rng, [N], 1, d, 16, keys=keys)
    for H in (2, 6, 12):
        qd, q = normal(rng, (1, H, 2, d))
        o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld, causal="bottom_right")
        O, L = host(o)[0], lse.cpu().numpy()[0]
        assert np.isfinite(O[:, 0]).all() and np.isfinite(L[:, 0]).all()
        assert np.isnan(O[:, 1]).all() and np.isnan(L[:, 1]).all()
    assert fa.fa_poll_status() == fa.FA_OK


def test_pages_far_apart(fa):
    """A cache beyond 2^32 bytes, its pages in use at both ends."""
    torch = torch_cuda()
    d, page, Hkv = 128, 256, 8
    n = (5 << 30) // (Hkv * page * 144)
    cache = torch.empty((n, Hkv, page * 144), dtype=torch.uint8, device="cuda")
    assert cache.numel() > 2 ** 32
    table = np.array([[n - 1, 0, n // 2], [n - 2, 1, n // 2 + 1]], np.int32)
    rng = np.random.default_rng(1)
    kd, k = normal(rng, (2, Hkv, 600, d))
    vd, v = normal(rng, (2, Hkv, 600, d))
    fa.fa_kv4_write(kd, vd, cache, ints(table), ints([0, 0]))
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    fa.fa_kv4_read(cache, ints(table), ints([0, 0]), ko, vo)
    assert np.array_equal(host(ko), kv4.to_bf16(kv4.held(k))) and np.array_equal(host(vo), kv4.to_bf16(kv4.held(v)))
    qd, q = normal(rng, (2, 8, 1, d))
    o, lse = fa.kv4_forward(qd, cache, ints(table), ints([600, 512]))
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, kv4.held(k), kv4.held(v), [600, 512], d ** -0.5, "none")


@pytest.mark.parametrize("d,rows,pages", [(64, 1, 2 ** 20), (128, 9, 2 ** 16)])
def test_very_long_sequences(fa, d, rows, pages):
    """2^30 positions, the most there may be, and 2^26: a table whose entries
    are all one of four pages.  O is that of the pages each seen once, L is
    larger by the logarithm of how often.  A warp adds up s steps one after the
    other, in each two products to O (fp32, perhaps cut: 2^-23 of the sum each)
    and at most four weights to their sum (rounded: 2^-24 each); where all go
    the same way O is off by s 2^-21 of the largest value, L by s 2^-22."""
    torch = torch_cuda()
    rng = np.random.default_rng(d)
    page, each = 1024, pages // 4
    f = Filled(fa, rng, [4 * page], 1, d, page)
    qd, q = normal(rng, (1, rows, 1, d))
    o, lse = fa.kv4_forward(qd, f.cache, ints(np.tile(f.table[0, :4], each)[None]), ints([pages * page]))
    assert fa.fa_poll_status() == fa.FA_OK
    k, v = torch.from_numpy(f.k).cuda(), torch.from_numpy(f.v).cuda()
    O, L, bo, bl = attend64(qd.double().view(1, 1, rows, d), k, v, ints([4 * page]), d ** -0.5)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    steps = pages * page / 32 * -(-rows // 8) / (sms * 8)  # 8 warps a CTA at least
    bo = bo + steps * 2.0 ** -21 * v.abs().amax()
    assert ((o.double().view(O.shape) - O).abs() <= bo).all(), ((o.double().view(O.shape) - O).abs() / bo).max()
    dl = (lse.double().view(L.shape) - (L + np.log(each))).abs()
    assert (dl <= bl + steps * 2.0 ** -22 + 2.0 ** -20 * np.log(each)).all(), (dl / bl).max()


def test_many_sequences(fa):
    """More sequences than a CTA has threads, most of them short or empty."""
    rng = np.random.default_rng(8)
    B, d = 1500, 64
    lens = [int(x) for x in rng.integers(0, 40, B)]
    f = Filled(fa, rng, lens, 1, d, 16)
    qd, q = normal(rng, (B, 2, 1, d))
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, "none")


def test_results_do_not_change_from_run_to_run(fa):
    torch = torch_cuda()
    rng = np.random.default_rng(4)
    f = Filled(fa, rng, [3000, 100, 777], 2, 128, 64)
    qd, _ = normal(rng, (3, 8, 2, 128))
    a = fa.kv4_forward(qd, f.cache, f.td, f.ld, causal="bottom_right")
    for _ in range(3):
        b = fa.kv4_forward(qd, f.cache, f.td, f.ld, causal="bottom_right")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------- bad indices

@pytest.mark.parametrize("d", (64, 128))
def test_bad_pages_are_skipped_and_reported(fa, d):
    torch = torch_cuda()
    rng = np.random.default_rng(6)
    page, lens = 16, [100, 64]
    f = Filled(fa, rng, lens, 1, d, page)
    num_pages = f.cache.shape[0]
    assert fa.fa_poll_status() == fa.FA_OK
    bad = f.table.copy()
    bad[0, 2], bad[1, 1], bad[1, 3] = num_pages, -5, 2 ** 31 - 1
    keep = [np.r_[0:32, 48:100], np.r_[0:16, 32:48]]  # positions whose page is in range
    qd, q = normal(rng, (2, 2, 1, d))
    o, lse = fa.kv4_forward(qd, f.cache, ints(bad), f.ld)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    assert fa.fa_poll_status() == fa.FA_OK
    for b in range(2):
        check_attend(o[b:b + 1], lse[b:b + 1], q[b:b + 1], f.k[b:b + 1][:, :, keep[b]], f.v[b:b + 1][:, :, keep[b]],
                     [len(keep[b])], d ** -0.5, "none")
    # Reading: rows of a bad page stay as they were; writing: nothing moves.
    ko, vo = (torch.full((2, 1, 64, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_kv4_read(f.cache, ints(bad), ints([0, 0]), ko, vo)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    assert (host(ko)[0, :, 32:48] == 7).all() and (host(vo)[1, :, 48:64] == 7).all()
    assert np.array_equal(host(ko)[0, 0, :32], kv4.to_bf16(f.k[0, 0, :32]))
    before = f.cache.clone()
    fa.fa_kv4_write(ko[:, :, :16].contiguous(), vo[:, :, :16].contiguous(), f.cache, ints(bad), ints([32, 16]))
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    assert torch.equal(before, f.cache)


def test_bad_pages_among_many_tokens(fa):
    """Where a CTA takes four blocks of tokens, those of a bad page are left
    out and the others are not."""
    torch = torch_cuda()
    rng = np.random.default_rng(24)
    B, Hkv, N, d, page = 8, 10, 256, 64, 16
    kd, k = normal(rng, (B, Hkv, N, d))
    vd, v = normal(rng, (B, Hkv, N, d))
    table, n = make_table(rng, B, N // page)
    bad = table.copy()
    bad[rng.random(bad.shape) < 0.2] = n
    assert (bad == n).any()
    cache = fa.kv4_cache(n, Hkv, page, d)
    fa.fa_kv4_write(kd, vd, cache, ints(bad), ints([0] * B))
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    there = np.repeat(bad != n, page, 1)[:, None, :, None]
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    fa.fa_kv4_read(cache, ints(table), ints([0] * B), ko, vo)  # pages that were not written hold zeros
    assert fa.fa_poll_status() == fa.FA_OK
    for out, x in ((ko, k), (vo, v)):
        assert np.array_equal(host(out), np.where(there, kv4.to_bf16(kv4.held(x)), 0))
    fa.fa_kv4_write(kd, vd, cache, ints(table), ints([0] * B))
    ko.fill_(7.0), vo.fill_(7.0)
    fa.fa_kv4_read(cache, ints(bad), ints([0] * B), ko, vo)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    for out, x in ((ko, k), (vo, v)):
        assert np.array_equal(host(out), np.where(there, kv4.to_bf16(kv4.held(x)), 7))


def test_bad_lengths_and_positions_are_clamped_and_reported(fa):
    torch = torch_cuda()
    rng = np.random.default_rng(7)
    d, page = 64, 16
    f = Filled(fa, rng, [32, 32], 1, d, page)
    table = ints(f.table[:, :2].copy())
    qd, q = normal(rng, (2, 1, 1, d))
    o, lse = fa.kv4_forward(qd, f.cache, table, ints([-3, 1000]))
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    check_attend(o, lse, q, f.k, f.v, [0, 32], d ** -0.5, "none")
    before = f.cache.clone()
    x = torch.ones((2, 1, 4, d), dtype=torch.bfloat16, device="cuda")
    for start, count in (([-4, 32], None), ([2 ** 31 - 1, -2 ** 31], None), ([0, 0], [-1, 0]), ([32, 40], [5, 0])):
        fa.fa_kv4_write(x, x, f.cache, table, ints(start), None if count is None else ints(count))
        assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
        assert torch.equal(before, f.cache)
    out = torch.full_like(x, 7.0)
    fa.fa_kv4_read(f.cache, table, ints([30, -2]), out, out.clone())
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    got = host(out)
    assert (got[0, :, 2:] == 7).all() and (got[1, :, :2] == 7).all()
    assert np.array_equal(got[0, 0, :2], kv4.to_bf16(f.k[0, 0, 30:32]))
    # Another call is not disturbed by an unread report.
    fa.kv4_forward(qd, f.cache, table, ints([-3, 1000]))
    o, lse = fa.kv4_forward(qd, f.cache, table, f.ld)
    a, b, c, _ = (torch.randn((1, 2, 300, 64), device="cuda").to(torch.bfloat16) for _ in range(4))
    first = fa.forward(a, b, c, causal=True)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    second = fa.forward(a, b, c, causal=True)
    assert torch.equal(first[0], second[0])
    check_attend(o, lse, q, f.k, f.v, [32, 32], d ** -0.5, "none")


def test_a_timeout_does_not_hide_a_bad_index(fa):
    rng = np.random.default_rng(13)
    f = Filled(fa, rng, [32], 1, 64, 16)
    qd, _ = normal(rng, (1, 1, 1, 64))
    for bad_first in (True, False):
        assert fa.fa_poll_status() == fa.FA_OK
        if not bad_first:
            fa.fa_selftest_wait_timeout(10_000_000)
        fa.kv4_forward(qd, f.cache, f.td, ints([-1]))
        if bad_first:
            fa.fa_selftest_wait_timeout(10_000_000)
        assert [fa.fa_poll_status() for _ in range(3)] == [fa.FA_ERR_TIMEOUT, fa.FA_ERR_BAD_INDEX, fa.FA_OK]


def test_binding_refusals(fa, caller):
    torch = torch_cuda()
    rng = np.random.default_rng(9)
    f = Filled(fa, rng, [32], 2, 64, 16)
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    zero = ints([0])
    ok = (q, f.cache, f.td, f.ld)
    fa.kv4_forward(*ok)
    for i, bad in ((0, q.float()), (0, q.transpose(1, 2)), (1, f.cache.float()), (1, f.cache[:, :, :-1]),
                   (1, f.cache[:, :, ::2]), (2, f.td.long()), (2, f.td[0]), (2, f.td.repeat(2, 1)), (3, f.ld.float()),
                   (3, f.ld.repeat(2)), (3, f.ld.cpu())):
        args = list(ok)
        args[i] = bad
        with pytest.raises((ValueError, TypeError, fa.FaError)):
            fa.kv4_forward(*args)
    o, lse = torch.empty_like(q), torch.empty((1, 4, 1), device="cuda")
    for bad_o, bad_lse in ((o[:, :2], lse), (o.half(), lse), (o, lse.half()), (o, lse[:, :, 0]), (o.cpu(), lse),
                           (o, lse.cpu())):
        with pytest.raises(ValueError):
            fa.fa_kv4_fwd(q, f.cache, f.td, f.ld, bad_o, bad_lse)
    with pytest.raises(fa.FaError):
        fa.fa_kv4_fwd(q, f.cache, f.td, f.ld, o, lse, scale=-1.0)
    for causal in (3, -1, 2 ** 32, 2 ** 32 + 1):
        with pytest.raises(fa.FaError):
            fa.fa_kv4_fwd(q, f.cache, f.td, f.ld, o, lse, causal=causal)
    fa.fa_kv4_fwd(q, f.cache, f.td, f.ld, o, lse, causal=fa.FA_CAUSAL_BOTTOM_RIGHT, scale=1, stream=0)
    with pytest.raises(fa.FaError) as e:  # 24-token pages
        fa.kv4_forward(q, torch.zeros((4, 2, 24 * 72), dtype=torch.uint8, device="cuda"), f.td, f.ld)
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FaError) as e:
        fa.kv4_forward(torch.zeros((1, 4, 65, 64), dtype=torch.bfloat16, device="cuda"), f.cache, f.td, f.ld)
    assert e.value.status == fa.FA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        fa.fa_kv4_write(k[:, :1].contiguous(), k[:, :1].contiguous(), f.cache, f.td, zero)  # heads differ
    with pytest.raises(ValueError):
        fa.fa_kv4_write(k, k[:, :, :3].contiguous(), f.cache, f.td, zero)
    with pytest.raises(ValueError):
        fa.fa_kv4_read(f.cache, f.td, zero, k, k, ints([1, 2]))
    assert fa.fa_poll_status() == fa.FA_OK


def test_misaligned_storage_is_refused(fa, caller):
    torch = torch_cuda()
    raw = torch.zeros(4 * 2 * 16 * 72 + 16, dtype=torch.uint8, device="cuda")
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    qq = torch.zeros(1 + q.numel(), dtype=torch.bfloat16, device="cuda")[1:].view(q.shape)
    table, lens = ints([[0, 1]]), ints([20])
    cache = raw[:4 * 2 * 16 * 72].view(4, 2, -1)
    fa.kv4_forward(q, cache, table, lens)
    for a, c in ((qq, cache), (q, raw[8:8 + 4 * 2 * 16 * 72].view(4, 2, -1))):
        with pytest.raises(fa.FaError) as e:
            fa.kv4_forward(a, c, table, lens)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    # int32 arrays that start anywhere in another one are fine.
    many = ints([7, 0, 1, 20])
    o, lse = fa.kv4_forward(q, cache, many[1:3].view(1, 2), many[3:])
    assert fa.fa_poll_status() == fa.FA_OK and (host(o) == 0).all()


def test_workspace_allocation_failure_is_reported(fa, monkeypatch):
    rng = np.random.default_rng(10)
    f = Filled(fa, rng, [9000], 1, 64, 16)  # cut between CTAs, so that partial results need workspace
    qd, q = normal(rng, (1, 2, 1, 64))
    monkeypatch.setenv("FA_TEST_FAIL_ALLOC", "1")
    with pytest.raises(fa.FaError) as e:
        fa.kv4_forward(qd, f.cache, f.td, f.ld)
    assert e.value.status == fa.FA_ERR_NO_MEMORY
    monkeypatch.delenv("FA_TEST_FAIL_ALLOC")
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, [9000], 64 ** -0.5, "none")


@pytest.mark.parametrize("rows", (1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 24, 25, 33))
@pytest.mark.parametrize("d", DIMS)
def test_every_count_of_query_rows(fa, d, rows):
    """Rows per key/value head about the borders between the tilings, over a
    table that makes units cut between CTAs and one that does not."""
    rng = np.random.default_rng(100 * d + rows)
    lens = [47, 600, 5]
    f = Filled(fa, rng, lens, 2, d, 32)
    qd, q = normal(rng, (3, 2 * rows, 1, d))
    # 6 heads' units, room for 6144 steps each: two row tiles a unit above 8 rows.
    wide = np.full((3, 6144), -1, np.int32)
    wide[:, :f.table.shape[1]] = f.table
    short = Filled(fa, rng, [47, 33, 0], 2, d, 16)
    for g, table, n in ((f, ints(wide), lens), (f, f.td, lens), (short, short.td, [47, 33, 0])):
        o, lse = fa.kv4_forward(qd, g.cache, table, g.ld)
        assert fa.fa_poll_status() == fa.FA_OK
        check_attend(o, lse, q, g.k, g.v, n, d ** -0.5, "none", f"rows={rows}")


def attend64(q, k, v, lens, scale):
    """O, L and the bounds of check_attend, without a mask, for all sequences
    at once: float64 tensors q [B, Hkv, R, d], k, v [B, Hkv, N, d]."""
    torch = torch_cuda()
    n = lens[:, None, None, None].double()
    seen = torch.arange(k.shape[2], device="cuda")[None, None, None, :] < lens[:, None, None, None]
    S = (scale * q @ k.transpose(-1, -2)).masked_fill(~seen, -np.inf)
    L = torch.logsumexp(S, -1)
    P = torch.where(seen, torch.exp(S - L[..., None]), 0.0)
    e = 2.0 ** -19 * ((scale * q.abs() @ k.abs().transpose(-1, -2)) * seen).amax(-1)
    O = P @ v
    bo = 2.0 ** -8 * O.abs() + (2.0 ** -11 + 2.0 ** -13 + 2.0 ** -20 + 2 * e)[..., None] * (P @ v.abs())
    bo = bo + n * 2.0 ** -29 * (P * v.abs().amax(-1)[:, :, None]).amax(-1)[..., None]
    return O, L, bo, e + 2.0 ** -20 * L.abs().clamp(min=1)


@pytest.mark.parametrize("rows,B", [(1, 64), (4, 64), (8, 64), (16, 64), (20, 64), (24, 80)])
@pytest.mark.parametrize("d", DIMS)
def test_several_whole_units_a_cta(fa, d, rows, B):
    """More units than SMs, each of at most 24 steps: CTAs take several units
    whole, and their stretches of the list begin where units do."""
    torch = torch_cuda()
    rng = np.random.default_rng(d + rows)
    Hkv, page, N = 8, 64, 760
    f = Filled(fa, rng, [N] * 3, Hkv, d, page, room=8)  # three stored sequences, which all others share
    at = np.arange(B) % 3
    lens = rng.integers(0, N + 1, B)
    lens[:5] = (N, 0, 1, 768 - 8, 32)
    plan = fa.fa_kv4_fwd_plan(B, Hkv * rows, Hkv, 1, d, page, 12, torch.cuda.get_device_properties(0).multi_processor_count)
    assert plan["whole"] == 1 and plan["launches"] == 1 and plan["grid"] < plan["units"] and plan["max_steps"] == 24
    if rows in (16, 24):  # the units with two and three tiles of rows
        assert plan["unit_rows"] == (8 if d == 256 else 24 if rows == 24 and d <= 96 else 16)
    qd, _ = normal(rng, (B, Hkv * rows, 1, d))
    o, lse = fa.kv4_forward(qd, f.cache, ints(f.table[at][:, :12]), ints(lens))
    assert fa.fa_poll_status() == fa.FA_OK
    k, v = (torch.from_numpy(x).cuda()[torch.from_numpy(at).cuda()] for x in (f.k, f.v))
    n = torch.from_numpy(lens).cuda()
    O, L, bo, bl = attend64(qd.double().view(B, Hkv, rows, d), k, v, n, d ** -0.5)
    o, lse = o.double().view(B, Hkv, rows, d), lse.double().view(B, Hkv, rows)
    empty = n == 0
    assert (o[empty] == 0).all() and torch.isneginf(lse[empty]).all() and bool(empty.any())
    full = ~empty
    assert ((o - O)[full].abs() <= bo[full] + 1e-38).all(), ((o - O).abs() / bo)[full].max()
    assert ((lse - L)[full].abs() <= bl[full]).all(), ((lse - L).abs() / bl)[full].max()


def test_waits_that_give_up_are_reported(fa):
    """With no time to wait, the kernel may give up on its copies: it records
    FA_ERR_TIMEOUT, returns, and the next call is correct."""
    rng = np.random.default_rng(12)
    f = Filled(fa, rng, [5000, 3000], 2, 128, 64)
    qd, q = normal(rng, (2, 4, 1, 128))
    before = fa.fa_set_wait_timeout_ns(0)
    try:
        fa.kv4_forward(qd, f.cache, f.td, f.ld)
        assert fa.fa_poll_status() in (fa.FA_OK, fa.FA_ERR_TIMEOUT)
    finally:
        fa.fa_set_wait_timeout_ns(before)
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, [5000, 3000], 128 ** -0.5, "none")


@pytest.mark.parametrize("d,H,lens", [(128, 4, [5000, 3000]), (64, 2, [40, 0]), (96, 40, [900, 4000]), (256, 8, [7, 600])])
def test_every_wait_runs_out(fa, d, H, lens):
    """Copies that never arrive in full: every wait gives up after its limit
    and the drain after its own (0.1 s), the call is reported once and the next
    one is correct."""
    torch = torch_cuda()
    rng = np.random.default_rng(d)
    f = Filled(fa, rng, lens, 2, d, 64)
    qd, q = normal(rng, (2, H, 1, d))
    o, lse = torch.empty_like(qd), torch.empty((2, H, 1), device="cuda")
    assert fa.fa_poll_status() == fa.FA_OK
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    fa.fa_selftest_kv4_timeout(qd, f.cache, f.td, f.ld, o, lse, 20_000_000)
    end.record()
    assert fa.fa_poll_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_poll_status() == fa.FA_OK
    end.synchronize()
    assert 120 <= start.elapsed_time(end) < 2000  # ms: the wait's limit, then the drain's
    o, lse = fa.kv4_forward(qd, f.cache, f.td, f.ld)
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, "none")
    with pytest.raises(fa.FaError) as e:
        fa.fa_selftest_kv4_timeout(qd, f.cache, f.td, f.ld, o, lse, 3_000_000_000)
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        fa.fa_selftest_kv4_timeout(qd, f.cache, f.td, f.ld, o, lse[:1], 20_000_000)


# --------------------------------------------------------- used together

@pytest.mark.parametrize("d", (64, 128, 256))
def test_prompt_chunk_and_steps(fa, caller, d):
    """A prompt is written, a second chunk attends over the history read back
    (the bf16 kernels) and is written too, then single tokens are appended and
    attended to: every result is that of the held values."""
    torch = torch_cuda()
    rng = np.random.default_rng(d)
    B, H, Hkv, page, prompt, chunk, steps = 2, 4, 2, 32, 150, 140, 5
    total = prompt + chunk + steps
    kd, k = normal(rng, (B, Hkv, total, d))
    vd, v = normal(rng, (B, Hkv, total, d))
    qd, q = normal(rng, (B, H, total, d))
    hk, hv = kv4.held(k), kv4.held(v)
    table, n = make_table(rng, B, -(-total // page))
    cache, td = fa.kv4_cache(n, Hkv, page, d), ints(table)

    def piece(x, a, b):
        return x[:, :, a:b].contiguous()

    at = lambda x: ints([x] * B)  # noqa: E731
    fa.fa_kv4_write(piece(kd, 0, prompt), piece(vd, 0, prompt), cache, td, at(0))
    end = prompt + chunk
    fa.fa_kv4_write(piece(kd, prompt, end), piece(vd, prompt, end), cache, td, at(prompt))
    ko, vo = (torch.empty((B, Hkv, end, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_kv4_read(cache, td, at(0), ko, vo)
    o, lse = fa.forward(piece(qd, prompt, end), ko, vo, causal="bottom_right")
    assert np.array_equal(host(ko), kv4.to_bf16(hk[:, :, :end]))
    from parity import check_lse, check_o
    rk, rv = (kv4.to_bf16(x[:, :, :end]).repeat(H // Hkv, 1) for x in (hk, hv))
    O, L = att.forward(q[:, :, prompt:end], rk, rv, d ** -0.5, True, offset=prompt)
    check_o(host(o), O, "chunk")
    check_lse(lse.cpu().numpy(), L, "chunk")
    for s in range(steps):
        n_now = end + s + 1
        fa.fa_kv4_write(piece(kd, n_now - 1, n_now), piece(vd, n_now - 1, n_now), cache, td, at(n_now - 1))
        qs = piece(qd, n_now - 1, n_now)
        o, lse = fa.kv4_forward(qs, cache, td, at(n_now), causal="bottom_right")
        check_attend(o, lse, q[:, :, n_now - 1:n_now], hk, hv, [n_now] * B, d ** -0.5, "bottom_right", f"step {s}")
    assert fa.fa_poll_status() == fa.FA_OK


def test_captured_steps_and_two_graphs(fa):
    """A decoding step (append, attend) captured once and replayed with new
    inputs; two captured steps of two caches replayed at the same time on two
    streams."""
    torch = torch_cuda()
    rng = np.random.default_rng(20)
    d, H, Hkv, page, steps = 128, 8, 2, 16, 6
    jobs = []
    for lens in ([2000, 37], [5, 3001]):
        f = Filled(fa, rng, lens, Hkv, d, page, room=steps)
        qd, q = normal(rng, (steps, 2, H, 1, d))
        kd, k = normal(rng, (steps, 2, Hkv, 1, d))
        vd, v = normal(rng, (steps, 2, Hkv, 1, d))
        j = {"f": f, "q": q, "kd": kd, "vd": vd, "qd": qd, "hk": kv4.held(k), "hv": kv4.held(v),
             "in": [torch.empty_like(x[0]) for x in (qd, kd, vd)], "pos": ints(lens), "len": ints(lens),
             "o": torch.empty((2, H, 1, d), dtype=torch.bfloat16, device="cuda"),
             "lse": torch.empty((2, H, 1), dtype=torch.float32, device="cuda"), "stream": torch.cuda.Stream()}
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=j["stream"]):
            j["len"].copy_(j["pos"] + 1)
            fa.fa_kv4_write(j["in"][1], j["in"][2], f.cache, f.td, j["pos"])
            fa.fa_kv4_fwd(j["in"][0], f.cache, f.td, j["len"], j["o"], j["lse"], causal="bottom_right")
            j["pos"].add_(1)
        j["graph"] = g
        jobs.append(j)
    torch.cuda.synchronize()
    got = [[], []]
    for s in range(steps):
        for i, j in enumerate(jobs):
            with torch.cuda.stream(j["stream"]):
                for x, src in zip(j["in"], (j["qd"], j["kd"], j["vd"])):
                    x.copy_(src[s])
                j["graph"].replay()
                got[i].append((j["o"].clone(), j["lse"].clone()))
    torch.cuda.synchronize()
    assert fa.fa_poll_status() == fa.FA_OK
    for i, j in enumerate(jobs):
        f = j["f"]
        for b in range(2):
            n0 = f.lens[b]
            k = np.concatenate([f.k[b, :, :n0], j["hk"][:, b, :, 0].transpose(1, 0, 2)], 1)
            v = np.concatenate([f.v[b, :, :n0], j["hv"][:, b, :, 0].transpose(1, 0, 2)], 1)
            for s in range(steps):
                o, lse = got[i][s]
                check_attend(o[b:b + 1], lse[b:b + 1], j["q"][s, b:b + 1], k[None], v[None], [n0 + s + 1], d ** -0.5,
                             "bottom_right", f"graph {i} step {s}")


def test_sequences_that_share_pages(fa):
    """A prompt's pages stand in several sequences' tables, a page twice in
    one of them."""
    rng = np.random.default_rng(23)
    d, page, n = 128, 32, 150
    f = Filled(fa, rng, [n], 2, d, page)
    full = f.table[0, :4]
    table = np.stack([full, full[[0, 1, 1, 0]], full[[3, 2, 1, 0]]])
    lens = [128, 100, 128]
    at = np.concatenate([np.arange(128)[None], np.r_[0:64, 32:64, 0:32][None], np.r_[96:128, 64:96, 32:64, 0:32][None]])
    k, v = (np.stack([x[0][:, i] for i in at]) for x in (f.k, f.v))
    qd, q = normal(rng, (3, 8, 2, d))
    o, lse = fa.kv4_forward(qd, f.cache, ints(table), ints(lens), causal="bottom_right")
    assert fa.fa_poll_status() == fa.FA_OK
    check_attend(o, lse, q, k, v, lens, d ** -0.5, "bottom_right")
    torch = torch_cuda()
    ko, vo = (torch.empty((3, 2, 128, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_kv4_read(f.cache, ints(table), ints([0] * 3), ko, vo)
    assert np.array_equal(host(ko), kv4.to_bf16(k)) and np.array_equal(host(vo), kv4.to_bf16(v))


CAPTURED_FIRST = """
import torch
import exact_attention_92_gb300 as fa
x = torch.randn((1, 1, 64, 64), device="cuda").to(torch.bfloat16)
fa.forward(x, x, x)  # the library's first call on the device may not be captured
torch.cuda.synchronize()
for d, rows, pages in ((128, 1, 200), (64, 16, 9000), (96, 6, 3)):
    cache = fa.kv4_cache(4, 1, 16, d)
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, :3] = torch.tensor([2, 0, 3], device="cuda")
    zero, n = (torch.full((1,), i, dtype=torch.int32, device="cuda") for i in (0, 40))
    k, v = (torch.randn((1, 1, 40, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, rows, 1, d), device="cuda").to(torch.bfloat16)
    ko, vo, o = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)
    lse = torch.empty((1, rows, 1), device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_kv4_write(k, v, cache, table, zero)
        fa.fa_kv4_read(cache, table, zero, ko, vo)
        fa.fa_kv4_fwd(q, cache, table, n, o, lse)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
    got, got_ko = o.clone(), ko.clone()
    fa.fa_kv4_read(cache, table, zero, ko, vo)
    fa.fa_kv4_fwd(q, cache, table, n, o, lse)
    assert fa.fa_poll_status() == fa.FA_OK
    assert torch.equal(o, got) and torch.equal(ko, got_ko) and bool((ko != 0).any())
    s = torch.softmax(q[0, :, 0].float() @ ko[0, 0].float().T / d ** 0.5, -1)
    assert (s @ vo[0, 0].float() - o[0, :, 0].float()).abs().max() < 0.05
print("done")
"""


def test_first_calls_may_be_captured(fa):
    """Kernels that no call has launched before, captured in a new process."""
    import os
    import subprocess
    import sys

    r = subprocess.run([sys.executable, "-c", CAPTURED_FIRST], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr


def test_calls_at_once_on_two_streams(fa):
    torch = torch_cuda()
    rng = np.random.default_rng(21)
    jobs = []
    for d, lens in ((128, [4000, 900]), (64, [1000, 5000])):
        f = Filled(fa, rng, lens, 2, d, 64)
        qd, q = normal(rng, (2, 6, 1, d))
        jobs.append((f, d, lens, qd, q, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for rep in range(5):
        for f, d, lens, qd, q, st in jobs:
            with torch.cuda.stream(st):
                outs.append(fa.kv4_forward(qd, f.cache, f.td, f.ld))
    torch.cuda.synchronize()
    assert fa.fa_poll_status() == fa.FA_OK
    for i, (o, lse) in enumerate(outs):
        f, d, lens, qd, q, _ = jobs[i % 2]
        check_attend(o, lse, q, f.k, f.v, lens, d ** -0.5, "none")


def test_calls_from_several_threads(fa, caller):
    """Host threads, each with a stream and a cache of its own, call at once."""
    import threading

    torch = torch_cuda()
    rng = np.random.default_rng(25)
    jobs, errors = [], []
    for d, lens in ((128, [2000, 31]), (64, [700, 900]), (96, [5, 0]), (256, [300, 1500])):
        f = Filled(fa, rng, lens, 2, d, 32)
        qd, q = normal(rng, (2, 6, 1, d))
        jobs.append((f, d, lens, qd, q, torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def work(f, d, lens, qd, q, st, outs):
        try:
            with torch.cuda.stream(st):
                for _ in range(20):
                    outs.append(fa.kv4_forward(qd, f.cache, f.td, f.ld))
        except Exception as e:  # reported by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and fa.fa_poll_status() == fa.FA_OK
    for f, d, lens, qd, q, st, outs in jobs:
        assert len(outs) == 20
        check_attend(*outs[0], q, f.k, f.v, lens, d ** -0.5, "none")
        assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs)


def test_launches_are_counted(fa):
    torch = torch_cuda()
    rng = np.random.default_rng(22)
    ids = (fa.FA_KERNEL_KV4_WRITE, fa.FA_KERNEL_KV4_READ, fa.FA_KERNEL_KV4_FWD, fa.FA_KERNEL_KV4_MERGE)
    before = [fa.fa_launch_count(i) for i in ids]
    f = Filled(fa, rng, [40], 1, 64, 16)
    out = torch.empty((1, 1, 40, 64), dtype=torch.bfloat16, device="cuda")
    fa.fa_kv4_read(f.cache, f.td, ints([0]), out, out.clone())
    fa.kv4_forward(out[:, :, :1].contiguous(), f.cache, f.td, f.ld)
    torch.cuda.synchronize()
    assert [fa.fa_launch_count(i) - n for i, n in zip(ids, before)] == [1, 1, 1, 0]
    # The call follows its plan: a table for many tokens means a merge.
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    wide = ints(np.repeat(f.table, 200, 1))
    for table in (f.td, wide):
        plan = fa.fa_kv4_fwd_plan(1, 1, 1, 1, 64, 16, table.shape[1], sms)
        before = [fa.fa_launch_count(i) for i in ids[2:]]
        fa.kv4_forward(out[:, :, :1].contiguous(), f.cache, table, f.ld)
        assert [fa.fa_launch_count(i) - n for i, n in zip(ids[2:], before)] == [1, plan["launches"] - 1]
    assert plan["launches"] == 2


@pytest.mark.parametrize("d", DIMS)
def test_cache_calls_behind_a_backward(fa, d):
    """A call over the cache may start while the kernels of a backward ahead
    of it are still running: the gradients written into a cache are the final
    ones, and reading into the backward's own inputs disturbs none of them.
    Few keys under many query rows: dQ's units are done long before dK's."""
    torch = torch_cuda()
    rng = np.random.default_rng(d)
    Nq, Nk, page = 16384, 100, 16
    qd, _ = normal(rng, (1, 1, Nq, d))
    kd, _ = normal(rng, (1, 1, Nk, d))
    vd, _ = normal(rng, (1, 1, Nk, d))
    gd, _ = normal(rng, (1, 1, Nq, d))
    o, lse = fa.forward(qd, kd, vd)
    want = fa.backward(qd, kd, vd, o, lse, gd)
    torch.cuda.synchronize()
    table, n = make_table(rng, 1, -(-Nk // page))
    cache, other, td, zero = fa.kv4_cache(n, 1, page, d), fa.kv4_cache(n, 1, page, d), ints(table), ints([0])
    for _ in range(5):
        k, v = kd.clone(), vd.clone()
        dq, dk, dv = torch.zeros_like(qd), torch.zeros_like(k), torch.zeros_like(v)
        torch.cuda.synchronize()
        fa.fa_bwd_general(qd, k, v, o, lse, gd, dq, dk, dv)
        fa.fa_kv4_read(other, td, zero, k, v)  # zeros
        torch.cuda.synchronize()
        for got, w in zip((dq, dk, dv), want):
            assert torch.equal(got, w)
        dk.zero_(), dv.zero_()
        torch.cuda.synchronize()
        fa.fa_bwd_general(qd, kd, vd, o, lse, gd, dq, dk, dv)
        fa.fa_kv4_write(dk, dv, cache, td, zero)
        fa.fa_kv4_read(cache, td, zero, k, v)
        for got, w in ((k, want[1]), (v, want[2])):
            assert np.array_equal(host(got), kv4.to_bf16(kv4.held(host(w))))
    assert fa.fa_poll_status() == fa.FA_OK
