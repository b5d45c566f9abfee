"""Values that are not finite over packed sequences: a row that sees one comes out NaN in O and L, however its keys are cut
between CTAs and warpgroups; every other row is the oracle's (bounds in packed_util)."""

import numpy as np
import pytest

from gpu_util import ensure_built, host, torch_cuda
from oracle import packed as oracle
from packed_util import check_forward, i32, make, scale_of, starts

pytestmark = pytest.mark.gpu

# Whole units without a plan; halves of one; small and whole blocks cut by a plan; a prefix with blocks of its own (16 tiles
# of it a sequence would be walked 40 times); a prefix walked with the sequence's keys.
CASES = {
    "direct": ([200, 70], [200, 70], 4, 2, 0),
    "halves": ([3], [1500], 8, 2, 0),
    "cut_small": ([3, 2], [20000, 9], 4, 1, 0),
    "cut_whole": ([300, 5], [9000, 70], 2, 1, 0),
    "shared": ([1] * 40, [(7 * i) % 150 for i in range(40)], 8, 2, 8000),
    "walked": ([300, 1, 200], [300, 5, 900], 4, 2, 700),
}


@pytest.fixture(scope="module")
def fa():
    torch_cuda()
    return ensure_built()


def _inputs(case, d, seed):
    lq, lk, H, Hkv, P = CASES[case]
    q, k, v = make(lq, lk, H, Hkv, d, seed)
    kp, vp = make([1], [P], H, Hkv, d, seed + 1)[1:] if P else (None, None)
    return lq, lk, q, k, v, kp, vp


def _call(fa, lq, lk, q, k, v, kp, vp):
    args = (i32(starts(lq)), i32(starts(lk)), None, "bottom_right")
    return fa.packed_forward(q, k, v, *args) if kp is None else fa.prefix_forward(q, kp, vp, k, v, *args)


def _check(o, lse, want, bad, d):
    """`bad` [Tq] rows, every head of which is NaN; the others are `want`'s."""
    torch = torch_cuda()
    assert bad.any()
    at = torch.from_numpy(np.nonzero(bad)[0]).cuda()
    assert bool(torch.isnan(o[at]).all()), "a row that sees a NaN lost it in O"
    assert bool(torch.isnan(lse[:, at]).all()), "a row that sees a NaN lost it in L"
    keep = np.nonzero(~bad)[0].tolist()
    check_forward(o, lse, want, d, keep)


def _want(lq, lk, q, k, v, kp, vp, d):
    pre = None if kp is None else (host(kp), host(vp))
    return oracle.forward(host(q), host(k), host(v), starts(lq), starts(lk), scale_of(d), "bottom_right", None, pre)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("case", CASES)
def test_query(fa, case, d):
    """One channel of one query row, NaN or an infinity (whose scores have both signs: the softmax of an infinity is NaN)."""
    for value in (float("nan"), float("inf")):
        lq, lk, q, k, v, kp, vp = _inputs(case, d, 200)
        want = _want(lq, lk, q, k, v, kp, vp, d)
        row = lq[0] - 1
        q[row, :, 5] = value
        o, lse = _call(fa, lq, lk, q, k, v, kp, vp)
        bad = np.zeros(sum(lq), dtype=bool)
        bad[row] = True
        _check(o, lse, want, bad, d)
        assert fa.fa_poll_status() == fa.FA_OK


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("case", CASES)
def test_key(fa, case, d):
    """One channel of one key of the first sequence with keys, of its first, of a middle and of its last tile."""
    for part in (0.0, 0.4, 1.0):
        lq, lk, q, k, v, kp, vp = _inputs(case, d, 210)
        want = _want(lq, lk, q, k, v, kp, vp, d)
        b = next(i for i, n in enumerate(lk) if n)
        key = int(part * (lk[b] - 1))
        k[starts(lk)[b] + key, :, 3] = float("nan")
        o, lse = _call(fa, lq, lk, q, k, v, kp, vp)
        bad = np.zeros(sum(lq), dtype=bool)
        for i in range(lq[b]):
            bad[starts(lq)[b] + i] = key <= i + lk[b] - lq[b]
        _check(o, lse, want, bad, d)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("case", ["shared", "walked"])
def test_key_of_the_prefix(fa, case, d):
    """Every row sees it."""
    torch = torch_cuda()
    for part in (0.0, 0.5, 1.0):
        lq, lk, q, k, v, kp, vp = _inputs(case, d, 220)
        kp[int(part * (kp.shape[0] - 1)), :, 7] = float("nan")
        o, lse = _call(fa, lq, lk, q, k, v, kp, vp)
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case", ["halves", "cut_small", "shared"])
def test_all_keys_of_a_part(fa, case, d):
    """The first, or the second, half of the keys all NaN: a part has no score that is a number."""
    torch = torch_cuda()
    for half in (0, 1):
        lq, lk, q, k, v, kp, vp = _inputs(case, d, 230)
        keys, n = (k, lk[0]) if kp is None else (kp, kp.shape[0])
        keys[half * n // 2:(half + 1) * n // 2] = float("nan")
        o, lse = _call(fa, lq, lk, q, k, v, kp, vp)
        rows = lq[0] if kp is None else sum(lq)
        assert bool(torch.isnan(o[:rows]).all()) and bool(torch.isnan(lse[:, :rows]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_gradients(fa, d):
    """A NaN key of a sequence that is cut: dq of the rows that see it, and dk, dv of every key of theirs, are NaN; the other
    sequence's are those of the clean call."""
    torch = torch_cuda()
    lq, lk, H, Hkv, _ = CASES["cut_whole"]
    q, k, v = make(lq, lk, H, Hkv, d, 240)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(241)).to(torch.bfloat16).cuda()
    cu = (i32(starts(lq)), i32(starts(lk)))

    def grads():
        o, lse = fa.packed_forward(q, k, v, *cu, causal="none")
        return fa.packed_backward(q, k, v, o, lse, do, *cu, causal="none")

    clean = grads()
    k[4000, :, 3] = float("nan")
    dirty = grads()
    for x, y, n in zip(dirty, clean, (lq[0], lk[0], lk[0])):
        assert bool(torch.isnan(x[:n]).all())
        assert torch.equal(x[n:], y[n:])
