"""Packed sequences: what other sequences hold, their bad bounds, and what shared memory held before, move no bit of a
sequence's results."""

import pytest

from gpu_util import ensure_built, torch_cuda
from packed_util import i32, make, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    torch_cuda()
    return ensure_built()


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("H,Hkv,pad,prefix", [(2, 2, 0, 0), (6, 2, 0, 0), (2, 2, 9000, 0), (8, 1, 9000, 0), (2, 2, 9000, 300),
                                              (2, 2, 0, 300)])
def test_large_neighbours(fa, d, H, Hkv, pad, prefix):
    """Queries of the next sequence, and of no sequence, that share a tile with the first one's: their scores grow by hundreds
    from one key tile to the next.  (`pad` rows of no sequence: room that takes a plan.)"""
    torch = torch_cuda()
    lq, lk = [5, 20], [1100, 40]
    q, k, v = make(lq, lk, H, Hkv, d, 300, pad=pad + 30)
    _, kp, vp = make([1], [max(1, prefix)], H, Hkv, d, 301)
    cu = (i32(starts(lq)), i32(starts(lk)))

    def call():
        return fa.prefix_forward(q, kp, vp, k, v, *cu) if prefix else fa.packed_forward(q, k, v, *cu)

    o, lse = call()
    for first in (5, 25):  # of the next sequence; of none
        was = q.clone()
        q[first:] *= 256
        got, got_l = call()
        assert torch.equal(got[:first], o[:first]) and torch.equal(got_l[:, :first], lse[:, :first])
        q.copy_(was)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("H,Hkv,lens", [(3, 1, [84] * 8), (12, 4, [1300, 900, 30]), (7, 1, [18] * 40), (5, 5, [84] * 8)])
def test_what_shared_memory_held(fa, d, H, Hkv, lens):
    """Rows of a tile that no copy writes (126 and 127 of a group of three) hold an earlier call's queries, large or zero."""
    torch = torch_cuda()
    q, k, v = make(lens, [n + 700 for n in lens], H, Hkv, d, 310)
    cu = (i32(starts(lens)), i32(starts([n + 700 for n in lens])))
    fill, fk, fv = make([256 * 160], [100], 1, 1, d, 311)
    fill_cu = (i32([0, 256 * 160]), i32([0, 100]))
    spare, spare_l = torch.zeros_like(fill), torch.zeros(1, fill.shape[0], device="cuda")
    out = []
    for scale in (0.0, 256.0, 0.0):
        big = fill * scale
        o, lse = torch.zeros_like(q), torch.zeros(H, q.shape[0], device="cuda")
        torch.cuda.synchronize()
        fa.fa_packed_fwd(big, fk, fv, spare, spare_l, *fill_cu)
        fa.fa_packed_fwd(q, k, v, o, lse, *cu)
        torch.cuda.synchronize()
        out.append((o, lse))
    for o, lse in out[1:]:
        assert torch.equal(o, out[0][0]) and torch.equal(lse, out[0][1])


@pytest.mark.parametrize("d", [64, 128])
def test_bad_first_and_last_bounds_behind_a_shared_prefix(fa, d):
    """Only the sequence with the bad bound is skipped: the others have the bits of a call in which it is empty.  (Forty
    sequences behind 80 tiles: their rows go over the prefix together.)"""
    torch = torch_cuda()
    lq, H, Hkv, P = [3] * 40, 8, 2, 10240
    lk = [(7 * i) % 90 for i in range(40)]
    q, k, v = make(lq, lk, H, Hkv, d, 320)
    _, kp, vp = make([1], [P], H, Hkv, d, 321)
    T, at, cu_k = sum(lq), starts(lq), i32(starts(lk))

    def call(cu_q):
        o, lse = torch.full_like(q, 5.0), torch.full((H, T), 7.0, device="cuda")
        fa.fa_prefix_fwd(q, kp, vp, k, v, o, lse, i32(cu_q), cu_k)
        return o, lse, fa.fa_poll_status()

    for cu_q, clean, gone in (
            ([*at[:-1], 10], [*at[:-1], at[-2]], [(at[-2], T)]),      # the last one ends ahead of its start
            ([*at[:-1], -4], [*at[:-1], at[-2]], [(at[-2], T)]),
            ([*at[:-1], T + 9], [*at[:-1], at[-2]], [(at[-2], T)]),
            ([T + 5, *at[1:]], [at[1], *at[1:]], [(0, at[1])]),       # the first one starts behind the rows
            ([-3, *at[1:]], [at[1], *at[1:]], [(0, at[1])])):
        want, want_l, status = call(clean)
        assert status == fa.FA_OK
        o, lse, status = call(cu_q)
        assert status == fa.FA_ERR_BAD_INDEX
        assert torch.equal(o, want) and torch.equal(lse, want_l)
        for a, b in gone:
            assert bool((o[a:b] == 5).all()) and bool((lse[:, a:b] == 7).all())


@pytest.mark.parametrize("d", [64, 96, 128])
def test_calls_one_behind_the_other_read_their_own_units(fa, d):
    """Backward calls back to back, whose workspace is the same memory and whose units, L and D change from call to call: each
    has the bits that it has alone.  (The dQ kernel reads these ahead of its wait for the kernel before.)"""
    torch = torch_cuda()
    room, H, Hkv = 4000, 4, 2
    q, k, v = make([room], [room], H, Hkv, d, 330)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(331)).to(torch.bfloat16).cuda()
    cases = []
    for lens in ([3990], [5, 1200, 0, 700, 64, 1300], [129] * 30, [1000] * 4):
        lens = lens + [0] * (30 - len(lens))
        cu = i32(starts(lens))
        o, lse = fa.packed_forward(q, k, v, cu, causal=True)
        torch.cuda.synchronize()
        cases.append((cu, o, lse, fa.packed_backward(q, k, v, o, lse, do, cu, causal=True)))
        torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for cu, o, lse, _ in cases:
            got.append(fa.packed_backward(q, k, v, o, lse, do, cu, causal=True))
    for i, grads in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(grads, cases[i % len(cases)][3]))
