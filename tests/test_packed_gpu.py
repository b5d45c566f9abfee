"""Attention over packed sequences on the GPU against the oracle in fp64 (bounds in packed_util)."""

import math

import numpy as np
import pytest

from gpu_util import ensure_built, host, torch_cuda
from oracle import packed as oracle
from packed_util import check_forward, i32, make, scale_of, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    torch_cuda()
    return ensure_built()


def _run(fa, lq, lk, H, Hkv, d, causal, used=None, seed=0, pad=0, prefix=0, q=None, k=None, v=None, scale=None):
    torch = torch_cuda()
    tensors = make(lq, lk, H, Hkv, d, seed, pad)
    q, k, v = (t if given is None else given for t, given in zip(tensors, (q, k, v)))
    cq, ck = starts(lq), starts(lk)
    scale = scale or scale_of(d)
    args = (i32(cq), i32(ck), None if used is None else i32(used), causal, scale)
    pre = None
    if prefix:
        _, kp, vp = make([1], [prefix], H, Hkv, d, seed + 1000)
        pre = (host(kp), host(vp))
        o, lse = fa.prefix_forward(q, kp, vp, k, v, *args)
    else:
        o, lse = fa.packed_forward(q, k, v, *args)
    assert fa.fa_poll_status() == fa.FA_OK
    want = oracle.forward(host(q), host(k), host(v), cq, ck, scale, causal, used, pre)
    check_forward(o, lse, want, d, slice(cq[0], cq[-1]))
    assert not host(o)[cq[-1]:].any() and bool(torch.isneginf(lse[:, cq[-1]:]).all())
    return o, lse


LENGTHS = [
    ([1], [1]),
    ([64], [64]),
    ([129], [129]),
    ([257, 1, 128, 0, 127, 300], [257, 1, 128, 0, 127, 300]),
    ([5, 3, 0, 17], [0, 200, 40, 17]),
    ([1, 1, 1, 1, 1], [700, 1, 0, 129, 128]),
    ([200, 33, 500], [130, 700, 500]),
]


@pytest.mark.parametrize("lq,lk", LENGTHS)
@pytest.mark.parametrize("causal", ["none", "top_left", "bottom_right"])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 2, 128), (3, 1, 96)])
def test_against_oracle(fa, lq, lk, causal, H, Hkv, d):
    _run(fa, lq, lk, H, Hkv, d, causal, pad=3)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (12, 2), (7, 7), (16, 1), (48, 1), (71, 1), (130, 1), (260, 2)])
def test_query_heads_of_a_group(fa, H, Hkv):
    _run(fa, [40, 1, 13], [40, 300, 13], H, Hkv, 64, "bottom_right")


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("H,Hkv,lens", [(4, 1, [3000, 5, 900]), (1, 1, [5000]), (8, 8, [1500, 700, 2]),
                                        (4, 1, [5000, 5, 900]), (8, 8, [2500, 2700, 2])])
def test_long_sequences_are_cut_between_ctas(fa, d, H, Hkv, lens):
    _run(fa, lens, lens, H, Hkv, d, "top_left", seed=2)


@pytest.mark.parametrize("d", [64, 128])
def test_decoding_over_a_padded_cache(fa, d):
    """One to nine new rows a sequence over a cache with room for more; what is behind the used keys is NaN."""
    torch = torch_cuda()
    lq, used, room = [1, 9, 1, 1, 4], [3000, 9, 1, 0, 777], 3008
    lk = [room] * 5
    _, k, v = make(lq, lk, 8, 2, d, 7)
    for b, n in enumerate(used):
        k[b * room + n:(b + 1) * room] = float("nan")
        v[b * room + n:(b + 1) * room] = float("nan")
    q, _, _ = make(lq, [1], 8, 2, d, 8)
    cq, ck = starts(lq), starts(lk)
    o, lse = fa.packed_forward(q, k, v, i32(cq), i32(ck), i32(used), "bottom_right")
    clean = [torch.nan_to_num(x) for x in (k, v)]
    want = oracle.forward(host(q), host(clean[0]), host(clean[1]), cq, ck, scale_of(d), "bottom_right", used)
    check_forward(o, lse, want, d)


@pytest.mark.parametrize("causal", ["none", "top_left"])
def test_nan_stays_in_its_sequence(fa, causal):
    """NaN and infinities in q, k, v of one sequence and of rows of no sequence change no bit of the others."""
    torch = torch_cuda()
    lens = [100, 70, 130, 29]
    q, k, v = make(lens, lens, 4, 2, 128, 3, pad=5)
    cu = i32(starts(lens))
    clean, clean_l = fa.packed_forward(q, k, v, cu, causal=causal)
    for x in (q, k, v):
        x[100:170] = float("nan")
        x[150:160] = float("inf")
        x[sum(lens):] = float("nan")
    o, lse = fa.packed_forward(q, k, v, cu, causal=causal)
    keep = [*range(100), *range(170, sum(lens))]
    assert torch.equal(o[keep], clean[keep]) and torch.equal(lse[:, keep], clean_l[:, keep])
    assert bool(torch.isnan(o[100:170]).any(-1).all())


def test_layouts_and_strides(fa):
    """Slices of a fused projection, [heads, tokens, d], outputs inside larger ones and at 16-byte places: the same bits as
    contiguous tensors."""
    torch = torch_cuda()
    lens, H, Hkv, d = [90, 200, 3], 6, 2, 128
    T = sum(lens)
    q, k, v = make(lens, lens, H, Hkv, d, 4)
    cu = i32(starts(lens))
    o, lse = fa.packed_forward(q, k, v, cu, causal=True)
    fused = torch.cat([q, k, v], 1)
    o2, l2 = fa.packed_forward(fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:], cu, causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    qh, kh, vh = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    big = torch.zeros(H, T + 7, d, dtype=torch.bfloat16, device="cuda")
    oh = big.transpose(0, 1)[:T]
    l3 = torch.zeros(H, T, device="cuda")
    fa.fa_packed_fwd(qh, kh, vh, oh, l3, cu, cu, causal=True)
    assert torch.equal(oh, o) and torch.equal(l3, lse) and not bool(big[:, T:].any())
    room = torch.zeros(T, H * d + 8, dtype=torch.bfloat16, device="cuda")
    odd = room[:, 8:].view(T, H, d)
    fa.fa_packed_fwd(q, k, v, odd, l3, cu, cu, causal=True)
    assert torch.equal(odd, o) and not bool(room[:, :8].any())


def test_rows_of_no_sequence_are_left_as_they_were(fa):
    torch = torch_cuda()
    lens, lead, pad = [60, 140], 9, 11
    q, k, v = make([lead + sum(lens) + pad], [lead + sum(lens) + pad], 4, 4, 64, 5)
    cu = i32([lead + x for x in starts(lens)])
    o, lse = torch.full_like(q, 7.0), torch.full((4, q.shape[0]), 3.0, device="cuda")
    fa.fa_packed_fwd(q, k, v, o, lse, cu, cu)
    assert bool((o[:lead] == 7).all()) and bool((o[-pad:] == 7).all())
    assert bool((lse[:, :lead] == 3).all()) and bool((lse[:, -pad:] == 3).all())
    want = oracle.forward(host(q), host(k), host(v), cu.tolist(), cu.tolist(), scale_of(64), "none")
    check_forward(o, lse, want, 64, slice(lead, lead + sum(lens)))


PREFIXES = [
    (1, [1], [1]),
    (128, [5, 0, 40], [5, 10, 40]),
    (1000, [1] * 40, [(7 * i) % 150 for i in range(40)]),
    (700, [300, 1, 200], [300, 5, 900]),
    (5000, [1, 2, 3], [0, 2, 300]),
    (257, [3] * 90, [3] * 90),
]


@pytest.mark.parametrize("P,lq,lk", PREFIXES)
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 2, 128), (3, 1, 96)])
def test_prefix_against_oracle(fa, P, lq, lk, H, Hkv, d):
    _run(fa, lq, lk, H, Hkv, d, "bottom_right", prefix=P, pad=2)


def test_prefix_without_own_keys(fa):
    torch = torch_cuda()
    q, kp, vp = make([4, 7], [300], 4, 2, 64, 6)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = fa.prefix_forward(q, kp, vp, none, none, i32([0, 4, 11]), i32([0, 0, 0]))
    want = oracle.forward(host(q), host(none), host(none), [0, 4, 11], [0, 0, 0], scale_of(64), "none",
                          prefix=(host(kp), host(vp)))
    check_forward(o, lse, want, 64)


def test_large_scores_and_long_rows(fa):
    """Logits up to hundreds: the running maximum moves, weights vanish."""
    torch = torch_cuda()
    lens = [1200, 300]
    q, k, v = make(lens, lens, 2, 1, 64, 9)
    _run(fa, lens, lens, 2, 1, 64, "top_left", q=q * 8, k=k * 4, v=v)
    _run(fa, lens, lens, 2, 1, 64, "none", q=q, k=k, v=v, scale=1e-3)


def test_repeatable_graphs_and_streams(fa):
    """The same bits from run to run, on another stream, and from a graph whose lengths change between replays."""
    torch = torch_cuda()
    lens = [700, 90, 1300, 0, 33]
    q, k, v = make(lens, lens, 8, 2, 128, 10)
    cu = i32(starts(lens))
    o, lse = fa.packed_forward(q, k, v, cu, causal=True)
    for _ in range(3):
        o2, l2 = fa.packed_forward(q, k, v, cu, causal=True)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o3, l3 = fa.packed_forward(q, k, v, cu, causal=True)
    s.synchronize()
    assert torch.equal(o, o3) and torch.equal(lse, l3)
    og, lg = torch.zeros_like(o), torch.zeros_like(lse)
    other, other_l = torch.zeros_like(o), torch.zeros_like(lse)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        fa.fa_packed_fwd(q, k, v, og, lg, cu, cu, causal=True)
    with torch.cuda.graph(graphs[1]):
        fa.fa_packed_fwd(q, k, v, other, other_l, cu, cu, causal=False)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(og, o) and torch.equal(lg, lse)
    full, _ = fa.packed_forward(q, k, v, cu, causal=False)
    assert torch.equal(other, full)
    lens2 = [10, 1900, 0, 200, 13]
    cu.copy_(i32(starts(lens2)))
    graphs[0].replay()
    torch.cuda.synchronize()
    want, want_l = fa.packed_forward(q, k, v, cu, causal=True)
    assert torch.equal(og, want) and torch.equal(lg, want_l)


def test_bad_bounds_are_skipped_and_reported(fa):
    """Bounds out of order or out of range (checked on the device ahead of every use): the sequence is skipped."""
    torch = torch_cuda()
    lens = [50, 60, 70]
    q, k, v = make(lens, lens, 2, 2, 64, 11)
    good = i32(starts(lens))
    o, lse = fa.packed_forward(q, k, v, good)
    T = sum(lens)
    for cu_q, cu_k, used, skipped in (
            ([0, 50, 110, T + 1], starts(lens), None, [2]), ([-1, 50, 110, T], starts(lens), None, [0]),
            (starts(lens), [0, 50, 110, T + 5], None, [2]), (starts(lens), starts(lens), [50, 61, 70], [1]),
            (starts(lens), starts(lens), [50, -1, 70], [1]), (starts(lens), [0, 50, -7, T], None, [1, 2])):
        out, l = torch.full_like(q, 5.0), torch.zeros_like(lse)
        fa.fa_packed_fwd(q, k, v, out, l, i32(cu_q), i32(cu_k), None if used is None else i32(used))
        assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
        assert fa.fa_poll_status() == fa.FA_OK
        at = starts(lens)
        for b in range(3):
            part = slice(at[b], at[b + 1])
            if b in skipped:
                assert bool((out[part] == 5).all())
            else:
                assert torch.equal(out[part], o[part])
    # With a prefix, rows that its blocks do not cover included.
    fa.prefix_forward(q, k[:9], v[:9], k, v, i32([120, 10, 60, 61]), i32(starts(lens)))
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX


def test_failed_workspace_is_reported(fa, monkeypatch):
    lens = [4500, 900]
    q, k, v = make(lens, lens, 2, 2, 64, 12)
    monkeypatch.setenv("FA_TEST_FAIL_ALLOC", "1")
    with pytest.raises(fa.FaError) as e:
        fa.packed_forward(q, k, v, i32(starts(lens)))
    assert e.value.status == fa.FA_ERR_NO_MEMORY
    monkeypatch.delenv("FA_TEST_FAIL_ALLOC")
    _run(fa, lens, lens, 2, 2, 64, "none")


def test_refusals(fa):
    torch = torch_cuda()
    lens = [50, 60]
    q, k, v = make(lens, lens, 4, 2, 64, 13)
    cu = i32(starts(lens))
    o, lse = torch.empty_like(q), torch.empty(4, 110, device="cuda")
    good = dict(q=q, k=k, v=v, o=o, lse=lse, cu_q=cu, cu_k=cu)
    for bad in (dict(q=q.float()), dict(q=q[None]), dict(k=k[:-1]), dict(v=v[..., :32]), dict(o=o[:, :2]),
                dict(lse=lse.double()), dict(lse=lse[:, :9]), dict(cu_q=cu.long()), dict(cu_q=cu[:1]), dict(cu_q=None),
                dict(cu_k=cu[:-1]), dict(cu_k=cu.cpu()), dict(used_k=cu), dict(q=q.cpu()),
                dict(o=o[:, :1].expand(110, 4, 64)), dict(q=q.transpose(1, 2)), dict(causal="up")):
        with pytest.raises((ValueError, TypeError)):
            fa.fa_packed_fwd(**{**good, **bad})
    for bad in (dict(scale=float("inf")), dict(scale=-1.0), dict(causal=3), dict(q=q[:, :3], o=o[:, :3], lse=lse[:3]),
                dict(k=k[:, :1].expand(110, 2, 64))):
        with pytest.raises(fa.FaError) as e:
            fa.fa_packed_fwd(**{**good, **bad})
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    wide = [torch.zeros(110, 2, 256, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    with pytest.raises(fa.FaError) as e:
        fa.fa_packed_fwd(*wide, lse[:2], cu, cu)
    assert e.value.status == fa.FA_ERR_UNSUPPORTED
    with pytest.raises(fa.FaError):
        fa.fa_prefix_fwd(q, k[:0], v[:0], k, v, o, lse, cu, cu)
    assert fa.fa_poll_status() == fa.FA_OK


def test_launches(fa):
    """The forward kernel alone over few keys; with a plan, and the merge where units can be cut."""
    ids = (fa.FA_KERNEL_PACKED_PLAN, fa.FA_KERNEL_PACKED_FWD, fa.FA_KERNEL_PACKED_MERGE)
    for lens, plans, merges in (([40, 50], 0, 0), ([13] * 33, 1, 0), ([3000, 2400], 1, 1)):
        q, k, v = make(lens, lens, 2, 2, 64, 14)
        before = [fa.fa_launch_count(i) for i in ids]
        fa.packed_forward(q, k, v, i32(starts(lens)))
        assert [fa.fa_launch_count(i) - n for i, n in zip(ids, before)] == [plans, 1, merges]
