"""Gradients over packed sequences on the GPU, against the oracle's in fp64 within the bounds that the oracle works out from
the roundings (weights and dS to bf16, D from the forward's bf16 O, fp32 logits and sums).  The oracle's gradients are tested against
differences without a GPU."""

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


def _normal(like, seed):
    torch = torch_cuda()
    return torch.randn(like.shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def _check(got, want, names=("dq", "dk", "dv")):
    for n, g in zip(names, got):
        over = np.abs(host(g) - want[n]) - want[n + "_bound"]
        bad = ~(over <= 0.0)
        assert not bad.any(), f"{n}: {int(bad.sum())} beyond the bound, by {np.nanmax(over):.3e}"


def _run(fa, lq, lk, H, Hkv, d, causal, seed=0, pad=0):
    q, k, v = make(lq, lk, H, Hkv, d, seed, pad)
    do = _normal(q, seed + 500)
    cq, ck = starts(lq), starts(lk)
    a, b = i32(cq), i32(ck)
    o, lse = fa.packed_forward(q, k, v, a, b, causal=causal)
    grads = fa.packed_backward(q, k, v, o, lse, do, a, b, causal=causal)
    assert fa.fa_poll_status() == fa.FA_OK
    want = oracle.backward(host(q), host(k), host(v), host(do), cq, ck, scale_of(d), causal)
    _check(grads, want)
    for g, end in zip(grads, (cq[-1], ck[-1], ck[-1])):
        rest = host(g)[end:]
        assert not rest.any()
    return grads


LENGTHS = [
    ([1], [1]),
    ([128], [128]),
    ([129], [129]),
    ([257, 1, 128, 0, 127, 300], [257, 1, 128, 0, 127, 300]),
    ([5, 3, 0, 17], [0, 200, 40, 17]),
    ([200, 33, 500, 64], [130, 700, 500, 5]),
]


@pytest.mark.parametrize("lq,lk", LENGTHS)
@pytest.mark.parametrize("causal", ["none", "top_left", "bottom_right"])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 2, 128), (3, 3, 128), (6, 2, 64), (3, 1, 96), (2, 2, 96)])
def test_against_oracle(fa, lq, lk, causal, H, Hkv, d):
    _run(fa, lq, lk, H, Hkv, d, causal, pad=3)


@pytest.mark.parametrize("d", [64, 96, 128])
def test_longer_sequences(fa, d):
    lens = [1500, 3, 700, 0, 129, 1, 256, 255]
    _run(fa, lens, lens, 4, 1, d, "top_left", seed=3)


def test_many_sequences(fa):
    """More sequences than the planning kernel has threads, most short."""
    lens = [(7 * i) % 5 for i in range(1500)]
    lens[700] = 400
    _run(fa, lens, lens, 2, 1, 64, "top_left", seed=4)


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("causal", ["none", "top_left"])
def test_nan_stays_in_its_sequence(fa, d, causal):
    torch = torch_cuda()
    lens = [100, 70, 130, 29]
    q, k, v = make(lens, lens, 4, 2, d, 3, pad=5)
    do = _normal(q, 9)
    cu = i32(starts(lens))

    def grads():
        o, lse = fa.packed_forward(q, k, v, cu, causal=causal)
        o[sum(lens):], lse[:, sum(lens):] = float("nan"), float("nan")
        return fa.packed_backward(q, k, v, o, lse, do, cu, causal=causal)

    clean = grads()
    for x in (q, k, v, do):
        x[100:170] = float("nan")
        x[150:160] = float("inf")
        x[sum(lens):] = float("nan")
    dirty = grads()
    keep = [*range(100), *range(170, sum(lens))]
    for a, b in zip(clean, dirty):
        assert torch.equal(a[keep], b[keep])
        assert not bool(b[sum(lens):].any())


def test_layouts_and_strides(fa):
    """Gradients into the parts of one fused buffer, [heads, tokens, d], 16-byte places: the same bits."""
    torch = torch_cuda()
    lens, H, Hkv, d = [90, 200, 3], 6, 2, 128
    T = sum(lens)
    q, k, v = make(lens, lens, H, Hkv, d, 4)
    do = _normal(q, 5)
    cu = i32(starts(lens))
    o, lse = fa.packed_forward(q, k, v, cu, causal=True)
    want = fa.packed_backward(q, k, v, o, lse, do, cu, causal=True)
    fused = torch.cat([q, k, v], 1)
    out = torch.zeros_like(fused)
    parts = (slice(0, H), slice(H, H + Hkv), slice(H + Hkv, H + 2 * Hkv))
    fa.fa_packed_bwd(*(fused[:, s] for s in parts), o, lse, do, *(out[:, s] for s in parts), cu, cu, causal=True)
    assert torch.equal(out, torch.cat(want, 1))
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v, o, do)]
    got = [torch.zeros_like(x) for x in turned[:3]]
    fa.fa_packed_bwd(*turned[:4], lse, turned[4], *got, cu, cu, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    odd = []
    for x in (q, k, v):
        room = torch.zeros(T, x.shape[1] * d + 8, dtype=torch.bfloat16, device="cuda")
        odd.append(room[:, 8:].view(x.shape))
    fa.fa_packed_bwd(q, k, v, o, lse, do, *odd, cu, cu, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(odd, want))


def test_rows_of_no_sequence_are_left_and_unseen_rows_are_zero(fa):
    torch = torch_cuda()
    lead, pad = 9, 11
    q, k, v = make([lead + 300 + pad], [lead + 700 + pad], 4, 2, 64, 5)
    do = _normal(q, 6)
    cu_q, cu_k = i32([lead, lead + 100, lead + 300]), i32([lead, lead + 400, lead + 700])
    o, lse = fa.packed_forward(q, k, v, cu_q, cu_k, causal="top_left")
    dq, dk, dv = (torch.full_like(x, 7.0) for x in (q, k, v))
    fa.fa_packed_bwd(q, k, v, o, lse, do, dq, dk, dv, cu_q, cu_k, causal="top_left")
    for x in (dq, dk, dv):
        assert bool((x[:lead] == 7).all()) and bool((x[-pad:] == 7).all())
    for x in (dk, dv):
        assert not bool(x[lead + 100:lead + 400].any()) and not bool(x[lead + 600:lead + 700].any())
    want = oracle.backward(host(q), host(k), host(v), host(do), cu_q.tolist(), cu_k.tolist(), scale_of(64), "top_left")
    inside = {"dq": slice(lead, lead + 300), "dk": slice(lead, lead + 700), "dv": slice(lead, lead + 700)}
    for n, g in (("dq", dq), ("dk", dk), ("dv", dv)):
        over = np.abs(host(g) - want[n]) - want[n + "_bound"]
        over = float(over[inside[n]].max())
        assert over <= 0.0


def test_repeatable_graphs_and_streams(fa):
    torch = torch_cuda()
    lens = [700, 90, 1300, 0, 33]
    q, k, v = make(lens, lens, 8, 2, 128, 10)
    do = _normal(q, 11)
    cu = i32(starts(lens))
    o, lse = fa.packed_forward(q, k, v, cu, causal=True)
    want = fa.packed_backward(q, k, v, o, lse, do, cu, causal=True)
    for _ in range(3):
        again = fa.packed_backward(q, k, v, o, lse, do, cu, causal=True)
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = fa.packed_backward(q, k, v, o, lse, do, cu, causal=True)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    out = [torch.zeros_like(x) for x in (q, k, v)]
    og, lg = torch.zeros_like(o), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_packed_fwd(q, k, v, og, lg, cu, cu, causal=True)
        fa.fa_packed_bwd(q, k, v, og, lg, do, *out, cu, cu, causal=True)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    cu.copy_(i32(starts([10, 1900, 0, 200, 13])))
    graph.replay()
    torch.cuda.synchronize()
    o2, l2 = fa.packed_forward(q, k, v, cu, causal=True)
    want = fa.packed_backward(q, k, v, o2, l2, do, cu, causal=True)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_training_step_of_rotary_packed_attention(fa):
    """Rotary positions, attention and back, as a layer runs them: the gradients of the queries and keys ahead of the
    rotation are those of the oracle turned back (one more rounding on either side)."""
    torch = torch_cuda()
    from oracle import rope as rope_oracle

    lens, H, Hkv, d = [130, 40, 257], 4, 2, 64
    q, k, v = make(lens, lens, H, Hkv, d, 20)
    do = _normal(q, 21)
    cu = i32(starts(lens))
    pos = i32([i for n in lens for i in range(n)])
    freq = fa.rope_frequencies(d)
    ph = fa.rope_phases(freq)
    qr, kr = fa.rope(q, k, ph, positions=pos)
    o, lse = fa.packed_forward(qr, kr, v, cu, causal=True)
    dqr, dkr, dv = fa.packed_backward(qr, kr, v, o, lse, do, cu, causal=True)
    dq, dk = fa.rope(dqr, dkr, ph, positions=pos, inverse=True)
    assert fa.fa_poll_status() == fa.FA_OK
    check_forward(o, lse, oracle.forward(host(qr), host(kr), host(v), starts(lens), starts(lens), scale_of(d), "top_left"), d)
    want = oracle.backward(host(qr), host(kr), host(v), host(do), starts(lens), starts(lens), scale_of(d), "top_left")
    _check((dqr, dkr, dv), want)
    theta = rope_oracle.angles(pos.cpu().numpy(), freq)[:, None]
    for got, name in ((dq, "dq"), (dk, "dk")):
        turned = rope_oracle.rotate(want[name], theta, d, inverse=True)
        both = want[name + "_bound"]
        both = np.concatenate([both[..., :d // 2] + both[..., d // 2:]] * 2, -1)  # of both channels of the pair
        bad = np.abs(host(got) - turned) > both * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(turned) + 1e-6
        assert not bad.any()


def test_bad_bounds_and_refusals(fa, monkeypatch):
    torch = torch_cuda()
    lens = [50, 60]
    q, k, v = make(lens, lens, 4, 2, 64, 13)
    cu = i32(starts(lens))
    o, lse = fa.packed_forward(q, k, v, cu)
    do = _normal(q, 14)
    clean = fa.packed_backward(q, k, v, o, lse, do, cu)
    fa.fa_poll_status()
    got = fa.packed_backward(q, k, v, o, lse, do, i32([0, 50, 999]), cu)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    assert torch.equal(got[0][:50], clean[0][:50]) and not bool(got[0][50:].any())
    good = dict(q=q, k=k, v=v, o=o, lse=lse, dout=do, dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                cu_q=cu, cu_k=cu)
    for bad in (dict(dout=do[:-1]), dict(dq=good["dq"].float()), dict(dk=good["dk"][:, :1]), dict(lse=lse[:, ::2]),
                dict(cu_k=cu[:-1]), dict(dv=good["dv"][:1].expand(110, 2, 64)), dict(q=None)):
        with pytest.raises((ValueError, TypeError)):
            fa.fa_packed_bwd(**{**good, **bad})
    for bad in (dict(scale=0.0), dict(causal=7)):
        with pytest.raises(fa.FaError) as e:
            fa.fa_packed_bwd(**{**good, **bad})
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    monkeypatch.setenv("FA_TEST_FAIL_ALLOC", "1")
    with pytest.raises(fa.FaError) as e:
        fa.fa_packed_bwd(**good)
    assert e.value.status == fa.FA_ERR_NO_MEMORY
