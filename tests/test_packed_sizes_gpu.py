"""Packed sequences where sizes leave the ordinary: more sequences and blocks than a CTA plans in shared memory, one
sequence over all of the device, offsets past 32 bits; calls side by side, through either caller, and one after another as
a server makes them.  Bounds are packed_util's."""

import threading

import numpy as np
import pytest

from gpu_util import ensure_built, host, torch_cuda
from oracle import packed as oracle
from oracle import rope as rope_oracle
from packed_util import check_forward, i32, make, scale_of, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    torch_cuda()
    return ensure_built()


def _check(fa, lq, lk, H, Hkv, d, causal, seed, used=None, prefix=0, pad=0):
    q, k, v = make(lq, lk, H, Hkv, d, seed, pad)
    cq, ck = starts(lq), starts(lk)
    args = (i32(cq), i32(ck), None if used is None else i32(used), causal)
    pre = None
    if prefix:
        _, kp, vp = make([1], [prefix], H, Hkv, d, seed + 1)
        pre = (host(kp), host(vp))
        o, lse = fa.prefix_forward(q, kp, vp, k, v, *args)
    else:
        o, lse = fa.packed_forward(q, k, v, *args)
    assert fa.fa_poll_status() == fa.FA_OK
    want = oracle.forward(host(q), host(k), host(v), cq, ck, scale_of(d), causal, used, pre)
    check_forward(o, lse, want, d, slice(cq[0], cq[-1]))


@pytest.mark.parametrize("prefix", [0, 400])
@pytest.mark.parametrize("B,H,most", [(3000, 2, 4), (1100, 128, 4), (700, 128, 6)])
def test_many_sequences(fa, B, H, most, prefix):
    """Blocks of two tokens (128 heads) or of many: over 1024 sequences, small blocks, whole blocks, and of both together."""
    g = np.random.default_rng(B + prefix)
    lq = g.integers(0, most, B).tolist()
    lk = [n + int(g.integers(0, 30)) for n in lq]
    _check(fa, lq, lk, H, 1, 64, "bottom_right", 50, prefix=prefix)


def test_many_sequences_backward_is_that_of_each(fa):
    """Over 1024 sequences: dq, dk, dv of the first, of one in the middle and of the last are those of calls of their own."""
    torch = torch_cuda()
    g = np.random.default_rng(5)
    lens = g.integers(1, 40, 1300).tolist()
    q, k, v = make(lens, lens, 2, 1, 64, 51)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(52)).to(torch.bfloat16).cuda()
    cu = starts(lens)
    o, lse = fa.packed_forward(q, k, v, i32(cu), causal=True)
    grads = fa.packed_backward(q, k, v, o, lse, do, i32(cu), causal=True)
    for b in (0, 1, 650, 1299):
        part = slice(cu[b], cu[b + 1])
        one = [x[part].contiguous() for x in (q, k, v, o, do)]
        alone = fa.packed_backward(*one[:4], lse[:, part].contiguous(), one[4], i32([0, lens[b]]), causal=True)
        assert all(torch.equal(x[part], y) for x, y in zip(grads, alone))


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("H,Hkv,n", [(8, 1, 70000), (3, 3, 20011)])
def test_one_sequence_over_the_whole_device(fa, d, H, Hkv, n):
    """Hundreds of parts of one row are merged."""
    _check(fa, [1], [n], H, Hkv, d, "none", 53)
    _check(fa, [2], [3], H, Hkv, d, "bottom_right", 54, prefix=n)


def test_answers_behind_a_long_prefix(fa):
    _check(fa, [1] * 24, [(5 * i) % 60 for i in range(24)], 8, 1, 128, "bottom_right", 55, prefix=30000)


def test_offsets_past_32_bits(fa):
    """Keys and queries whose elements lie past 2^31 of them; nothing else of the tensors is read or written."""
    torch = torch_cuda()
    room, H, Hkv, d = 9_000_000, 4, 2, 128
    used, lq = [300, 700], [5, 40]
    k, v = (torch.empty(room, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() > 2 ** 31
    q, ks, vs = make(lq, used, H, Hkv, d, 56)
    cu_k = [0, room - 1000, room]
    for big, small in ((k, ks), (v, vs)):
        big[:300] = small[:300]
        big[room - 1000:room - 300] = small[300:]
    o, lse = fa.packed_forward(q, k, v, i32(starts(lq)), i32(cu_k), i32(used), "bottom_right")
    assert fa.fa_poll_status() == fa.FA_OK
    want = oracle.forward(host(q), host(ks), host(vs), starts(lq), starts(used), scale_of(d), "bottom_right")
    check_forward(o, lse, want, d)
    del k, v
    T, H, n = 140_000, 128, 150
    far_q = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda")
    far_o, far_l = torch.zeros_like(far_q), torch.zeros(H, T, device="cuda")
    assert far_q.numel() > 2 ** 31
    q, ks, vs = make([n], [n], H, 8, d, 57)
    far_q[T - n:] = q
    fa.fa_packed_fwd(far_q, ks, vs, far_o, far_l, i32([T - n, T]), i32([0, n]), causal=True)
    assert fa.fa_poll_status() == fa.FA_OK
    want = oracle.forward(host(q), host(ks), host(vs), [0, n], [0, n], scale_of(d), "top_left")
    check_forward(far_o[T - n:], far_l[:, T - n:].contiguous(), want, d)
    assert not bool(far_o[:1000].any()) and not bool(far_o[T - n - 1000:T - n].any())


def test_calls_side_by_side(fa):
    """Threads of the host, each on a stream of its own: the bits of calls one after another."""
    torch = torch_cuda()
    cases = []
    for i, (lens, H, Hkv, d) in enumerate((([700, 33, 900], 8, 2, 128), ([64] * 40, 4, 4, 64), ([1, 1, 2000], 6, 3, 96))):
        q, k, v = make(lens, lens, H, Hkv, d, 60 + i)
        cu = i32(starts(lens))
        do = torch.randn(q.shape, generator=torch.Generator().manual_seed(70 + i)).to(torch.bfloat16).cuda()

        def call(q=q, k=k, v=v, cu=cu, do=do):
            o, lse = fa.packed_forward(q, k, v, cu, causal=True)
            return [o, lse, *fa.packed_backward(q, k, v, o, lse, do, cu, causal=True)]

        cases.append((call, call()))
    torch.cuda.synchronize()
    wrong = []

    def work(call, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = call()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append("bits")
        except Exception as e:  # noqa: BLE001 (reported by the test's own thread)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_either_caller(fa, monkeypatch):
    """The native caller, and ctypes where it was not built: the same bits, the same refusals."""
    torch = torch_cuda()
    from exact_attention_92_gb300 import _binding

    lens, H, Hkv, d = [300, 41], 4, 2, 64
    q, k, v = make(lens, lens, H, Hkv, d, 80)
    _, kp, vp = make([1], [200], H, Hkv, d, 81)
    cu, ph = i32(starts(lens)), fa.rope_phases(fa.rope_frequencies(d))
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(82)).to(torch.bfloat16).cuda()

    def everything():
        qr, kr = fa.rope(q, k, ph)
        o, lse = fa.packed_forward(qr, kr, v, cu, causal=True)
        grads = fa.packed_backward(qr, kr, v, o, lse, do, cu, causal=True)
        refused = []
        for bad in (lambda: fa.packed_forward(q, k, v, cu, scale=-1.0), lambda: fa.packed_forward(q, k, v, cu.long()),
                    lambda: fa.packed_forward(q, k[:, :1].expand(341, 2, 64), v, cu), lambda: fa.rope(q.float(), k, ph),
                    lambda: fa.prefix_forward(q, kp[:0], vp[:0], k, v, cu),
                    lambda: fa.packed_backward(q, k, v, o, lse[:, :9], do, cu)):
            with pytest.raises((fa.FaError, ValueError, TypeError)) as e:
                bad()
            refused.append((type(e.value), getattr(e.value, "status", None)))
        return [qr, kr, o, lse, *grads, *fa.prefix_forward(qr, kp, vp, kr, v, cu)], refused

    first = everything()
    monkeypatch.setattr(_binding, "_packed", False)
    second = everything()
    assert all(torch.equal(a, b) for a, b in zip(first[0], second[0]))
    assert first[1] == second[1]


def test_steps_of_a_server(fa):
    """A prompt behind a shared document and then steps: new rows are turned, put into the cache and answered."""
    torch = torch_cuda()
    P, H, Hkv, d, room = 300, 8, 2, 128, 256
    B = 3
    prompts = [100, 7, 150]
    _, kp, vp = make([1], [P], H, Hkv, d, 90)
    cache_k, cache_v = (torch.full((B * room, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    freq = fa.rope_frequencies(d)
    ph = fa.rope_phases(freq)
    used = [0] * B
    for step in range(4):
        lq = prompts if step == 0 else [1] * B
        q, k, v = make(lq, lq, H, Hkv, d, 91 + step)
        pos = [P + used[b] + i for b in range(B) for i in range(lq[b])]
        qr, kr = fa.rope(q, k, ph, positions=i32(pos))
        theta = rope_oracle.angles(np.asarray(pos), freq)[:, None]
        for got, x in ((qr, q), (kr, k)):
            want = rope_oracle.rotate(host(x), theta, d)
            assert bool((np.abs(host(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(host(x)).max()).all())
        at = [b * room + used[b] + i for b in range(B) for i in range(lq[b])]
        cache_k[at], cache_v[at] = kr, v
        used = [u + n for u, n in zip(used, lq)]
        o, lse = fa.prefix_forward(qr, kp, vp, cache_k, cache_v, i32(starts(lq)), i32(starts([room] * B)), i32(used),
                                   "bottom_right")
        assert fa.fa_poll_status() == fa.FA_OK
        clean = [host(torch.nan_to_num(x)) for x in (cache_k, cache_v)]
        want = oracle.forward(host(qr), *clean, starts(lq), starts([room] * B), scale_of(d), "bottom_right", used,
                              (host(kp), host(vp)))
        check_forward(o, lse, want, d)


@pytest.mark.parametrize("causal", ["none", "top_left", "bottom_right"])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 2, 128), (3, 1, 96)])
def test_ragged_lengths_with_a_plan(fa, causal, H, Hkv, d):
    """(Room for more tokens than there are: calls of few keys go without a plan.)"""
    lens = [257, 1, 128, 0, 127, 300, 1000, 129, 2]
    _check(fa, lens, lens, H, Hkv, d, causal, 100, pad=4000)
    _check(fa, [40, 0, 1, 300, 1], [1700, 5, 0, 130, 900], H, Hkv, d, causal, 101, pad=4000)


@pytest.mark.parametrize("causal", ["none", "top_left", "bottom_right"])
@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 64), (8, 2, 128), (3, 1, 96)])
@pytest.mark.parametrize("prefix", [0, 300])
def test_small_blocks_halved_between_warpgroups(fa, causal, H, Hkv, d, prefix):
    """Few units over up to 12 key tiles, without a plan; of one tile, or none, the second half is empty.  Whole blocks ahead
    of them, whose rows are still being stored."""
    block = 2 * (128 // (H // Hkv))
    _check(fa, [1, 3, 1, 0, 2, 1], [700, 90, 0, 5, 129, 257], H, Hkv, d, causal, 110, prefix=prefix)
    _check(fa, [2 * block + 1, 7], [2 * block + 1, 600], H, Hkv, d, causal, 111, prefix=prefix)
    _check(fa, [1], [1500], H, Hkv, d, causal, 112)


@pytest.mark.parametrize("prefix", [0, 500])
def test_nan_stays_in_its_sequence_with_a_plan(fa, prefix):
    torch = torch_cuda()
    lens = [700, 70, 1300, 29] + [3] * 40
    q, k, v = make(lens, lens, 4, 2, 128, 102, pad=5)
    _, kp, vp = make([1], [500], 4, 2, 128, 103)
    cu = i32(starts(lens))

    def call():
        return fa.prefix_forward(q, kp, vp, k, v, cu, causal=True) if prefix else fa.packed_forward(q, k, v, cu, causal=True)

    clean, clean_l = call()
    for x in (q, k, v):
        x[700:770] = float("nan")
        x[720:760] = float("inf")
        x[sum(lens):] = float("nan")
    o, lse = call()
    keep = [*range(700), *range(770, sum(lens))]
    assert torch.equal(o[keep], clean[keep]) and torch.equal(lse[:, keep], clean_l[:, keep])


@pytest.mark.parametrize("B", [7, 41, 1501])
def test_bounds_that_go_back_are_skipped(fa, B):
    """0, T, 0, T, ...: the sequences from the second on are out of order and skipped, so that there are never more blocks
    than rows; the first has what it has alone."""
    torch = torch_cuda()
    T, H, Hkv, d = 600, 2, 1, 64
    q, k, v = make([T], [T], H, Hkv, d, 104)
    do = torch.randn(q.shape, generator=torch.Generator().manual_seed(105)).to(torch.bfloat16).cuda()
    good, bad = i32([0, T]), i32([T * (b % 2) for b in range(B + 1)])
    _, kp, vp = make([1], [300], H, Hkv, d, 106)
    o, lse = fa.packed_forward(q, k, v, good, causal=True)
    want = fa.packed_backward(q, k, v, o, lse, do, good, causal=True)
    behind, _ = fa.prefix_forward(q, kp, vp, k, v, good, causal=True)
    assert fa.fa_poll_status() == fa.FA_OK
    got, got_l = fa.packed_forward(q, k, v, bad, causal=True)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    scale = float(o.abs().max())
    assert float((got.float() - o.float()).abs().max()) <= 2.0 ** -6 * scale  # (cut elsewhere, or not)
    assert torch.allclose(got_l, lse, rtol=1e-5, atol=1e-5)
    grads = fa.packed_backward(q, k, v, o, lse, do, bad, causal=True)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    got, _ = fa.prefix_forward(q, kp, vp, k, v, bad, causal=True)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    assert float((got.float() - behind.float()).abs().max()) <= 2.0 ** -6 * float(behind.abs().max())
    # Only the queries, or only the keys, go back.
    long_k = i32([0, T] + [T] * (B - 1))
    fa.packed_backward(q, k, v, o, lse, do, bad, long_k, causal=True)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX
    fa.packed_backward(q, k, v, o, lse, do, long_k, bad, causal=True)
    assert fa.fa_poll_status() == fa.FA_ERR_BAD_INDEX


def test_graphs_with_a_plan(fa):
    """Plan, clusters and merge (and the join behind a prefix) captured: the eager call's bits, the lengths of the replay, and
    two graphs replayed in turn on two streams."""
    torch = torch_cuda()
    H, Hkv, d, room = 8, 2, 128, 9000
    q, k, v = make([room], [room], H, Hkv, d, 120)
    _, kp, vp = make([1], [3000], H, Hkv, d, 121)
    first, second = [700, 90, 1300, 0, 33] + [1] * 40, [10, 1900, 0, 200, 13] + [2] * 40
    cu = i32(starts(first))

    def outputs():
        return torch.zeros_like(q), torch.zeros(H, room, device="cuda")

    calls = [lambda o, l: fa.fa_packed_fwd(q, k, v, o, l, cu, cu, causal=True),
             lambda o, l: fa.fa_prefix_fwd(q, kp, vp, k, v, o, l, cu, cu, causal=True)]
    eager = [outputs() for _ in calls]
    for call, out in zip(calls, eager):
        call(*out)
    graphs, held = [], []
    for call in calls:
        out, g = outputs(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(*out)
        graphs.append(g)
        held.append(out)
    streams = [torch.cuda.Stream() for _ in graphs]
    for lens in (first, second, first):
        cu.copy_(i32(starts(lens)))
        for out in (*held, *eager):
            for x in out:
                x.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for call, out in zip(calls, eager):
            call(*out)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for x, y in zip(held, eager) for a, b in zip(x, y))
    assert fa.fa_poll_status() == fa.FA_OK
