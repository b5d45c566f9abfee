"""Rotary positions on the GPU against the oracle in fp64.

Tolerance: the result is rounded once to bf16 (2^-8 relative).  Ahead of that, the angle is off by at most 2^-24 of a
half turn (fp32 of the upper 32 bits) and 2^-31 for the lower ones: 2e-7 radians; sincospif is within 2 units of the last
place, the two products and the sum round three times: together below 1e-6 of (|a| + |b|) * mscale.
"""

import numpy as np
import pytest

from oracle import rope as oracle

from gpu_util import ensure_built, host, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    torch_cuda()
    return ensure_built()


def _normal(shape, seed):
    torch = torch_cuda()
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _check(y, x, theta, rot, inter, mscale, inverse):
    """y, x [..., d] with theta broadcast against them."""
    x64 = host(x)
    want = oracle.rotate(x64, theta, rot, inter, mscale, inverse)
    size = np.zeros_like(x64)
    lo, hi = (np.s_[..., 0:rot:2], np.s_[..., 1:rot:2]) if inter else (np.s_[..., :rot // 2], np.s_[..., rot // 2:rot])
    size[lo] = size[hi] = np.abs(x64[lo]) + np.abs(x64[hi])
    err = np.abs(host(y) - want)
    over = float((err - np.abs(want) * 2.0 ** -8 - size * mscale * 1e-6).max())
    assert over <= 0.0
    same = np.array_equal(host(y)[..., rot:], x64[..., rot:])
    assert same


CASES = [  # d, rot, interleaved, H, Hkv
    (64, 64, False, 4, 2), (64, 64, True, 3, 1), (128, 128, False, 5, 5), (128, 32, True, 9, 3), (96, 64, True, 2, 1),
    (96, 96, False, 7, 7), (96, 24, False, 2, 2), (96, 24, True, 2, 2), (128, 2, False, 3, 1), (64, 6, True, 1, 1),
    (64, 62, False, 2, 1), (256, 128, False, 2, 2), (256, 256, True, 1, 1),
]


@pytest.mark.parametrize("d,rot,inter,H,Hkv", CASES)
@pytest.mark.parametrize("N", [1, 77])
def test_dense_against_oracle(fa, d, rot, inter, H, Hkv, N):
    torch = torch_cuda()
    B = 3
    q, k = _normal((B, H, N, d), 1), _normal((B, Hkv, N, d), 2)
    freq = fa.rope_frequencies(rot)
    pos = torch.randint(0, 1 << 20, (B, N), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    pos[0, 0] = 0
    pos[1, -1] = 2 ** 31 - 1
    pos[2, 0] = -5
    th = oracle.angles(pos.numpy(), freq)[:, None]
    ph = fa.rope_phases(freq)
    for inverse, ms in ((False, 1.0), (True, 1.25)):
        yq, yk = fa.rope(q, k, ph, positions=pos.cuda(), interleaved=inter, mscale=ms, inverse=inverse)
        _check(yq, q, th, rot, inter, ms, inverse)
        _check(yk, k, th, rot, inter, ms, inverse)


def test_positions_from_start_and_from_nothing(fa):
    torch = torch_cuda()
    q, k = _normal((4, 2, 9, 64), 1), _normal((4, 1, 9, 64), 2)
    freq = fa.rope_frequencies(64, base=500000.0)
    ph = fa.rope_phases(freq)
    start = torch.tensor([0, 7, 2 ** 31 - 1, 100000], dtype=torch.int32)
    pos = start.numpy().astype(np.int64)[:, None] + np.arange(9)
    yq, yk = fa.rope(q, k, ph, start=start.cuda())
    _check(yq, q, oracle.angles(pos, freq)[:, None], 64, False, 1.0, False)
    _check(yk, k, oracle.angles(pos, freq)[:, None], 64, False, 1.0, False)
    yq, none = fa.rope(q, None, ph)
    assert none is None
    _check(yq, q, oracle.angles(np.broadcast_to(np.arange(9), (4, 9)), freq)[:, None], 64, False, 1.0, False)


@pytest.mark.parametrize("T", [1, 1000, 20011])
def test_packed_slices_of_a_fused_projection(fa, T):
    """q and k lie inside [T, H + 2 Hkv, d]; out of place, and in place with the
    values beside them untouched."""
    torch = torch_cuda()
    H, Hkv, d, rot = 6, 2, 128, 96
    fused = _normal((T, H + 2 * Hkv, d), 4)
    keep = fused.clone()
    freq = torch.tensor(fa.rope_frequencies(rot, scaling="by_parts", factor=4.0, original=256))
    ph = fa.rope_phases(freq)
    freq = freq.double().tolist()  # what the call was given: the frequencies in fp32
    pos = (torch.arange(T) * 7 % 1001).to(torch.int32)
    th = oracle.angles(pos.numpy(), freq)[:, None]
    q, k = fused[:, :H], fused[:, H:H + Hkv]
    yq, yk = fa.rope(q, k, ph, positions=pos.cuda())
    _check(yq, q, th, rot, False, 1.0, False)
    _check(yk, k, th, rot, False, 1.0, False)
    assert torch.equal(fused, keep)
    fa.fa_rope(q, k, q, k, ph, positions=pos.cuda())
    assert torch.equal(fused[:, :H], yq) and torch.equal(fused[:, H:H + Hkv], yk)
    assert torch.equal(fused[:, H + Hkv:], keep[:, H + Hkv:])


def test_heads_by_tokens_layout(fa):
    """[heads, tokens, d] seen as [tokens, heads, d]."""
    torch = torch_cuda()
    x = _normal((3, 50, 64), 5)
    ph = fa.rope_phases(fa.rope_frequencies(64))
    out = torch.zeros_like(x)
    fa.fa_rope(x.transpose(0, 1), None, out.transpose(0, 1), None, ph)
    want, _ = fa.rope(x[None], None, ph)
    assert torch.equal(out, want[0])


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(fa, inter):
    """<g, R x> = <R^T g, x>, and R^T g against differences of <g, R x>.  Both
    sides sum 64 products whose factors were rounded to bf16 once: each off by
    2^-8 of its size."""
    torch = torch_cuda()
    x, g = _normal((1, 2, 5, 64), 6), _normal((1, 2, 5, 64), 7)
    ph = fa.rope_phases(fa.rope_frequencies(64))
    y, _ = fa.rope(x, None, ph, interleaved=inter, mscale=1.5)
    dx, _ = fa.rope(g, None, ph, interleaved=inter, mscale=1.5, inverse=True)
    a, b = host(g) * host(y), host(dx) * host(x)
    assert abs(a.sum() - b.sum()) <= 2.0 ** -8 * (np.abs(a).sum() + np.abs(b).sum())
    for at in ((0, 0, 0, 3), (0, 1, 4, 40), (0, 1, 2, 63)):
        x2 = x.clone()
        x2[at] += 4.0
        y2, _ = fa.rope(x2, None, ph, interleaved=inter, mscale=1.5)
        diff = (host(g) * (host(y2) - host(y))).sum() / (host(x2)[at] - host(x)[at])
        changed = np.abs(host(y2) - host(y)) > 0
        size = (np.abs(host(g)) * (np.abs(host(y2)) + np.abs(host(y))) * changed).sum() / 4.0
        assert abs(diff - host(dx)[at]) <= 2.0 ** -8 * (size * 1.1 + abs(host(dx)[at])) + 1e-5


def test_infinities_stay_in_their_pairs(fa):
    torch = torch_cuda()
    x = _normal((1, 1, 4, 64), 8)
    ph = fa.rope_phases(fa.rope_frequencies(32))
    clean, _ = fa.rope(x, None, ph)
    x[0, 0, 1, 3] = float("inf")
    x[0, 0, 2, 40] = float("nan")  # passed through
    y, _ = fa.rope(x, None, ph)
    bad = ~torch.isfinite(y)
    assert bad[0, 0, 1, 3] and bad[0, 0, 1, 19] and bad[0, 0, 2, 40] and int(bad.sum()) == 3
    assert torch.equal(y[~bad], clean[~bad])


def test_streams_and_graphs(fa):
    torch = torch_cuda()
    x = _normal((2, 4, 33, 128), 9)
    ph = fa.rope_phases(fa.rope_frequencies(128))
    start = torch.tensor([3, 4], dtype=torch.int32, device="cuda")
    want, _ = fa.rope(x, None, ph, start=start)
    s = torch.cuda.Stream()
    out = torch.zeros_like(x)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.fa_rope(x, None, out, None, ph, start=start)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    fa.fa_rope(x, None, out, None, ph, start=start, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fa_rope(x, None, out, None, ph, start=start)
    start += 5
    graph.replay()
    torch.cuda.synchronize()
    want, _ = fa.rope(x, None, ph, start=start)
    assert torch.equal(out, want)
    before = fa.fa_launch_count(fa.FA_KERNEL_ROPE)
    fa.rope(x, x, ph)
    assert fa.fa_launch_count(fa.FA_KERNEL_ROPE) == before + 1


def test_refusals(fa):
    torch = torch_cuda()
    x = _normal((2, 4, 8, 64), 10)
    ph = fa.rope_phases(fa.rope_frequencies(64))
    y = torch.empty_like(x)
    for bad in (dict(q=x.float()), dict(q=x.cpu()), dict(q=x[0, 0]), dict(q_out=y[:, :2]), dict(k=x[:1]),
                dict(q=x[..., ::2], q_out=y[..., ::2]), dict(phases=ph.int()), dict(phases=ph.cpu()),
                dict(positions=torch.zeros(2, 7, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(2, 8, dtype=torch.int64, device="cuda")),
                dict(start=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(k=None),
                dict(q_out=y[:, :1].expand(2, 4, 8, 64))):
        a = dict(q=x, k=x, q_out=y, k_out=torch.empty_like(x), phases=ph)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            fa.fa_rope(**a)
    for bad in (dict(mscale=float("nan")), dict(phases=torch.cat([ph, ph])), dict(phases=ph[:0])):
        a = dict(q=x, k=None, q_out=y, k_out=None, phases=ph)
        a.update(bad)
        with pytest.raises(fa.FaError) as e:
            fa.fa_rope(**a)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    odd = torch.empty(x.numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view(x.shape)
    with pytest.raises(fa.FaError):
        fa.fa_rope(odd, None, y, None, ph)
    assert fa.fa_poll_status() == fa.FA_OK
