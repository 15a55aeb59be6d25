"""Attention with a sliding window and sinks on the GPU, against the definition in 64 bits."""
import math

import pytest
import torch

import attention_forward_fa2_gb300 as fa
from attention_forward_fa2_gb300 import build as fabuild
import window_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _rand(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)


def _ok():
    rc, info = fa.check_status()
    assert rc == fa.FA_OK, (fa.strerror(rc), info)


def _dense(B, Nq, Nk, H, Hk, d, window, sinks, grad=True):
    q, k, v = _rand((B, Nq, H, d), 1), _rand((B, Nk, Hk, d), 2), _rand((B, Nk, Hk, d), 3)
    do = _rand((B, Nq, H, d), 4)
    o, lse = fa.forward_window(q, k, v, window, sinks)
    _ok()
    mask = R.visible(Nq, Nk, window, sinks, device="cuda")
    scale = 1 / math.sqrt(d)
    for b in range(B):
        o_ref, lse_ref, bound = R.forward(q[b], k[b], v[b], scale, mask)
        R.check(o[b], o_ref, bound, "o[%d]" % b)
        R.check_lse(lse[b], lse_ref, "lse[%d]" % b)
    if not grad:
        return
    grads = fa.backward_window(q, k, v, o, lse, do, window, sinks)
    _ok()
    for b in range(B):
        ref, bounds = R.backward(q[b], k[b], v[b], do[b], scale, mask)
        for name, g, r, t in zip(("dq", "dk", "dv"), grads, ref, bounds):
            R.check(g[b], r, t, "%s[%d]" % (name, b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (128, 0), (129, 130), (300, 128), (300, 300),
                                          (5000, 3)])
def test_windows_and_sinks(d, window, sinks):
    _dense(1, 700, 700, 4, 2, d, window, sinks)


@pytest.mark.parametrize("B,Nq,Nk,H,Hk,window,sinks", [
    (1, 1, 1, 1, 1, 1, 0),       # one query, one key
    (2, 1, 515, 8, 2, 40, 4),    # one query at the end of many keys
    (3, 129, 130, 2, 1, 64, 1),
    (2, 900, 300, 2, 2, 50, 5),  # two query tiles and more that see nothing, in each batch
    (2, 100, 900, 4, 1, 130, 140),
    (1, 513, 2049, 2, 2, 256, 0),  # keys older than every window: zero gradients
    (1, 40, 700, 2, 1, 20, 0),
    (2, 256, 256, 12, 3, 100, 16),
])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths_and_heads(B, Nq, Nk, H, Hk, d, window, sinks):
    _dense(B, Nq, Nk, H, Hk, d, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hk", [(6, 16, 8), (6, 8, 8), (4, 18, 6)])
@pytest.mark.parametrize("window,sinks", [(150, 0), (300, 130)])
def test_more_units_than_sms(B, H, Hk, d, window, sinks):
    """Enough tiles that units are pairs of them, and key blocks are not cut into parts."""
    _dense(B, 700, 750, H, Hk, d, window, sinks)


def test_long_sequence_many_chunks_of_the_sink_block():
    _dense(1, 6000, 6000, 2, 1, 128, 200, 4)


def test_full_window_is_the_causal_forward():
    q, k, v = _rand((2, 300, 4, 128), 1), _rand((2, 450, 2, 128), 2), _rand((2, 450, 2, 128), 3)
    o, lse = fa.forward_window(q, k, v, 1 << 40)
    oc, lsec = fa.forward_qk(q, k, v, causal=True)
    _ok()
    # Both are roundings of the same values, each within `bound` of them, and so at most
    # twice that apart (the two kernels take their reference maxima by different rules).
    for b in range(2):
        _, _, bound = R.forward(q[b], k[b], v[b], 128 ** -0.5, R.visible(300, 450, 0, 0, device="cuda"))
        R.check(o[b], oc[b].double(), 2 * bound, "o[%d]" % b)
    assert (lse - lsec).abs().max().item() <= 2 * R.LSE_TOL


LENS = [(0, 0), (1, 1), (127, 127), (0, 40), (128, 300), (129, 129), (77, 0), (513, 513), (300, 100)]


def _packed(lens, H, Hk, d, seed=0, tail=5):
    """Packed tensors with `tail` rows behind the last sequence that hold NaN."""
    cu_q = torch.tensor([0] + [a for a, _ in lens]).cumsum(0).to(torch.int32).cuda()
    cu_k = torch.tensor([0] + [b for _, b in lens]).cumsum(0).to(torch.int32).cuda()
    tq, tk = int(cu_q[-1]) + tail, int(cu_k[-1]) + tail
    out = [_rand((tq, H, d), seed + 1), _rand((tk, Hk, d), seed + 2), _rand((tk, Hk, d), seed + 3),
           _rand((tq, H, d), seed + 4)]
    for t in out:
        if tail:
            t[-tail:] = math.nan
    return out, cu_q, cu_k, max(a for a, _ in lens), max(b for _, b in lens)


def _packed_sequences(lens, H, Hk, d, window, sinks):
    (q, k, v, do), cu_q, cu_k, mq, mk = _packed(lens, H, Hk, d)
    B, mark = len(lens), 7.0
    kw = dict(cu_seqlens_q=cu_q, cu_seqlens_k=cu_k, max_seqlen_q=mq, max_seqlen_k=mk)
    out, lse = torch.full_like(q, mark), torch.full((B, H, mq), mark, device="cuda")
    fa.forward_window(q, k, v, window, sinks, out=out, lse=lse, **kw)
    grads = [torch.full_like(t, mark) for t in (q, k, v)]
    fa.backward_window(q, k, v, out, lse, do, window, sinks, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
    _ok()
    for t in (out, *grads):
        assert (t[-5:] == mark).all(), "rows behind the last sequence were written"
    for b, (n, m) in enumerate(lens):
        rq, rk = slice(int(cu_q[b]), int(cu_q[b]) + n), slice(int(cu_k[b]), int(cu_k[b]) + m)
        mask = R.visible(n, m, window, sinks, device="cuda")
        o_ref, lse_ref, bound = R.forward(q[rq], k[rk], v[rk], 1 / math.sqrt(d), mask)
        R.check(out[rq], o_ref, bound, "o[%d]" % b)
        R.check_lse(lse[b, :, :n], lse_ref, "lse[%d]" % b)
        assert (lse[b, :, n:] == mark).all()
        ref, bounds = R.backward(q[rq], k[rk], v[rk], do[rq], 1 / math.sqrt(d), mask)
        for name, g, r, t in zip(("dq", "dk", "dv"), (grads[0][rq], grads[1][rk], grads[2][rk]), ref, bounds):
            R.check(g, r, t, "%s[%d]" % (name, b))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(50, 0), (150, 130), (1000, 2)])
def test_packed_sequences(d, window, sinks):
    _packed_sequences(LENS, 4, 2, d, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(4, 2), (3, 3)])
def test_many_packed_sequences(d, H, Hk):
    _packed_sequences(LENS * 5, H, Hk, d, 150, 130)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sinks", [0, 4])
def test_one_long_and_many_short_sequences(d, sinks):
    _packed_sequences([(9, 9), (0, 30)] * 10 + [(1800, 1900)] + [(130, 130), (1, 1)] * 12, 4, 2, d, 200, sinks)


def test_gradients_are_those_of_differences():
    """Directional derivative of sum(o * dout) in 64 bits against the kernel's gradients."""
    d, n, window, sinks = 64, 200, 33, 3
    q, k, v, do = (_rand((1, n, 2, d), s) for s in range(4))
    o, lse = fa.forward_window(q, k, v, window, sinks)
    grads = fa.backward_window(q, k, v, o, lse, do, window, sinks)
    _ok()
    mask = R.visible(n, n, window, sinks, device="cuda")
    scale = 1 / math.sqrt(d)

    def loss(a, b, c):
        p, _ = R._weights(a, b, scale, mask)
        return (torch.einsum("hij,jhd->ihd", p, c) * do[0].double()).sum()
    xs = [t[0].double() for t in (q, k, v)]
    _, bounds = R.backward(q[0], k[0], v[0], do[0], scale, mask)
    for i, (g, bound) in enumerate(zip(grads, bounds)):
        u = _rand((n, 2, d), 90 + i).double()
        eps = 1e-5
        hi = [x + eps * u if j == i else x for j, x in enumerate(xs)]
        lo = [x - eps * u if j == i else x for j, x in enumerate(xs)]
        slope = ((loss(*hi) - loss(*lo)) / (2 * eps)).item()
        # Elementwise bounds summed along the direction, and the difference's own error.
        tol = (bound * u.abs()).sum().item() + 1e-4 * abs(slope) + 1e-4
        assert abs((g[0].double() * u).sum().item() - slope) <= tol


def test_dk_and_dv_repeat_exactly():
    q, k, v, do = (_rand((2, 1500, 4, 128), s) for s in range(4))
    o, lse = fa.forward_window(q, k, v, 200, 4)
    first = fa.backward_window(q, k, v, o, lse, do, 200, 4)
    again = fa.backward_window(q, k, v, o, lse, do, 200, 4)
    _ok()
    assert torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


def test_on_another_stream_and_in_a_graph():
    q, k, v, do = (_rand((1, 600, 4, 64), s) for s in range(4))
    o, lse = fa.forward_window(q, k, v, 100, 4)
    dq, dk, dv = fa.backward_window(q, k, v, o, lse, do, 100, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    fa.forward_window(q, k, v, 100, 4, out=o2, lse=lse2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    ws = torch.empty(fa.bwd_window_workspace_bytes(1, 600, 600, 4, 4, 64, 100, 4), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(t) for t in (q, k, v)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.forward_window(q, k, v, 100, 4, out=o2, lse=lse2)
        fa.backward_window(q, k, v, o2, lse2, do, 100, 4, workspace=ws, dq=outs[0], dk=outs[1], dv=outs[2])
    for t in (o2, lse2, *outs):
        t.zero_()
    graph.replay()
    _ok()
    assert torch.equal(o, o2) and torch.equal(dk, outs[1]) and torch.equal(dv, outs[2])
    _, bounds = R.backward(q[0], k[0], v[0], do[0], 1 / 8, R.visible(600, 600, 100, 4, device="cuda"))
    assert ((outs[0][0].double() - dq[0].double()).abs() <= 2 * bounds[0]).all()


def test_bad_lengths_are_reported_and_touch_nothing():
    (q, k, v, do), cu_q, cu_k, mq, mk = _packed([(100, 100), (200, 200)], 2, 2, 64, tail=0)
    B = 2
    for bad_q, bad_k in (([0, 100, 301], None), (None, [0, 100, 301]), ([0, 200, 100], None), (None, [0, -4, 200])):
        cq = cu_q if bad_q is None else torch.tensor(bad_q, dtype=torch.int32, device="cuda")
        ck = cu_k if bad_k is None else torch.tensor(bad_k, dtype=torch.int32, device="cuda")
        kw = dict(cu_seqlens_q=cq, cu_seqlens_k=ck, max_seqlen_q=mq, max_seqlen_k=mk)
        o, lse = torch.zeros_like(q), torch.zeros((B, 2, mq), device="cuda")
        fa.forward_window(q, k, v, 50, 2, out=o, lse=lse, **kw)
        assert fa.check_status()[0] == fa.FA_ERR_BAD_SEQLENS
        fa.backward_window(q, k, v, o, lse, do, 50, 2, **kw)
        assert fa.check_status()[0] == fa.FA_ERR_BAD_SEQLENS


def test_refusals():
    q, k = _rand((1, 8, 4, 64), 1), _rand((1, 8, 2, 64), 2)
    o, lse = fa.forward_window(q, k, k, 4)
    with pytest.raises(fa.FaError):
        fa.forward_window(q, k, k, 0)
    with pytest.raises(fa.FaError):
        fa.forward_window(q, k, k, 4, -1)
    with pytest.raises(ValueError):
        fa.forward_window(q.transpose(1, 2), k, k, 4)
    with pytest.raises(TypeError):
        fa.forward_window(q.half(), k, k, 4)
    with pytest.raises(ValueError):
        fa.forward_window(q, k, k[:, :7].contiguous(), 4)
    with pytest.raises(ValueError):
        fa.forward_window(q[0], k[0], k[0], 4, cu_seqlens_q=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        fa.backward_window(q, k, k, o, lse, q, 4, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        fa.backward_window(q, k, k, o, lse[:, :, :4].contiguous(), q, 4)
    _ok()
