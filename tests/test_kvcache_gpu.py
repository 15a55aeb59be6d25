"""The paged e4m3 cache on the GPU: what the append writes, and attention over it, against
plain computations in 64 bits.

Roundings counted (half a step, relative): e4m3 2^-4 of a value, 2^-10 of its scale below
the smallest normal; bf16 2^-8; f16 2^-11."""
import math

import pytest
import torch

import attention_forward_fa2_gb300 as fa
from attention_forward_fa2_gb300 import build as fabuild
import window_ref as R

pytestmark = pytest.mark.gpu
F16 = 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _built():
    fabuild.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(shape, seed):
    return torch.randn(shape, device="cuda", generator=_gen(seed)).to(torch.bfloat16)


def _status(want=fa.FA_OK):
    rc, info = fa.check_status()
    assert rc == want, (fa.strerror(rc), info)


def _e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def _tables(n, rot):
    half = rot // 2
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64, device="cuda") / half)
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, inter):
    """x [n, heads, d] in 64 bits; cos, sin [n, rot / 2]."""
    half = cos.shape[1]
    at = torch.arange(half, device=x.device)
    a, b = (2 * at, 2 * at + 1) if inter else (at, at + half)
    y = x.double().clone()
    c, s = cos.double()[:, None], sin.double()[:, None]
    y[..., a] = x[..., a].double() * c - x[..., b].double() * s
    y[..., b] = x[..., b].double() * c + x[..., a].double() * s
    return y


def _layout(lens, page, seed, spare=3):
    """A page table in shuffled order, -1 behind each sequence's last page."""
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need) + spare, device="cuda", generator=_gen(seed)).to(torch.int32)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, sum(need) + spare


def _noise_cache(pages, Hk, page, d, seed):
    """Pages that were used before: any code (NaN among them), scales of NaN."""
    c = fa.KvCache.empty(pages, page, Hk, d)
    for t in (c.k8, c.v8):
        t.copy_(torch.randint(0, 256, t.shape, device="cuda", generator=_gen(seed), dtype=torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.fill_(math.nan)
    return c


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check_page(codes, scale, old_codes, old_scale, s0, new, what):
    """One page and head: codes [page, d] after, `new` [m, d] exact values at slots s0 .."""
    m = new.shape[0]
    fin = new[torch.isfinite(new)].abs()
    amax = fin.max().item() if fin.numel() else 0.0
    s = float(scale)
    e = math.log2(s)
    assert e == int(e) and e >= -64, what
    if s0 and s == float(old_scale):
        assert amax <= 448 * s * (1 + 1e-6), what
    else:
        assert amax <= 448 * s * (1 + 1e-6) and (e == -64 or amax >= 224 * s * (1 - 1e-6)), what
    got = _e4m3(codes[s0:s0 + m]) * s
    err = (got - new).abs()
    bound = new.abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10 * s + 2.0 ** -22 * amax
    fine = torch.isfinite(new)
    assert (err <= bound)[fine].all(), what
    assert torch.isnan(got[torch.isnan(new)]).all(), what
    inf = torch.isinf(new)
    assert torch.equal(got[inf], 448.0 * s * torch.sign(new[inf])), what
    if s0:
        want = (_e4m3(old_codes[:s0]) * (float(old_scale) / s)).float().to(torch.float8_e4m3fn).double()
        assert torch.equal(_e4m3(codes[:s0]), want), what
    assert torch.equal(codes[s0 + m:], old_codes[s0 + m:]), what + ": slots behind the last token"


def _append_and_check(old, new, Hk, H, d, page, rot, inter, packed, seed=0, loud=False, fused=True, values=None):
    """Append behind `old` cached tokens and check every page, head and query."""
    B = len(old)
    table, pages = _layout([a + n for a, n in zip(old, new)], page, seed)
    cache = _noise_cache(pages, Hk, page, d, seed + 1)
    first = [table[b, a // page].item() if a % page else -1 for b, a in enumerate(old)]
    for f in first:
        if f >= 0:  # begun pages hold values under a scale of their own
            cache.k8[f] = (torch.randn(cache.k8[f].shape, device="cuda", generator=_gen(seed + 2)) * 100).to(
                torch.float8_e4m3fn).view(torch.uint8)
            cache.v8[f] = cache.k8[f].flip(0)
            cache.k_scale[f] = 2.0 ** (-12 if loud else 3)
            cache.v_scale[f] = 2.0 ** -7
    T = sum(new)
    x = _rand((T, H + 2 * Hk, d), seed + 3)
    if values is not None:
        values(x)
    q, k, v = (x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]) if fused else (
        x[:, :H].contiguous(), x[:, H:H + Hk].contiguous(), x[:, H + Hk:].contiguous())
    cos, sin = _tables(max(a + n for a, n in zip(old, new)), rot) if rot else (None, None)
    before = [t.clone() for t in (cache.k8, cache.v8, cache.k_scale, cache.v_scale)]
    kw = dict(q=q if H else None, cos=cos, sin=sin, interleaved=inter)
    cu = torch.tensor([0] + new).cumsum(0).tolist()
    if packed:
        out = fa.append_kvcache(cache, k, v, table, _ints(old), cu_seqlens=_ints(cu), max_seqlen=max(new), **kw)
    else:
        shape = lambda t: t.unflatten(0, (B, new[0]))  # noqa: E731
        kw["q"] = shape(q) if H else None
        out = fa.append_kvcache(cache, shape(k), shape(v), table, _ints(old), **kw)
        out = out.flatten(0, 1) if H else None
    _status()
    touched = set()
    for b in range(B):
        r = slice(cu[b], cu[b + 1])
        pos = torch.arange(old[b], old[b] + new[b], device="cuda")
        kk, qq = k[r].double(), q[r].double()
        if rot:
            kk, qq = _rotate(k[r], cos[pos], sin[pos], inter), _rotate(q[r], cos[pos], sin[pos], inter)
        if H:
            bound = R.BF16 * qq.abs() + 2.0 ** -22 * q[r].double().abs().amax(-1, keepdim=True)
            fine = torch.isfinite(qq)
            assert ((out[r].double() - qq).abs() <= bound)[fine].all()
        for pg in range(old[b] // page, -(-(old[b] + new[b]) // page)):
            s0, s1 = max(old[b] - pg * page, 0), min(old[b] + new[b] - pg * page, page)
            if s1 <= s0:
                continue
            i = int(table[b, pg])
            touched.add(i)
            t0 = pg * page + s0 - old[b]
            for h in range(Hk):
                for name, exact, c, s, oc, os_ in (("k", kk, cache.k8, cache.k_scale, before[0], before[2]),
                                                   ("v", v[r].double(), cache.v8, cache.v_scale, before[1], before[3])):
                    _check_page(c[i, h], s[i, h], oc[i, h], os_[i, h], s0, exact[t0:t0 + s1 - s0, h],
                                "%s of page %d head %d of sequence %d" % (name, pg, h, b))
    rest = [i for i in range(pages) if i not in touched]
    for t, o in zip((cache.k8, cache.v8), before[:2]):
        assert torch.equal(t[rest], o[rest]), "pages without new tokens were written"


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 16, True), (64, 48, False), (128, 128, False),
                                         (128, 96, True), (128, 80, False), (128, 0, False)])
def test_append_single_tokens(page, d, rot, inter):
    _append_and_check([0, 1, page - 1, page, 3 * page + 5], [1] * 5, 2, 5, d, page, rot, inter, False)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [3, 7, 20, 50, 200])
def test_append_several(page, d, n):
    _append_and_check([0, 5, page + 3, 2 * page], [n] * 4, 3, 6, d, page, d, n % 2 == 0, False, loud=True)


@pytest.mark.parametrize("d,page,inter", [(64, 32, False), (128, 64, True), (128, 128, False)])
def test_append_packed(d, page, inter):
    _append_and_check([0, 17, 64, 0, 130, 5], [300, 0, 1, 129, 64, 33], 2, 4, d, page, 64, inter, True)


def test_append_without_queries_or_fusion():
    _append_and_check([3, 40], [5, 5], 1, 0, 128, 16, 128, False, False, fused=False)


def test_append_infinities_and_nan():
    def values(x):
        x[0, :, 3] = math.inf
        x[1, :, 70] = -math.inf
        x[2, 5, 9] = math.nan
        x[3] = 0.0
        x[4] = 1e-30
    _append_and_check([0, 9], [3, 3], 2, 4, 128, 16, 0, False, False, values=values)


def test_append_far_positions_and_in_place():
    """Positions past 2^17, and q rotated in place."""
    page, d, old = 128, 128, 140_001
    table = _ints([[0] * (old // page) + [2, 1]])
    cache = _noise_cache(3, 1, page, d, 5)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    cos, sin = _tables(old + 40, d)
    q, k = _rand((1, 40, 3, d), 1), _rand((1, 40, 1, d), 2)
    q0 = q.clone()
    out = fa.append_kvcache(cache, k, k, table, _ints([old]), q=q, cos=cos, sin=sin, q_out=q)
    _status()
    assert out.data_ptr() == q.data_ptr()
    want = _rotate(q0[0], cos[old:old + 40], sin[old:old + 40], False)
    assert ((q[0].double() - want).abs() <= R.BF16 * want.abs() + 2.0 ** -20).all()


def test_append_reports_what_does_not_fit():
    cache = _noise_cache(4, 2, 16, 64, 1)
    before = cache.k8.clone()
    k = _rand((2, 5, 2, 64), 1)
    cos, sin = _tables(40, 64)
    for table, lens, pages_ok, code in (
            ([[0, 1], [2, 3]], [30, 0], 2, fa.FA_ERR_BAD_SEQLENS),    # past the table
            ([[0, 1], [2, 3]], [-1, 0], 2, fa.FA_ERR_BAD_SEQLENS),
            ([[0, 4], [2, 3]], [20, 0], 2, fa.FA_ERR_BAD_PAGE),
            ([[0, -1], [2, 3]], [16, 0], 2, fa.FA_ERR_BAD_PAGE)):
        fa.append_kvcache(cache, k, k, _ints(table), _ints(lens))
        _status(code)
        assert torch.equal(cache.k8[[0, 1, 3]], before[[0, 1, 3]])  # only sequence 1's page was written
    fa.append_kvcache(cache, k, k, _ints([[0, 1, 0], [2, 3, 0]]), _ints([36, 0]), cos=cos, sin=sin)  # past the tables
    _status(fa.FA_ERR_BAD_SEQLENS)
    x = k.flatten(0, 1)
    for cu in ([0, 5, 11], [0, -1, 5], [0, 9, 5]):
        fa.append_kvcache(cache, x, x, _ints([[0, 1], [2, 3]]), _ints([0, 0]), cu_seqlens=_ints(cu), max_seqlen=5)
        _status(fa.FA_ERR_BAD_SEQLENS)


# ------------------------------------------------------------------ attention
def _full_cache(lens, Hk, page, d, seed, spread=0.0):
    """A cache of normal values; page scales vary by 2^(+-spread); noise in slots and pages of nobody."""
    table, pages = _layout(lens, page, seed)
    c = _noise_cache(pages, Hk, page, d, seed + 1)
    for b, n in enumerate(lens):
        for j in range(-(-n // page)):
            i, m = int(table[b, j]), min(page, n - j * page)
            for codes, scale, s in ((c.k8, c.k_scale, 4), (c.v8, c.v_scale, 5)):
                x = torch.randn((Hk, m, d), device="cuda", generator=_gen(1000 * seed + 10 * i + s))
                codes[i, :, :m] = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                e = torch.randn(Hk, device="cuda", generator=_gen(77 * seed + i + s)) * spread
                scale[i] = torch.exp2(torch.round(e if s == 5 else e.clamp(-2, 1)) - 6)
    return c, table


def _values(cache, table, b, n):
    at = table[b, :-(-n // cache.page)].long()
    return [(_e4m3(c[at]) * s[at].double()[..., None, None]).permute(0, 2, 1, 3).flatten(0, 1)[:n]
            for c, s in ((cache.k8, cache.k_scale), (cache.v8, cache.v_scale))]


def _reference(q, k, v, v_scale_max, scale, mask, few):
    """(o, lse, bound): as window_ref.forward, with f16 weights where the rows are few."""
    H = q.shape[1]
    kk, vv = R._spread(k, H), R._spread(v, H)
    p, lse = R._weights(q.double(), kk, scale, mask)
    o = torch.einsum("hij,jhd->ihd", p, vv)
    a = torch.einsum("hij,jhd->ihd", p, vv.abs())
    bound = ((F16 if few else R.BF16) + R.FP32) * a + R.BF16 * o.abs() + 1e-6
    if few:  # weights below f16's range: half of 2^-24 each, relative to the largest term
        bound = bound + 2.0 ** -25 * 448 * 0.3 * v_scale_max * k.shape[0]
    return o, lse, bound


def _attend_and_check(lens, n, H, Hk, d, page, causal=True, window=0, sinks=0, packed=None, seed=0, spread=0.0, max_k=None):
    new = packed or [n] * len(lens)
    c, table = _full_cache(lens, Hk, page, d, seed, spread)
    q = _rand((sum(new), H, d), seed + 9)
    B, mq = len(lens), max(new)
    out, lse = torch.full_like(q, 7.0), torch.full((B, H, mq), 7.0, device="cuda")
    max_k = max(lens) if max_k is None else max_k
    kw = dict(causal=causal, window=window, sinks=sinks)
    cu = torch.tensor([0] + new).cumsum(0).tolist()
    if packed:
        fa.forward_kvcache(q, c, table, _ints(lens), max_k, cu_seqlens_q=_ints(cu), max_seqlen_q=mq, out=out, lse=lse, **kw)
    else:
        fa.forward_kvcache(q.unflatten(0, (B, n)), c, table, _ints(lens), max_k, out=out.unflatten(0, (B, n)), lse=lse, **kw)
    _status()
    for b in range(B):
        r = slice(cu[b], cu[b + 1])
        k, v = _values(c, table, b, lens[b])
        mask = R.visible(new[b], lens[b], window, sinks, causal, device="cuda")
        used = c.v_scale[table[b, :-(-lens[b] // page)].long()]
        few = mq * (H // Hk) <= 128
        o_ref, lse_ref, bound = _reference(q[r], k, v, used[~used.isnan()].max().item() if lens[b] else 0.0,
                                           1 / math.sqrt(d), mask, few)
        R.check(out[r], o_ref, bound, "o[%d]" % b)
        R.check_lse(lse[b, :, :new[b]], lse_ref, "lse[%d]" % b)
        assert (lse[b, :, new[b]:] == 7.0).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(page, d):
    _attend_and_check([1, 2, 15, 16, 17, 127, 128, 129, 700, 0, 1500], 1, 8, 2, d, page)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 4), (12, 3), (16, 1), (20, 1), (64, 2)])
def test_heads(H, Hk, d):
    _attend_and_check([333, 1], 1, H, Hk, d, 32)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,H,Hk", [(2, 8, 2), (5, 4, 4), (7, 8, 2), (16, 4, 1), (33, 2, 2), (13, 5, 1), (30, 8, 2)])
@pytest.mark.parametrize("causal", [True, False])
def test_few_queries(n, H, Hk, d, causal):
    """Row groups of 8 and 16 rows, sequences shorter than the queries among them."""
    _attend_and_check([n, n + 1, 500, 3, 0], n, H, Hk, d, 16, causal=causal)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 130), (129, 3), (640, 0), (5000, 4)])
@pytest.mark.parametrize("n", [1, 6, 150])
def test_windows_and_sinks(window, sinks, n, d):
    _attend_and_check([n, 129, 700, 1300], n, 8, 2, d, 32, window=window, sinks=sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_long_query_chunks(d, causal):
    _attend_and_check([600, 900, 300, 2, 0], 300, 8, 2, d, 64, causal=causal)


@pytest.mark.parametrize("packed", [None, [260, 1, 0, 200, 300, 77, 260, 129] * 2])
def test_long_chunks_of_many_heads(packed):
    """More than six units an SM: they are handed out whole instead of cut into ranges."""
    _attend_and_check([300, 500, 260, 411] * 4 if packed is None else [300, 500, 10, 411] * 4, 260, 32, 2, 64, 32,
                      packed=packed, window=0 if packed is None else 150, sinks=0 if packed is None else 3)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [[1, 3, 0, 2], [129, 0, 1, 300]])
def test_packed_queries(d, packed):
    _attend_and_check([5, 400, 77, 555], 0, 8, 2, d, 16, packed=packed)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,n,H,Hk,window,sinks", [(20, 1, 8, 4, 0, 0), (20, 3, 16, 4, 300, 4), (13, 2, 10, 5, 0, 0),
                                                   (1, 1, 4, 1, 0, 0)])
def test_few_units(B, n, H, Hk, d, window, sinks):
    """Clusters of several sizes, some of whose members have no step of a short sequence."""
    _attend_and_check([(997 * b + 700) % 1000 if b % 4 else 1000 for b in range(B)], n, H, Hk, d, 32, window=window,
                      sinks=sinks, seed=11)


def test_page_scales_that_differ_widely():
    for n in (1, 4):
        _attend_and_check([900, 200], n, 8, 2, 128, 16, spread=6.0)


def test_many_splits_and_loose_bound():
    _attend_and_check([9000], 1, 4, 1, 128, 64)
    _attend_and_check([90, 9000], 1, 4, 1, 64, 128, max_k=40_000)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_pages_that_were_never_written(n, d):
    """Scale 0: keys and values of 0.  Every key of such pages has score 0 and counts."""
    Hk, H, page, m = 2, 4, 32, 300
    c, table = _full_cache([m], Hk, page, d, 5)
    empty = table[0, [1, 2, 7]].long()
    for t in (c.k8, c.v8, c.k_scale, c.v_scale):
        t[empty] = 0
    q = _rand((1, n, H, d), 6)
    o, lse = fa.forward_kvcache(q, c, table, _ints([m]), m)
    _status()
    k, v = _values(c, table, 0, m)
    vs = c.v_scale[table[0].long()].max().item()
    ref, lref, bound = _reference(q[0], k, v, vs, 1 / math.sqrt(d), R.visible(n, m, 0, 0, device="cuda"), n * H // Hk <= 128)
    R.check(o[0], ref, bound, "o")
    R.check_lse(lse[0], lref, "lse")
    o, lse = fa.forward_kvcache(q, fa.KvCache.empty(c.num_pages, page, Hk, d), table, _ints([m]), m)
    _status()
    assert (o == 0).all()
    R.check_lse(lse[0], torch.log(torch.arange(m - n + 1, m + 1, device="cuda").double()).expand(H, n), "lse of an empty cache")


@pytest.mark.parametrize("n", [1, 100])
def test_lengths_against_no_keys_at_all(n):
    c, table = _full_cache([64, 64, 64], 2, 16, 64, 1)
    q = _rand((3, n, 4, 64), 2)
    o, lse = fa.forward_kvcache(q, c, table, _ints([0, 0, 0]), 0)
    _status()
    assert (o == 0).all() and torch.isneginf(lse).all()
    fa.forward_kvcache(q, c, table, _ints([0, 0, 3]), 0)
    _status(fa.FA_ERR_BAD_SEQLENS)


def test_rows_behind_the_last_sequence_are_left():
    c, table = _full_cache([40, 300], 2, 16, 64, 5)
    for new in ([3, 2], [150, 200]):
        T = sum(new) + 4
        q, cu = _rand((T, 4, 64), 1), _ints([0, new[0], sum(new)])
        out = torch.full_like(q, 7.0)
        fa.forward_kvcache(q, c, table, _ints([40, 300]), 300, cu_seqlens_q=cu, max_seqlen_q=max(new), out=out)
        _status()
        assert (out[-4:] == 7.0).all() and not (out[:-4] == 7.0).all(-1).any()
    k = _rand((9, 2, 64), 2)
    out = torch.full((9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    before = c.k8.clone()
    fa.append_kvcache(c, k, k, table, _ints([30, 200]), q=_rand((9, 4, 64), 3), q_out=out, cu_seqlens=_ints([0, 2, 5]),
                      max_seqlen=3)
    _status()
    assert (out[5:] == 7.0).all() and not (out[:5] == 7.0).all(-1).any()
    assert int((before != c.k8).any(-1).sum()) <= 2 * 5 + 2 * 2 * 15  # new slots, and older ones of the two pages


def test_offsets_past_32_bits():
    """Pages that begin past 2^32 bytes of codes, in every path."""
    Hk, page, d = 8, 128, 128
    pages = (1 << 32) // (Hk * page * d) + 40
    c = fa.KvCache.empty(pages, page, Hk, d)
    lens = [300, 129]
    table = _ints([[pages - 1, pages - 3, pages - 8], [pages - 2, pages - 5, 0]])
    x = _rand((sum(lens), 4 * Hk + 2 * Hk, d), 1)
    cu = _ints([0, 300, 429])
    fa.append_kvcache(c, x[:, 32:40], x[:, 40:], table, _ints([0, 0]), cu_seqlens=cu, max_seqlen=300)
    _status()
    for b in range(2):
        k, v = _values(c, table, b, lens[b])
        rows = x[int(cu[b]):int(cu[b + 1])].double()
        for got, want in ((k, rows[:, 32:40]), (v, rows[:, 40:])):
            assert ((got - want).abs() <= want.abs() * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -10 * 2.0 ** -6).all()
    for n in (1, 60):
        q = _rand((2, n, 32, d), 2)
        o, lse = fa.forward_kvcache(q, c, table, _ints(lens), 300)
        _status()
        for b in range(2):
            k, v = _values(c, table, b, lens[b])
            ref, lref, bound = _reference(q[b], k, v, 2.0 ** -6, d ** -0.5, R.visible(n, lens[b], 0, 0, device="cuda"), n == 1)
            R.check(o[b], ref, bound, "o")
            R.check_lse(lse[b], lref, "lse")


def test_on_another_stream():
    """The calls run on the stream they are given, and what they allocate belongs to it."""
    c, table = _full_cache([900], 2, 32, 128, 6)
    q, lens = _rand((1, 1, 8, 128), 1), _ints([900])
    o, lse = fa.forward_kvcache(q, c, table, lens, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = fa.forward_kvcache(q, c, table, lens, 900, stream=side)
    k = _rand((1, 1, 2, 128), 2)
    qr = fa.append_kvcache(c, k, k, table, _ints([100]), q=q, stream=side)
    side.synchronize()
    _status()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(qr, q)


def test_two_calls_at_once():
    """Two streams, each with a workspace of its own: the same bits as one after the other."""
    c, table = _full_cache([3000, 1700], 4, 64, 128, 7)
    lens = _ints([3000, 1700])
    qs = [_rand((2, n, 16, 128), n) for n in (1, 40)]
    one = [fa.forward_kvcache(q, c, table, lens, 3000) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        two = [fa.forward_kvcache(q, c, table, lens, 3000, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(one, two):
            assert torch.equal(a, x) and torch.equal(b, y)
    _status()


def test_outliers_in_queries_keep_their_row():
    """Rows of very different size, one infinite: the others are right."""
    c, table = _full_cache([300], 1, 16, 128, 3)
    q = _rand((1, 1, 4, 128), 4)
    q[0, 0, 0] *= 1e-20
    q[0, 0, 1] *= 30
    q[0, 0, 2, 5] = math.inf
    o, lse = fa.forward_kvcache(q, c, table, _ints([300]), 300, scale=0.02)
    _status()
    k, v = _values(c, table, 0, 300)
    rows = [0, 1, 3]
    o_ref, lse_ref, bound = _reference(q[0][:, rows], k, v, c.v_scale[table[0].long()].max().item(), 0.02,
                                       R.visible(1, 300, 0, 0, device="cuda"), True)
    R.check(o[0][:, rows], o_ref, bound, "o")
    R.check_lse(lse[0][rows], lse_ref, "lse")


def test_attention_reports_what_does_not_fit():
    c, table = _full_cache([100, 100], 2, 16, 64, 1)
    q = _rand((2, 1, 4, 64), 2)
    for n in (1, 100):
        x = q.expand(2, n, 4, 64).contiguous()
        for lens, max_k in (([101, 100], 100), ([-1, 100], 100), ([200, 100], 300)):
            fa.forward_kvcache(x, c, table, _ints(lens), max_k)
            _status(fa.FA_ERR_BAD_SEQLENS)
        for bad in (-1, c.num_pages):
            t = table.clone()
            t[1, 3] = bad
            fa.forward_kvcache(x, c, t, _ints([100, 100]), 100)
            _status(fa.FA_ERR_BAD_PAGE)
            fa.forward_kvcache(x, c, t, _ints([100, 40]), 100)  # not a page of the 40 tokens
            _status()
        y = x.flatten(0, 1)
        for cu in ([0, n, 2 * n + 1], [0, -1, 2], [1, 0, 1]):
            fa.forward_kvcache(y, c, table, _ints([100, 100]), 100, cu_seqlens_q=_ints(cu), max_seqlen_q=n)
            _status(fa.FA_ERR_BAD_SEQLENS)


def test_refusals():
    c = fa.KvCache.empty(4, 16, 2, 64)
    q, k = _rand((1, 1, 4, 64), 1), _rand((1, 1, 2, 64), 2)
    table, lens = _ints([[0, 1]]), _ints([3])
    with pytest.raises(ValueError):
        fa.KvCache(c.k8, c.v8[:2], c.k_scale, c.v_scale)
    with pytest.raises(TypeError):
        fa.KvCache(c.k8.view(torch.int8), c.v8, c.k_scale, c.v_scale)
    with pytest.raises(fa.FaError):
        fa.append_kvcache(fa.KvCache.empty(4, 8, 2, 64), k, k, table, lens)
    with pytest.raises(ValueError):
        fa.append_kvcache(c, k.transpose(2, 3).contiguous().transpose(2, 3), k, table, lens)
    with pytest.raises(ValueError):
        fa.append_kvcache(c, k, k, table, _ints([3, 4]))
    with pytest.raises(ValueError):
        fa.append_kvcache(c, k, k, table, lens, cos=torch.zeros(9, 32, device="cuda"))
    with pytest.raises(fa.FaError):
        fa.append_kvcache(c, k, k, table, lens, cos=torch.zeros(9, 12, device="cuda"), sin=torch.zeros(9, 12, device="cuda"))
    with pytest.raises(fa.FaError):  # rows that do not begin on 16 bytes
        x = _rand((1, 4, 129 * 2 + 4,), 3)[..., 4:260].unflatten(-1, (4, 64))
        fa.append_kvcache(c, x[:, :, :2], x[:, :, 2:], table, lens)
    with pytest.raises(fa.FaError):  # the same row for every token
        x = _rand((1, 1, 2, 64), 3).expand(1, 4, 2, 64)
        fa.append_kvcache(c, x, x, table, lens)
    with pytest.raises(ValueError):
        fa.forward_kvcache(_rand((1, 1, 3, 64), 1), c, table, lens, 3)
    with pytest.raises(ValueError):
        fa.forward_kvcache(q.transpose(1, 2), c, table, lens, 3)
    with pytest.raises(ValueError):
        fa.forward_kvcache(q, c, table.long().int().expand(2, 2), lens, 3)
    with pytest.raises(fa.FaError):
        fa.forward_kvcache(q, c, table, lens, 3, causal=False, window=4)
    with pytest.raises(ValueError):
        fa.forward_kvcache(q, c, table, lens, 10 ** 6, workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))


def test_serving_run_captured():
    """Prompts in, then tokens one by one across page borders: append, attend and the lengths
    replayed from one graph, each step against the cache's own values; then the same loop on
    another stream gives the same bits."""
    B, H, Hk, d, page, steps, window, sinks = 3, 8, 2, 128, 16, 20, 48, 4
    prompts = [70, 5, 33]
    total = [p + steps for p in prompts]
    cos, sin = _tables(max(total), d)

    def serve(stream, graph):
        table, pages = _layout(total, page, 1)
        cache = _noise_cache(pages, Hk, page, d, 2)
        cu = _ints([0] + torch.tensor(prompts).cumsum(0).tolist())
        x = _rand((sum(prompts), H + 2 * Hk, d), 3)
        q = fa.append_kvcache(cache, x[:, H:H + Hk], x[:, H + Hk:], table, _ints([0] * B), q=x[:, :H], cos=cos, sin=sin,
                              cu_seqlens=cu, max_seqlen=max(prompts))
        o0, _ = fa.forward_kvcache(q, cache, table, _ints(prompts), max(prompts), window=window, sinks=sinks,
                                   cu_seqlens_q=cu, max_seqlen_q=max(prompts))
        held, after = _ints(prompts), _ints([p + 1 for p in prompts])
        tok, o, lse = torch.zeros((B, 1, H + 2 * Hk, d), dtype=torch.bfloat16, device="cuda"), None, None

        def step():
            qq = fa.append_kvcache(cache, tok[:, :, H:H + Hk], tok[:, :, H + Hk:], table, held, q=tok[:, :, :H], cos=cos,
                                   sin=sin)
            out = fa.forward_kvcache(qq, cache, table, after, max(total), window=window, sinks=sinks)
            held.add_(1)
            after.add_(1)
            return qq, out
        outs, g = [o0], None
        for t in range(steps):
            tok.copy_(_rand(tok.shape, 100 + t))
            if graph and t == 1:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    qq, (o, lse) = step()
            if g is not None:
                g.replay()
            else:
                qq, (o, lse) = step()
            if graph:
                torch.cuda.synchronize()
                for b in range(B):
                    n = prompts[b] + t + 1
                    k, v = _values(cache, table, b, n)
                    used = cache.v_scale[table[b, :-(-n // page)].long()]
                    ref, lref, bound = _reference(qq[b], k, v, used.max().item(), 1 / math.sqrt(d),
                                                  R.visible(1, n, window, sinks, device="cuda"), True)
                    R.check(o[b], ref, bound, "step %d sequence %d" % (t, b))
                    R.check_lse(lse[b], lref, "step %d sequence %d" % (t, b))
            outs.append(o.clone())
        return outs
    first = serve(None, True)
    _status()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = serve(side, False)
    torch.cuda.synchronize()
    _status()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
