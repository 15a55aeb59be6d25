"""Cases for the cache and window operators: what is measured, and their plain form.

Three operators.  "append" rotates new keys (and queries) to their positions and writes keys and
values into a paged cache of e4m3 codes with one power-of-two scale per page and head.  "attend" is
attention of new queries over such a cache.  "window" is attention with a sliding window and a few
first tokens that stay visible, forward and backward.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # A few chat sequences decoding one token each with a small model: latency of one call.
        dict(name="append_one_b4", op="append", B=4, new=1, ctx=1000, H=16, Hk=4, d=128, page=16, rot=128,
             inter=False, packed=False, mix=1),
        # A full decoding batch of a server.
        dict(name="append_one_b256", op="append", B=256, new=1, ctx=4096, H=32, Hk=8, d=128, page=64, rot=128,
             inter=False, packed=False, mix=2),
        # Ragged prompts entering the cache together, partial rotation of neighbouring pairs.
        dict(name="append_prompts", op="append", B=12, new=2047, ctx=500, H=32, Hk=8, d=64, page=32, rot=32,
             inter=True, packed=True, mix=3),
        # One sequence, short context: the smallest call.
        dict(name="attend_one_b1", op="attend", B=1, Nq=1, ctx=1021, H=16, Hk=4, d=128, page=16, window=0, sinks=0,
             packed=False, mix=4),
        # A decoding batch of ragged lengths.
        dict(name="attend_one_b64", op="attend", B=64, Nq=1, ctx=8191, H=32, Hk=8, d=128, page=64, window=0,
             sinks=0, packed=False, mix=5),
        # Two very long documents, one token each.
        dict(name="attend_long_b2", op="attend", B=2, Nq=1, ctx=131075, H=32, Hk=8, d=128, page=128, window=0,
             sinks=0, packed=False, mix=6),
        # Checking four drafted tokens in a window with sinks, small heads.
        dict(name="attend_draft_window", op="attend", B=33, Nq=4, ctx=6001, H=16, Hk=4, d=64, page=32, window=1024,
             sinks=4, packed=False, mix=7),
        # Prompt chunks of ragged length over what the cache holds already.
        dict(name="attend_chunk", op="attend", B=3, Nq=1024, ctx=8192, H=16, Hk=4, d=128, page=64, window=0, sinks=0,
             packed=True, mix=8),
        # Scoring a short batch in a window.
        dict(name="window_fwd_n1000", op="window", B=2, N=1000, H=8, Hk=8, d=64, window=256, sinks=1, packed=False,
             grad=False, mix=9),
        # Training on the sequence length of the benchmark.
        dict(name="window_train_n4096", op="window", B=2, N=4096, H=16, Hk=4, d=128, window=512, sinks=4,
             packed=False, grad=True, mix=10),
        # Training on packed documents of ragged length.
        dict(name="window_train_packed", op="window", B=9, N=2048, H=8, Hk=2, d=64, window=300, sinks=16,
             packed=True, grad=True, mix=11),
        # Training on one long document.
        dict(name="window_train_n16384", op="window", B=1, N=16384, H=8, Hk=2, d=128, window=1024, sinks=64,
             packed=False, grad=True, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "window"))
    d = rng.choice((64, 128))
    Hk = rng.choice((1, 2, 4, 8))
    mix = rng.randrange(1, 1 << 20)
    if op == "append":
        new = rng.choice((1, 1, _log(rng, 2, 2048)))
        return dict(op=op, B=_log(rng, 1, 256 if new == 1 else 12), new=new, ctx=_log(rng, 16, 4096),
                    H=Hk * rng.choice((1, 2, 4)), Hk=Hk, d=d, page=rng.choice((16, 32, 64, 128)),
                    rot=rng.choice((32, 64, d)), inter=rng.random() < 0.5, packed=new > 1, mix=mix)
    if op == "attend":
        kind = rng.choice(("one", "one", "few", "chunk"))
        Nq = 1 if kind == "one" else _log(rng, 2, 32) if kind == "few" else _log(rng, 33, 1024)
        B = _log(rng, 1, 3 if kind == "chunk" else 64)
        ctx = max(Nq + 1, _log(rng, 64, 8192 if kind == "chunk" else 500_000 // max(B, 4)))
        windowed = rng.random() < 0.4
        return dict(op=op, B=B, Nq=Nq, ctx=ctx, H=Hk * rng.choice((1, 2, 4)), Hk=Hk, d=d,
                    page=rng.choice((16, 32, 64, 128)), window=_log(rng, 16, 4096) if windowed else 0,
                    sinks=rng.choice((0, 1, 4, 16, 130)) if windowed else 0, packed=kind == "chunk", mix=mix)
    N = _log(rng, 64, 4096)
    Hk = min(Hk, 4)
    return dict(op=op, B=_log(rng, 1, 4), N=N, H=Hk * rng.choice((1, 2, 4)), Hk=Hk, d=d, window=_log(rng, 1, N),
                sinks=rng.choice((0, 1, 4, 64, 200)), packed=rng.random() < 0.4, grad=rng.random() < 0.6, mix=mix)


def _lengths(case):
    """(tokens in the cache or keys, new tokens or queries) of each sequence: from the case alone."""
    rng = random.Random(case["mix"])
    B = case["B"]
    if case["op"] == "append":
        old = [rng.randint(0, case["ctx"]) for _ in range(B)]
        new = [rng.randint(0, case["new"]) if case["packed"] else case["new"] for _ in range(B)]
        new[0], old[-1] = case["new"], case["ctx"]
        return old, new
    if case["op"] == "attend":
        new = [rng.randint(1, case["Nq"]) if case["packed"] else case["Nq"] for _ in range(B)]
        new[0] = case["Nq"]
        ctx = [max(n, rng.randint(case["ctx"] // 4, case["ctx"])) for n in new]
        ctx[-1] = case["ctx"]
        return ctx, new
    n = [rng.randint(1, case["N"]) if case["packed"] else case["N"] for _ in range(B)]
    n[0] = case["N"]
    return n, n


def _pairs(n_q, n_k, window, sinks):
    """Visible (query, key) pairs: query i at position p = i + n_k - n_q sees keys j <= p with
    p - j < window or j < sinks (window 0: every key up to p)."""
    total = 0
    for p in range(n_k - n_q, n_k):
        seen = p + 1
        if window and seen > window:
            seen = window + min(sinks, seen - window)
        total += seen
    return total


def work(case):
    d, H, Hk = case["d"], case["H"], case["Hk"]
    k_len, q_len = _lengths(case)
    T = sum(q_len)
    if case["op"] == "append":
        pages = sum((o % case["page"] + n + case["page"] - 1) // case["page"] for o, n in zip(k_len, q_len))
        byts = T * (2 * Hk * d * 2 + 2 * Hk * d + 2 * H * d * 2 + case["rot"] * 4) + pages * (2 * Hk * 4 + 4)
        return {"bytes": byts, "flops": T * (Hk + H) * case["rot"] * 3 + T * 2 * Hk * d * 2}
    if case["op"] == "attend":
        w, s = case["window"], case["sinks"]
        keys = 0  # keys that some query of the sequence sees
        for n, q in zip(k_len, q_len):
            lo = max(0, n - q + 1 - w) if w else 0
            keys += n - max(0, lo - s)
        pairs = sum(_pairs(q, n, w, s) for n, q in zip(k_len, q_len))
        byts = keys * 2 * Hk * d + -(-keys // case["page"]) * (2 * Hk * 4 + 4) + T * H * (d * 4 + 4)
        return {"bytes": byts, "flops": 4 * pairs * H * d}
    pairs = sum(_pairs(n, n, case["window"], case["sinks"]) for n in k_len)
    byts = T * (2 * H * d * 2 + 2 * Hk * d * 2 + H * 4)
    if case["grad"]:
        byts += T * (4 * H * d * 2 + 4 * Hk * d * 2 + H * 4)
    return {"bytes": byts, "flops": (14 if case["grad"] else 4) * pairs * H * d}


# ------------------------------------------------------------------- inputs
def _pow2_scale(amax):
    """Smallest power of two s >= 2^-64 with amax <= 448 s."""
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=-64)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -64)))


def _to_codes(x, scale):
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _cu(lens, dev):
    return torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)


def _filled_cache(pages, Hk, page, d, g, dev):
    """A cache of normal values whose size differs from page to page and head to head."""
    out = []
    for _ in ("k", "v"):
        codes = torch.empty((pages, Hk, page, d), dtype=torch.uint8, device=dev)
        scale = torch.empty((pages, Hk), dtype=torch.float32, device=dev)
        step = max(1, (1 << 26) // (Hk * page * d))
        for a in range(0, pages, step):
            n = min(step, pages - a)
            x = torch.randn((n, Hk, page, d), device=dev, generator=g)
            x *= torch.exp(0.3 * torch.randn((n, Hk, 1, 1), device=dev, generator=g))
            scale[a:a + n] = _pow2_scale(x.abs().amax((2, 3)))
            codes[a:a + n] = _to_codes(x, scale[a:a + n, :, None, None])
        out += [codes, scale]
    return out


def _tables(total, page, g, dev):
    """Pages of each sequence in an order that a long-running server ends up with, a few of them in
    nobody's hands; -1 behind a sequence's last page."""
    need = [-(-n // page) for n in total]
    pages = sum(need) + 3
    order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    width = max(max(need), 1)
    table = torch.full((len(total), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pages


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    d, H, Hk, B = case["d"], case["H"], case["Hk"], case["B"]
    k_len, q_len = _lengths(case)
    T = sum(q_len)
    s = {"case": case, "max_q": max(q_len), "max_k": max(k_len)}

    def rows(heads, dense=not case["packed"]):
        x = torch.randn((T, heads, d), device=dev, generator=g).to(torch.bfloat16)
        return x.view(B, T // B, heads, d) if dense else x

    if case["op"] == "append":
        # The projection's output: q, k and v of a token side by side.
        x = torch.randn((T, H + 2 * Hk, d), device=dev, generator=g).to(torch.bfloat16)
        x = x if case["packed"] else x.view(B, T // B, H + 2 * Hk, d)
        s["q"], s["k"], s["v"] = x[..., :H, :], x[..., H:H + Hk, :], x[..., H + Hk:, :]
        s["table"], pages = _tables([o + n for o, n in zip(k_len, q_len)], case["page"], g, dev)
        s["k8"], s["k_scale"], s["v8"], s["v_scale"] = _filled_cache(pages, Hk, case["page"], d, g, dev)
        most = max(o + n for o, n in zip(k_len, q_len))
        half = case["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        angle = torch.arange(most, device=dev, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["lens"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
        s["cu"] = _cu(q_len, dev) if case["packed"] else None
    elif case["op"] == "attend":
        s["q"] = rows(H)
        s["table"], pages = _tables(k_len, case["page"], g, dev)
        s["k8"], s["k_scale"], s["v8"], s["v_scale"] = _filled_cache(pages, Hk, case["page"], d, g, dev)
        s["lens"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
        s["cu"] = _cu(q_len, dev) if case["packed"] else None
        s["lse"] = torch.zeros((B, H, s["max_q"]), device=dev)
    else:
        s["q"], s["k"], s["v"] = rows(H), rows(Hk), rows(Hk)
        s["dout"] = rows(H) if case["grad"] else None
        s["cu"] = _cu(q_len, dev) if case["packed"] else None
        s["lse"] = torch.zeros((B, H, s["max_q"]), device=dev)
    return s


# -------------------------------------------------------------- a pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "window": _own_window}[op](s)
    return {"append": _plain_append, "attend": _plain_attend, "window": _plain_window}[op](s)


def _own_append(s):
    import attention_forward_fa2_gb300 as fa
    cache = fa.KvCache(s["k8"], s["v8"], s["k_scale"], s["v_scale"])
    q = fa.append_kvcache(cache, s["k"], s["v"], s["table"], s["lens"], q=s["q"], cos=s["cos"], sin=s["sin"],
                          interleaved=s["case"]["inter"], cu_seqlens=s["cu"], max_seqlen=s["max_q"])
    return {"q": q, "k8": s["k8"].view(torch.float8_e4m3fn), "v8": s["v8"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_attend(s):
    import attention_forward_fa2_gb300 as fa
    c = s["case"]
    cache = fa.KvCache(s["k8"], s["v8"], s["k_scale"], s["v_scale"])
    o, lse = fa.forward_kvcache(s["q"], cache, s["table"], s["lens"], s["max_k"], window=c["window"],
                                sinks=c["sinks"], cu_seqlens_q=s["cu"], max_seqlen_q=s["max_q"], lse=s["lse"])
    return {"o": o, "lse": lse}


def _own_window(s):
    import attention_forward_fa2_gb300 as fa
    c = s["case"]
    more = {} if s["cu"] is None else dict(cu_seqlens_q=s["cu"], cu_seqlens_k=s["cu"], max_seqlen_q=s["max_q"],
                                           max_seqlen_k=s["max_k"])
    o, lse = fa.forward_window(s["q"], s["k"], s["v"], c["window"], c["sinks"], lse=s["lse"], **more)
    if not c["grad"]:
        return {"o": o, "lse": lse}
    dq, dk, dv = fa.backward_window(s["q"], s["k"], s["v"], o, lse, s["dout"], c["window"], c["sinks"], **more)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ----------------------------------------------------------- plain forms
def _token_places(s):
    """Sequence and index within it of every new token, in packed order."""
    B = s["case"]["B"]
    if s["cu"] is None:
        n = s["max_q"]
        t = torch.arange(B * n, device=s["q"].device)
        return t // n, t % n
    total = s["q"].shape[0]
    cu = s["cu"].long()
    t = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, t - cu[b]


def _rotate(x, cos, sin, inter):
    """x [T, heads, d] fp32; cos, sin [T, 1, rot / 2]."""
    half = cos.shape[-1]
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :half], r[..., half:])
    ya, yb = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((ya, yb), -1).flatten(-2) if inter else torch.cat((ya, yb), -1)
    return torch.cat((y, rest), -1)


def _plain_append(s):
    c = s["case"]
    page, d = c["page"], c["d"]
    b, i = _token_places(s)
    lens = s["lens"].long()
    pos = lens[b] + i
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    qf = _rotate(s["q"].reshape(-1, c["H"], d).float(), cos, sin, c["inter"])
    pid = s["table"][b, pos // page].long()
    slot = pos % page
    # The page that a sequence had begun before: its older tokens stay, under the larger scale.
    began = (lens % page) > 0
    first = s["table"].long().gather(1, (lens // page).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].clamp(min=0)
    fresh = torch.ones(s["k8"].shape[0], dtype=torch.bool, device=lens.device)
    fresh[first[began]] = False
    older = (torch.arange(page, device=lens.device)[None] < (lens % page)[:, None])[:, None, :, None] & began[:, None, None, None]
    for x, codes, scale in ((_rotate(s["k"].reshape(-1, c["Hk"], d).float(), cos, sin, c["inter"]), s["k8"], s["k_scale"]),
                            (s["v"].reshape(-1, c["Hk"], d).float(), s["v8"], s["v_scale"])):
        amax = torch.full_like(scale, -1.0)
        amax.scatter_reduce_(0, pid[:, None].expand(-1, c["Hk"]), x.abs().amax(-1), "amax")
        want = _pow2_scale(amax.clamp(min=0))
        want = torch.where(fresh[:, None], want, torch.maximum(want, scale))
        new = torch.where(amax >= 0, want, scale)
        held = codes[first]
        value = held.view(torch.float8_e4m3fn).float() * scale[first][:, :, None, None]
        held = torch.where(older, _to_codes(value, new[first][:, :, None, None]), held)
        codes.index_copy_(0, first[began], held[began])
        codes[pid, :, slot] = _to_codes(x, new[pid][:, :, None])
        scale.copy_(new)
    return {"q": qf.to(torch.bfloat16).view(s["q"].shape), "k8": s["k8"].view(torch.float8_e4m3fn),
            "v8": s["v8"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _seen(n_q, n_k, most_q, most_k, window, sinks):
    """[B, most_q, most_k]: whether query i of a sequence sees key j; n_q, n_k [B]."""
    p = torch.arange(most_q, device=n_q.device)[None, :, None] + (n_k - n_q)[:, None, None]
    j = torch.arange(most_k, device=n_q.device)[None, None, :]
    ok = (j <= p) & (torch.arange(most_q, device=n_q.device)[None, :, None] < n_q[:, None, None])
    return ok & ((p - j < window) | (j < sinks)) if window else ok


def _padded(x, b, i, B, most):
    """Rows [T, heads, d] of packed sequences as fp32 [B, heads, most, d], zeros behind the last."""
    out = torch.zeros((B, most, x.shape[1], x.shape[2]), device=x.device)
    out[b, i] = x.float()
    return out.transpose(1, 2)


def _softmax(score, seen):
    score = score.masked_fill(~seen, -math.inf)
    m = score.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(score - m)
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l > 0, l, torch.ones_like(l)), (m + torch.log(l))[..., 0]


def _plain_attend(s):
    c = s["case"]
    B, H, Hk, d, most, n = c["B"], c["H"], c["Hk"], c["d"], s["max_q"], s["max_k"]
    b, i = _token_places(s)
    q = _padded(s["q"].reshape(-1, H, d), b, i, B, most).reshape(B, Hk, H // Hk, most, d)
    t = s["table"].clamp(min=0).long()
    k, v = ((codes[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]).transpose(1, 2)
            .reshape(B, Hk, 1, -1, d)[:, :, :, :n] for codes, scale in ((s["k8"], s["k_scale"]), (s["v8"], s["v_scale"])))
    n_q = torch.bincount(b, minlength=B)
    seen = _seen(n_q, s["lens"].long(), most, n, c["window"], c["sinks"])[:, None, None]
    p, lse = _softmax((q / math.sqrt(d)) @ k.transpose(-1, -2), seen)
    o = (p @ v).reshape(B, H, most, d).transpose(1, 2)
    s["lse"][b, :, i] = lse.reshape(B, H, most)[b, :, i]
    return {"o": o[b, i].to(torch.bfloat16).view(s["q"].shape), "lse": s["lse"]}


def _plain_window(s):
    c = s["case"]
    B, H, Hk, d, most = c["B"], c["H"], c["Hk"], c["d"], s["max_q"]
    b, i = _token_places(s)
    q = _padded(s["q"].reshape(-1, H, d), b, i, B, most).reshape(B, Hk, H // Hk, most, d)
    k, v = (_padded(s[x].reshape(-1, Hk, d), b, i, B, most)[:, :, None] for x in "kv")
    n = torch.bincount(b, minlength=B)
    scale = 1.0 / math.sqrt(d)
    p, lse = _softmax((q * scale) @ k.transpose(-1, -2), _seen(n, n, most, most, c["window"], c["sinks"])[:, None, None])
    o = p @ v

    def packed(x, heads, like):
        return x.reshape(B, heads, most, d).transpose(1, 2)[b, i].to(torch.bfloat16).view(like.shape)

    s["lse"][b, :, i] = lse.reshape(B, H, most)[b, :, i]
    out = {"o": packed(o, H, s["q"]), "lse": s["lse"]}
    if not c["grad"]:
        return out
    do = _padded(s["dout"].reshape(-1, H, d), b, i, B, most).reshape(q.shape)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = do @ v.transpose(-1, -2)
    ds -= (do * o).sum(-1, keepdim=True)
    ds *= p
    dq = (ds @ k) * scale
    dk = (ds.transpose(-1, -2) @ q).sum(2) * scale
    return dict(out, dq=packed(dq, H, s["q"]), dk=packed(dk, Hk, s["k"]), dv=packed(dv, Hk, s["v"]))


# ------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    k_len, q_len = _lengths(case)
    starts = [sum(q_len[:b]) for b in range(case["B"] + 1)]
    return {"append": _exact_append, "attend": _exact_attend, "window": _exact_window}[case["op"]](s, k_len, q_len, starts)


def _exact_append(s, k_len, q_len, starts):
    c = s["case"]
    page, d, half = c["page"], c["d"], c["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)

    def turned(x, first):
        p = torch.arange(first, first + x.shape[0], device="cuda", dtype=torch.float64)
        z = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p[:, None] * freq)[:, None]
        y = x.clone()
        at = torch.arange(half, device="cuda")
        a, b = (2 * at, 2 * at + 1) if c["inter"] else (at, at + half)
        w = torch.complex(x[..., a], x[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        return y

    q, k, v = (s[n].reshape(-1, s[n].shape[-2], d).double() for n in "qkv")
    table = s["table"].tolist()
    out_q = torch.empty_like(q)
    old = {n: s[n + "8"].view(torch.float8_e4m3fn).double() for n in "kv"}
    codes = {n: old[n].clone() for n in "kv"}
    scales = {n: s[n + "_scale"].double() for n in "kv"}
    for b, (have, add) in enumerate(zip(k_len, q_len)):
        if not add:
            continue
        own_rows = slice(starts[b], starts[b] + add)
        out_q[own_rows] = turned(q[own_rows], have)
        for name, x in (("k", turned(k[own_rows], have)), ("v", v[own_rows])):
            for n in range(have // page, (have + add - 1) // page + 1):
                at = table[b][n]
                lo, hi = max(have, n * page), min(have + add, (n + 1) * page)
                block = x[lo - have:hi - have].transpose(0, 1)
                need = block.abs().amax((1, 2)) / 448.0
                scale = torch.exp2(torch.ceil(torch.log2(need.clamp(min=2.0 ** -64))))
                if lo > n * page:
                    scale = torch.maximum(scale, scales[name][at])
                    kept = old[name][at, :, :lo - n * page] * scales[name][at][:, None, None]
                    codes[name][at, :, :lo - n * page] = (kept / scale[:, None, None]).to(torch.float8_e4m3fn).double()
                codes[name][at, :, lo - n * page:hi - n * page] = (block / scale[:, None, None]).float().to(torch.float8_e4m3fn).double()
                scales[name][at] = scale
    return {"q": out_q.view(s["q"].shape), "k8": codes["k"], "v8": codes["v"], "k_scale": scales["k"], "v_scale": scales["v"]}


def _visible(n_q, n_k, window, sinks):
    m = torch.ones((n_q, n_k), dtype=torch.bool, device="cuda").tril(n_k - n_q)
    if window:
        m &= ~torch.ones_like(m).tril(n_k - n_q - window) | (torch.arange(n_k, device="cuda") < sinks)
    return m


def _exact_attend(s, k_len, q_len, starts):
    c = s["case"]
    H, Hk, d, page = c["H"], c["Hk"], c["d"], c["page"]
    q = s["q"].reshape(-1, H, d).double()
    o, lse = torch.empty_like(q), torch.zeros_like(s["lse"], dtype=torch.float64)
    for b, (n, m) in enumerate(zip(k_len, q_len)):
        at = s["table"][b, :-(-n // page)].long()
        k, v = ((s[x + "8"][at].view(torch.float8_e4m3fn).double() * s[x + "_scale"][at].double()[..., None, None])
                .permute(1, 0, 2, 3).reshape(Hk, -1, d)[:, :n] for x in "kv")
        hidden = ~_visible(m, n, c["window"], c["sinks"])
        for h in range(H):
            x = (q[starts[b]:starts[b] + m, h] @ k[h * Hk // H].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            o[starts[b]:starts[b] + m, h] = torch.softmax(x, -1) @ v[h * Hk // H]
            lse[b, h, :m] = torch.logsumexp(x, -1)
    return {"o": o.view(s["q"].shape), "lse": lse}


def _exact_window(s, k_len, q_len, starts):
    c = s["case"]
    H, Hk, d = c["H"], c["Hk"], c["d"]
    q, k, v = (s[x].reshape(-1, s[x].shape[-2], d).double() for x in "qkv")
    do = s["dout"].reshape(-1, H, d).double() if c["grad"] else None
    o, lse = torch.empty_like(q), torch.zeros_like(s["lse"], dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b, n in enumerate(k_len):
        r = slice(starts[b], starts[b] + n)
        hidden = ~_visible(n, n, c["window"], c["sinks"])
        for h in range(H):
            g = h * Hk // H
            x = (q[r, h] @ k[r, g].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            lse[b, h, :n] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            o[r, h] = p @ v[r, g]
            if do is None:
                continue
            dp = do[r, h] @ v[r, g].T
            dx = p * (dp - (p * dp).sum(-1, keepdim=True)) / math.sqrt(d)
            dq[r, h] = dx @ k[r, g]
            dk[r, g] += dx.T @ q[r, h]
            dv[r, g] += p.T @ do[r, h]
    out = {"o": o.view(s["q"].shape), "lse": lse}
    if do is not None:
        out |= {"dq": dq.view(s["q"].shape), "dk": dk.view(s["k"].shape), "dv": dv.view(s["v"].shape)}
    return out
