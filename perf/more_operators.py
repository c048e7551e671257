"""Cases for the operators of a paged cache held in 4 bits and of sliding windows
over a paged cache: keys and values normed, rotated and appended in 4 bits, cached
tokens read back into the layer's layout, attention of drafted tokens over the
4-bit cache, and attention through a window that keeps the first tokens.

``run`` computes a case in elementary torch operations (32 bits; 64 for the
angles and for what is rounded to 4 bits) or, with ``own`` set, through the
library's entry points.

The 4-bit cache: blocks of 16 channels of one token and head, each value an e2m1
number times the block's e4m3 scale.  uint8 [num_pages, Hkv, bytes] with, per
page of P tokens and head, the codes of K as [d/32, P, 16] (byte y of chunk c:
channels 32c + 2y in the low and 32c + 2y + 1 in the high four bits), its scales
[P, d/16], and both again for V.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step: 64 new tokens, normed, rotated, into the cache, and what it holds of them
        dict(name="append_decode64", op="append", B=64, n=1, Hq=32, Hkv=8, d=128, rot=128, inter=False, norm=True,
             page=64, layer=False, varlen=False, far=16384),
        # the prefill of a 32K prompt: layer layout and cache in one pass, the cache read back
        dict(name="append_prefill32k", op="append", B=1, n=32768, Hq=32, Hkv=8, d=128, rot=128, inter=False, norm=True,
             page=64, layer=True, varlen=False, far=0),
        # a packed batch of ragged prompts, half of each head rotated in interleaved pairs, cache only
        dict(name="append_varlen", op="append", B=37, n=2001, Hq=32, Hkv=8, d=128, rot=64, inter=True, norm=True,
             page=16, layer=False, varlen=True, far=0),
        # a cached document of 128K tokens read back: the prefix of a prompt that continues it
        dict(name="gather_128k", op="gather", B=1, n=131072, lo=131072, Hkv=8, d=128, page=64),
        # prefixes of a ragged batch, small pages, heads of 64
        dict(name="gather_ragged", op="gather", B=37, n=9001, lo=563, Hkv=8, d=64, page=16),
        # smallest attention call: one request of the small layer, one token
        dict(name="kv4_one", op="kv4", S=1, n=1, Hq=2, Hkv=1, d=64, lo=2047, hi=2047, page=16, mask=False,
             ragged=False, sink=0, window=0),
        # a decode step of the 64-request batch
        dict(name="kv4_decode64", op="kv4", S=64, n=1, Hq=32, Hkv=8, d=128, lo=1024, hi=16384, page=64, mask=False,
             ragged=False, sink=0, window=0),
        # speculative step: ragged trees of up to 48 drafted tokens, small pages
        dict(name="kv4_draft48", op="kv4", S=16, n=48, Hq=32, Hkv=8, d=128, lo=4096, hi=32768, page=16, mask=True,
             ragged=True, sink=0, window=0),
        # one document of a million tokens, a chain of five drafted tokens
        dict(name="kv4_1m", op="kv4", S=1, n=5, Hq=32, Hkv=8, d=128, lo=1048571, hi=1048571, page=64, mask=False,
             ragged=False, sink=0, window=0),
        # a decode step of the 64-request batch through the mixed layer's sink and window
        dict(name="window_decode64", op="window", S=64, n=1, Hq=32, Hkv=8, d=128, lo=1024, hi=16384, page=64,
             mask=False, ragged=False, sink=128, window=1024),
        # ragged trees through the small layer's sink and window, small pages
        dict(name="window_draft48", op="window", S=16, n=48, Hq=32, Hkv=8, d=128, lo=4096, hi=32768, page=16,
             mask=True, ragged=True, sink=64, window=512),
        # the next 1024 tokens of a 128K prompt
        dict(name="window_chunk", op="window", S=1, n=1024, Hq=32, Hkv=8, d=128, lo=131072, hi=131072, page=128,
             mask=False, ragged=False, sink=128, window=1024),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "gather", "kv4", "kv4", "window"])
    heads = rng.choice([(2, 1), (32, 8), (8, 8), (16, 2), (5, 5), (12, 4), (7, 1)])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        varlen = rng.random() < 0.4
        B = _logint(rng, 1, 64)
        n = _logint(rng, 1, max(1, 60000 // (B * max(1, heads[0] // 4))))
        rot = rng.choice([d, d, d // 2, 16, 48])
        return dict(op=op, B=B, n=n, Hq=heads[0], Hkv=heads[1], d=d, rot=rot, inter=rng.random() < 0.4,
                    norm=rng.random() < 0.7, page=page, layer=rng.random() < 0.5, varlen=varlen,
                    far=rng.choice([0, 16384, 1 << 20]))
    if op == "gather":
        B = _logint(rng, 1, 64)
        n = _logint(rng, 1, max(1, 1000000 // (B * heads[1])))
        return dict(op=op, B=B, n=n, lo=max(1, n // rng.randint(1, 16)), Hkv=heads[1], d=d, page=page)
    S = _logint(rng, 1, 64)
    n = _logint(rng, 1, 100)
    most = min(131072, 400000 // S, (1 << 30) // (S * heads[0] * n))
    hi = _logint(rng, 1, max(1, most))
    windowed = op == "window" or rng.random() < 0.3
    return dict(op=op, S=S, n=n, Hq=heads[0], Hkv=heads[1], d=d, lo=max(1, hi // rng.randint(1, 8)), hi=hi, page=page,
                mask=rng.random() < 0.6, ragged=rng.random() < 0.5, sink=rng.choice([0, 4, 64, 128]) if windowed else 0,
                window=_logint(rng, 16, 4096) if windowed else 0)


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """(lengths, new tokens) of the requests of a case: its own, whatever the seed, so that outputs keep their shapes."""
    r = np.random.default_rng(11)
    if case["op"] == "append":
        B, n = case["B"], case["n"]
        return _lengths(r, B, max(1, n // 16), n) if case["varlen"] else np.full(B, n), None
    if case["op"] == "gather":
        return _lengths(r, case["B"], case["lo"], case["n"]), None
    S, T = case["S"], case["n"]
    lens = _lengths(r, S, case["lo"], case["hi"])
    return lens, r.integers(_ceil(T, 2), T + 1, S) if case["ragged"] else np.full(S, T)


def _lengths(r, S, lo, hi):
    """Log-uniform lengths in [lo, hi]."""
    x = np.exp(r.uniform(math.log(lo), math.log(hi + 0.999), S))
    return np.clip(x.astype(np.int64), lo, hi)


def _ceil(a, b):
    return -(-a // b)


def _trees(r, S, n):
    """Random parents: ancestor bits [S, n, ceil(n/32)] and depths [S, n] of S trees of n drafted tokens."""
    anc = np.zeros((S, n, n), bool)
    depth = np.zeros((S, n), np.int32)
    rows = np.arange(S)
    for i in range(n):
        if i > 0:
            par = r.integers(-1, i, S) if i > 1 else np.zeros(S, np.int64)
            has = par >= 0
            anc[has, i] = anc[rows[has], par[has]]
            depth[has, i] = depth[rows[has], par[has]] + 1
        anc[:, i, i] = True
    words = _ceil(n, 32)
    padded = np.zeros((S, n, words * 32), bool)
    padded[:, :, :n] = anc
    bits = (padded.reshape(S, n, words, 32).astype(np.uint32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
    return bits.view(np.int32), depth


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _table(r, lens, page, max_pages, num_pages):
    """A page table whose pages lie anywhere in the pool."""
    perm = r.permutation(num_pages)
    table = np.full((len(lens), max_pages), -1, np.int64)
    used = 0
    for s, x in enumerate(lens):
        p = _ceil(int(x), page)
        table[s, :p] = perm[used:used + p]
        used += p
    return table


def _random_cache(g, num_pages, Hkv, page, d):
    """A pool of 4-bit pages: equally likely codes (near those of normal values), scales around 0.35, some keys large."""
    h, s = page * d // 2, page * d // 16
    data = torch.randint(0, 256, (num_pages, Hkv, 2 * (h + s)), generator=g, device=DEV, dtype=torch.uint8)
    for off in (h, 2 * h + s):
        scale = 0.35 * torch.exp(0.3 * torch.randn(num_pages, Hkv, s, generator=g, device=DEV))
        if off == h:
            scale[::7, :, :d // 16] *= 4.0  # keys that queries look at: softmax rows with peaks
        data[..., off:off + s] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    return data


def _prepare_append(case, r, g):
    B, n, Hq, Hkv, d, page = (case[k] for k in ("B", "n", "Hq", "Hkv", "d", "page"))
    lens, _ = _sizes(case)
    tok = int(lens.sum())
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = torch.randn(tok, (Hq + 2 * Hkv) * d, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((Hq + 2 * Hkv) * d, generator=g, device=DEV))  # channels of unequal size
    x = x.to(torch.bfloat16)
    start = r.integers(0, case["far"] + 1, B)
    pos = np.repeat(start, lens) + np.arange(tok) - np.repeat(cu[:-1], lens)
    pages = [_ceil(int(v), page) for v in lens]
    num_pages = sum(pages) + 3
    table = _table(r, lens, page, max(pages), num_pages)
    i = np.arange(tok) - np.repeat(cu[:-1], lens)
    slots = table[np.repeat(np.arange(B), lens), i // page] * page + i % page
    w = (1 + 0.3 * torch.randn(2, d, generator=g, device=DEV)).to(torch.bfloat16)
    held = torch.zeros(2, B, Hkv, int(lens.max()), d, dtype=torch.bfloat16, device=DEV)
    return dict(x=x, Hq=Hq, Hkv=Hkv, d=d, B=B, n=n, cu=[int(v) for v in cu], cu_dev=_i32(cu), lens=_i32(lens), tok=tok,
                positions=_i32(pos), slots=_i32(slots), table=_i32(table), w=w, page=page, rot=case["rot"],
                data=_random_cache(g, num_pages, Hkv, page, d), inter=case["inter"], norm=case["norm"],
                layer=case["layer"], varlen=case["varlen"], theta=500000.0, eps=1e-6, held_k=held[0], held_v=held[1])


def _prepare_gather(case, r, g):
    B, n, Hkv, d, page = (case[k] for k in ("B", "n", "Hkv", "d", "page"))
    lens, _ = _sizes(case)
    num_pages = int(sum(_ceil(int(x), page) for x in lens)) + 3
    table = _table(r, lens, page, _ceil(n, page), num_pages)
    held = torch.zeros(2, B, Hkv, n, d, dtype=torch.bfloat16, device=DEV)
    return dict(data=_random_cache(g, num_pages, Hkv, page, d), table=_i32(table), lens=_i32(lens), page=page, d=d,
                held_k=held[0], held_v=held[1])


def _prepare_attend(case, r, g):
    S, n, Hq, Hkv, d, page = (case[k] for k in ("S", "n", "Hq", "Hkv", "d", "page"))
    ctx, tl = _sizes(case)
    lens = ctx + tl
    num_pages = int(sum(_ceil(int(x), page) for x in lens)) + 3
    table = _table(r, lens, page, _ceil(case["hi"] + n, page), num_pages)
    mask, depth = _trees(r, S, n) if case["mask"] else (None, None)
    st = dict(table=_i32(table), lens=_i32(lens), tree_len=_i32(tl) if case["ragged"] else None,
              mask=None if mask is None else _i32(mask), depth=None if mask is None else _i32(depth),
              longest=int(lens.max()), page=page, d=d, sink=case["sink"], window=case["window"],
              o=torch.zeros(S, Hq, n, d, dtype=torch.bfloat16, device=DEV), lse=torch.zeros(S, Hq, n, device=DEV))
    q = torch.randn(S, Hkv, Hq // Hkv, n, d, generator=g, device=DEV)
    if case["op"] == "kv4":
        st["data"] = _random_cache(g, num_pages, Hkv, page, d)
    else:
        u = torch.randn(Hkv, 1, d, generator=g, device=DEV)
        k = torch.randn(num_pages, Hkv, page, d, generator=g, device=DEV)
        k[::7, :, :1] += 2.0 * u  # keys that every query looks at
        q += 0.7 * u[:, None]
        st["k_pages"] = k.to(torch.bfloat16)
        st["v_pages"] = torch.randn(num_pages, Hkv, page, d, generator=g, device=DEV).to(torch.bfloat16)
    st["q"] = q.reshape(S, Hq, n, d).to(torch.bfloat16)
    return st


def prepare(case, seed):
    r = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    make = {"append": _prepare_append, "gather": _prepare_gather, "kv4": _prepare_attend, "window": _prepare_attend}
    st = make[case["op"]](case, r, g)
    st["op"] = case["op"]
    return st


# ------------------------------------------------------------------ plain forms
def _parts(data, page, d, which):
    """The codes [.., d/32, page, 16] and the scales [.., page, d/16] of K (which = 0) or V (1) in pages [.., bytes]."""
    h, s = page * d // 2, page * d // 16
    off = which * (h + s)
    return (data[..., off:off + h].unflatten(-1, (d // 32, page, 16)),
            data[..., off + h:off + h + s].unflatten(-1, (page, d // 16)))


def _held(data, page, d, which):
    """The values that pages [.., bytes] hold, fp32 [.., page, d]."""
    codes, scales = _parts(data, page, d, which)
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).transpose(-3, -2).flatten(-2)
    scales = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (table[x.int()].unflatten(-1, (d // 16, 16)) * scales[..., None]).flatten(-2)


def _quantise(x):
    """fp64 values [.., d] -> (codes uint8 [.., d], scales e4m3 [.., d/16])."""
    x = x.unflatten(-1, (-1, 16))
    a = (x.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0)
    step = torch.exp2((torch.frexp(a)[1] - 4).clamp(min=-9).double())  # of four significant bits, 2^-9 at least
    scale = torch.round(a / step) * step
    t = torch.where(scale > 0, x.abs() / scale, 0.0)
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=DEV)
    border[1::2] = torch.nextafter(border[1::2], torch.zeros_like(border[1::2]))  # between two codes: the even one
    code = torch.bucketize(t, border).to(torch.uint8)
    return (code | (torch.signbit(x).to(torch.uint8) << 3)).flatten(-2), scale[..., 0].float().to(torch.float8_e4m3fn)


def _store(st, slots, which, x):
    """Tokens x [tokens, Hkv, d] (fp64) to their slots of the 4-bit cache."""
    page, d = st["page"], st["d"]
    codes, scales = _quantise(x)
    c = codes.unflatten(-1, (d // 32, 16, 2))
    dst_c, dst_s = _parts(st["data"], page, d, which)
    pg, off = slots // page, slots % page
    dst_c[pg, :, :, off] = c[..., 0] | (c[..., 1] << 4)
    dst_s[pg, :, off] = scales.view(torch.uint8)


def _norm_rope(st, x, w, dtype):
    """Heads x [tokens, H, d] normed and rotated in `dtype` (not rounded)."""
    rot, inter = st["rot"], st["inter"]
    x = x.to(dtype)
    if st["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + st["eps"]) * w.to(dtype)
    f = st["theta"] ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=DEV) / rot)
    ang = st["positions"].double()[:, None, None] * f
    cos, sin = ang.cos().to(dtype), ang.sin().to(dtype)
    a = x[..., :rot].unflatten(-1, (rot // 2, 2)) if inter else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.stack([a[..., 0] * cos - a[..., 1] * sin, a[..., 1] * cos + a[..., 0] * sin], -1)
    return torch.cat([(y if inter else y.transpose(-1, -2)).flatten(-2), x[..., rot:]], -1)


def _to_layer(st, x):
    """Token-major [tokens, H, d] into the layer layout: [B, H, n, d], or one [H, n_s, d] block per sequence."""
    H = x.shape[1]
    if not st["varlen"]:
        return x.view(st["B"], st["n"], H, -1).transpose(1, 2).contiguous()
    s = torch.repeat_interleave(torch.arange(st["B"], device=DEV), st["lens"], output_size=st["tok"])
    t0 = st["cu_dev"].long()[s]
    i = torch.arange(st["tok"], device=DEV) - t0
    rows = (H * t0 + i)[:, None] + torch.arange(H, device=DEV)[None] * st["lens"].long()[s][:, None]
    out = torch.empty(st["tok"] * H, x.shape[-1], dtype=x.dtype, device=DEV)
    out[rows.reshape(-1)] = x.reshape(-1, x.shape[-1])
    return out.reshape(-1)


def _plain_gather(st):
    page, d = st["page"], st["d"]
    n = st["held_k"].shape[2]
    ids = st["table"][:, :_ceil(n, page)].long().clamp(min=0)
    live = (torch.arange(n, device=DEV) < st["lens"].long()[:, None])[:, None, :, None]
    for which, name in ((0, "held_k"), (1, "held_v")):
        x = _held(st["data"][ids], page, d, which).transpose(1, 2).flatten(2, 3)[:, :, :n]
        st[name].copy_(torch.where(live, x.to(torch.bfloat16), st[name]))
    return dict(held_k=st["held_k"], held_v=st["held_v"])


def _plain_append(st):
    Hq, Hkv, d = st["Hq"], st["Hkv"], st["d"]
    q, k, v = st["x"].view(-1, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], 1)
    out = dict(q=_to_layer(st, _norm_rope(st, q, st["w"][0], torch.float32).to(torch.bfloat16)))
    k = _norm_rope(st, k, st["w"][1], torch.float64)  # in 64 bits: values next to a border of two codes
    slots = st["slots"].long()
    _store(st, slots, 0, k)
    _store(st, slots, 1, v.double())
    if st["layer"]:
        out |= dict(k=_to_layer(st, k.to(torch.bfloat16)), v=_to_layer(st, v))
    return out | _plain_gather(st)


def _plain_attend(st):
    q, table, page, window, sink = st["q"], st["table"], st["page"], st["window"], st["sink"]
    S, Hq, n, d = q.shape
    Hkv = st["data" if st["op"] == "kv4" else "k_pages"].shape[1]
    lens = st["lens"].long()[:, None]
    tl = torch.full_like(lens, n) if st["tree_len"] is None else st["tree_len"].long()[:, None]
    ctx = lens - tl
    # key positions [S, L]: all of them, or the first ones and those that the window of the first row reaches
    if window and sink + window + n < st["longest"]:
        first = torch.arange(sink, device=DEV).expand(S, sink)
        lo = (ctx - window + 1).clamp(min=0)
        key = torch.cat([first, lo.clamp(min=sink) + torch.arange(window + n - 1, device=DEV)], 1)
    else:
        key = torch.arange(st["longest"], device=DEV).expand(S, -1)
    there = key < lens
    at = torch.where(there, key, 0)
    pages = torch.gather(table, 1, at // page).long()
    if st["op"] == "kv4":
        def rows(which):
            ids = table[:, :_ceil(st["longest"], page)].long().clamp(min=0)
            if key.shape[1] == st["longest"]:
                return _held(st["data"][ids], page, d, which).transpose(1, 2).flatten(2, 3)[:, :, :st["longest"]]
            codes, scales = _parts(st["data"], page, d, which)
            one = torch.cat([codes[pages, :, :, at % page].flatten(-2), scales[pages, :, at % page]], -1)
            pad = torch.cat([one, one], -1)  # a page of one token
            return _held(pad, 1, d, 0).squeeze(-2).transpose(1, 2)
        k, v = rows(0), rows(1)
    else:
        k, v = (st[name][pages, :, at % page].transpose(1, 2).float() for name in ("k_pages", "v_pages"))
    key, there = key[:, None], there[:, None]
    ctx, tl = ctx[:, :, None], tl[:, :, None]
    row = torch.arange(n, device=DEV)[None, :, None]
    rel = key - ctx
    if st["mask"] is None:
        seen, ahead = (rel <= row).expand(S, n, -1), row
    else:
        words = torch.gather(st["mask"], 2, (rel.clamp(0, n - 1) // 32).expand(S, n, -1))
        seen = (rel < 0) | ((words >> (rel.clamp(min=0) % 32)) & 1).bool()
        ahead = st["depth"].long()[:, :, None]
    if window:
        near = (rel > ahead - window) | (key < sink)
        seen = seen & (near if st["mask"] is None else near | (rel >= 0))
    seen = (seen & there)[:, None, None]
    s = (q.float().view(S, Hkv, -1, d) @ k.transpose(2, 3)).view(S, Hkv, Hq // Hkv, n, -1) / math.sqrt(d)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    v = torch.where(there[..., None], v, 0.0)
    o = ((e / z).view(S, Hkv, Hq // Hkv * n, -1) @ v).view(S, Hq, n, d).to(torch.bfloat16)
    live = (row < tl)[:, None]
    st["o"].copy_(torch.where(live, o, st["o"]))
    st["lse"].copy_(torch.where(live[..., 0], (m + z.log()).view(S, Hq, n), st["lse"]))
    return dict(o=st["o"], lse=st["lse"])


# ------------------------------------------------------------------ one pass
def _own_gather(st, msa, pages):
    msa.kv4_gather(pages, st["table"], st["lens"], st["held_k"].shape[2], k=st["held_k"], v=st["held_v"])
    return dict(held_k=st["held_k"], held_v=st["held_v"])


def _own(st):
    import long_context_prefill_gb300 as msa

    op = st["op"]
    if op == "window":
        msa.attn_tree_window(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"], st["sink"], st["window"],
                             tree_len=st["tree_len"], tree_mask=st["mask"], depth=st["depth"], o=st["o"], lse=st["lse"])
        return dict(o=st["o"], lse=st["lse"])
    pages = msa.KV4Pages(st["data"], st["page"], st["d"])
    if op == "gather":
        return _own_gather(st, msa, pages)
    if op == "kv4":
        msa.attn_tree_kv4(st["q"], pages, st["table"], st["lens"], sink=st["sink"], window=st["window"],
                          tree_len=st["tree_len"], tree_mask=st["mask"], depth=st["depth"] if st["window"] else None,
                          o=st["o"], lse=st["lse"])
        return dict(o=st["o"], lse=st["lse"])
    Hq, Hkv, d = st["Hq"], st["Hkv"], st["d"]
    cfg = msa.rope_cfg(rot_dim=st["rot"], theta=st["theta"], interleaved=st["inter"], norm=st["norm"], eps=st["eps"],
                       q_weight=st["w"][0], k_weight=st["w"][1])
    q, k, v = st["x"].view(-1, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], 1)
    keep = dict(positions=st["positions"], layer_kv=st["layer"])
    if st["varlen"]:
        q, k, v = msa.qk_norm_rope_varlen_kv4(q, k, v, st["cu"], cfg, pages, st["slots"], **keep)
    else:
        q, k, v = (t.unflatten(0, (st["B"], st["n"])) for t in (q, k, v))
        q, k, v = msa.qk_norm_rope_kv4(q, k, v, cfg, pages, st["slots"], **keep)
    out = dict(q=q) | (dict(k=k, v=v) if st["layer"] else {})
    return out | _own_gather(st, msa, pages)


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "gather": _plain_gather, "kv4": _plain_attend, "window": _plain_attend}[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, add = _sizes(case)
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    held = 2 * (d // 2 + d // 16)  # bytes of a token of a head, K and V
    if case["op"] == "gather":
        keys = int(lens.sum())
        return dict(bytes=keys * Hkv * (held + 4 * d) + keys // page * 4, flops=2 * keys * Hkv * d)
    if case["op"] == "append":
        tok, Hq = int(lens.sum()), case["Hq"]
        heads = (Hq + 2 * Hkv) + Hq + (2 * Hkv if case["layer"] else 0) + 2 * Hkv  # in, out, read back
        return dict(bytes=tok * (heads * d * 2 + Hkv * held + 8), flops=tok * ((Hq + Hkv) * d * (7 if case["norm"] else 3) + 6 * Hkv * d))
    Hq, rows = case["Hq"], int(add.sum()) * case["Hq"]
    keys, pairs = 0, 0
    for c, t in zip(lens, add):
        c, t = int(c), int(t)
        if case["window"]:
            lo = max(0, c - case["window"] + 1)
            k = min(case["sink"], lo) + c + t - lo
            p = min(k, case["sink"] + case["window"]) * t
        else:
            k, p = c + t, (c + t) * t
        keys, pairs = keys + k, pairs + p
    held = held if case["op"] == "kv4" else 4 * d
    return dict(bytes=keys * Hkv * held + rows * (d * 4 + 4) + keys // page * 4, flops=4 * pairs * Hq * d)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "gather":
        return _exact_gather(st, st["data"])
    return _exact_attend(st)


def _exact_values(data, page, d, which):
    """Values held by pages [.., bytes], in fp64 [.., page, d], from the bits of codes and scales."""
    half, size = d // 2, page * (d // 2 + d // 16)
    x = data[..., which * size:(which + 1) * size]
    lead = x.shape[:-1]
    b = x[..., :page * half].reshape(*lead, d // 32, page, 16).transpose(-3, -2).reshape(*lead, page, half).int()
    code = torch.empty(*lead, page, d, dtype=torch.int32, device=DEV)
    code[..., 0::2], code[..., 1::2] = b % 16, b // 16
    exp, man = (code // 2) % 4, code % 2
    mag = torch.where(exp == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2(exp.double() - 1))
    s = x[..., page * half:].reshape(*lead, page, d // 16).int()
    e, m = (s // 8) % 16, s % 8
    scale = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8.0) * torch.exp2(e.double() - 7))
    return torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(16, -1)


def _exact_gather(st, data):
    page, d = st["page"], st["d"]
    out = [st["held_k"].double(), st["held_v"].double()]
    for b, L in enumerate(st["lens"].tolist()):
        ids = st["table"][b, :_ceil(L, page)].long()
        for which in (0, 1):
            x = _exact_values(data[ids], page, d, which)
            out[which][b, :, :L] = x.transpose(0, 1).flatten(1, 2)[:, :L]
    return dict(held_k=out[0], held_v=out[1])


def _exact_blocks(x):
    """Every block of 16 of fp64 x rounded to its scale and codes, as values."""
    b = x.reshape(-1, 16)
    a = (b.abs().amax(1) / 6).clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6)))
    scale = (torch.round(a / torch.exp2(e - 3)) * torch.exp2(e - 3)).clamp(max=448.0)[:, None]  # ties to even
    t = torch.where(scale > 0, b.abs() / scale, 0.0)
    step = torch.where(t < 2, 0.5, torch.where(t < 4, 1.0, 2.0))
    return (torch.copysign((torch.round(t / step) * step).clamp(max=6.0), b) * scale).reshape(x.shape)


def _exact_append(st):
    if st["x"].numel() > 1 << 31:
        return None
    Hq, Hkv, d, rot = st["Hq"], st["Hkv"], st["d"], st["rot"]
    half = rot // 2
    x = st["x"].double().view(st["tok"], Hq + 2 * Hkv, d)
    ang = torch.outer(st["positions"].double(), torch.tensor([st["theta"] ** (-2 * i / rot) for i in range(half)],
                                                             dtype=torch.float64, device=DEV))
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    first = torch.arange(0, rot, 2, device=DEV) if st["inter"] else torch.arange(half, device=DEV)
    second = first + (1 if st["inter"] else half)
    parts = []
    for h0, h1, w in ((0, Hq, st["w"][0]), (Hq, Hq + Hkv, st["w"][1]), (Hq + Hkv, Hq + 2 * Hkv, None)):
        y = x[:, h0:h1]
        if w is not None:
            if st["norm"]:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + st["eps"]) * w.double()
            z = y.clone()
            z[..., first] = y[..., first] * cos - y[..., second] * sin
            z[..., second] = y[..., second] * cos + y[..., first] * sin
            y = z
        parts.append(y)

    def layer(y):
        seqs = [y[a:b].transpose(0, 1) for a, b in zip(st["cu"][:-1], st["cu"][1:])]
        return torch.cat([t.reshape(-1) for t in seqs]) if st["varlen"] else torch.stack(seqs)

    out = dict(q=layer(parts[0]))
    if st["layer"]:
        out |= dict(k=layer(parts[1]), v=layer(parts[2]))
    for name, y in (("held_k", parts[1]), ("held_v", parts[2])):
        out[name] = st[name].double()
        y = _exact_blocks(y)
        for b, (c0, c1) in enumerate(zip(st["cu"][:-1], st["cu"][1:])):
            out[name][b, :, :c1 - c0] = y[c0:c1].transpose(0, 1)
    return out


def _exact_attend(st):
    S, Hq, n, d = st["q"].shape
    kv4, page = st["op"] == "kv4", st["page"]
    Hkv = st["data" if kv4 else "k_pages"].shape[1]
    g = Hq // Hkv
    lens = st["lens"].tolist()
    tls = [n] * S if st["tree_len"] is None else st["tree_len"].tolist()
    if sum(a * b for a, b in zip(lens, tls)) * Hq * d > 1 << 42:
        return None
    o, lse = st["o"].double(), st["lse"].double()
    words = None if st["mask"] is None else st["mask"].cpu().numpy().view(np.uint32)
    for b in range(S):
        L, T = lens[b], tls[b]
        C = L - T
        ids = st["table"][b, :_ceil(L, page)].long()
        see = torch.ones(T, L, dtype=torch.bool, device=DEV)
        if words is None:
            see[:, C:] = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
        else:
            bits = np.unpackbits(words[b].view(np.uint8).reshape(n, -1), axis=1, bitorder="little")[:T, :T]
            see[:, C:] = torch.from_numpy(bits.astype(bool)).to(DEV)
        if st["window"]:
            for i in range(T):
                p = C + (i if words is None else int(st["depth"][b, i]))
                end = max(0, min(L if words is None else C, p - st["window"] + 1))
                see[i, min(st["sink"], end):end] = False
        for h in range(Hkv):
            if kv4:
                k, v = (_exact_values(st["data"][ids, h], page, d, w).reshape(-1, d)[:L] for w in (0, 1))
            else:
                k, v = (st[name][ids, h].reshape(-1, d)[:L].double() for name in ("k_pages", "v_pages"))
            s = torch.einsum("gid,jd->gij", st["q"][b, h * g:(h + 1) * g, :T].double(), k) * d ** -0.5
            s = s.masked_fill(~see, -math.inf)
            lse[b, h * g:(h + 1) * g, :T] = torch.logsumexp(s, -1)
            o[b, h * g:(h + 1) * g, :T] = torch.softmax(s, -1) @ v
    return dict(o=o, lse=lse)
