"""Cases for the paged-cache operators: page tables and slot maps built on the
GPU, per-head norms of q and k with the rotation, and attention of drafted
tokens over the paged cache.

``run`` computes a case in elementary torch operations (32 bits, 64 for the
angles) or, with ``own`` set, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a batch of 64 requests (the varlen batch's lengths), the tokens rolled back after it
        dict(name="tables_decode64", op="tables", S=64, lo=1024, hi=16384, add=1, page=64, padded=True, tree=False),
        # the whole varlen batch prefilled at once into an empty cache, and freed again
        dict(name="tables_prefill", op="tables", S=64, lo=1024, hi=16384, add=0, page=16, padded=False, tree=False),
        # a draft step of many requests: ragged trees, positions by depth, small pages
        dict(name="tables_tree1021", op="tables", S=1021, lo=256, hi=8192, add=48, page=16, padded=True, tree=True),
        # one decode step: 64 new tokens, normed, rotated, K and V into the cache
        dict(name="rope_decode64", op="rope", B=64, n=1, Hq=32, Hkv=8, d=128, rot=128, inter=False, norm=True,
             page=64, layer=False, varlen=False, far=16384),
        # the prefill of a 32K prompt: layer layout and cache in one pass
        dict(name="rope_prefill32k", op="rope", B=1, n=32768, Hq=32, Hkv=8, d=128, rot=128, inter=False, norm=True,
             page=64, layer=True, varlen=False, far=0),
        # a packed batch of ragged prompts, half of each head rotated in interleaved pairs
        dict(name="rope_varlen", op="rope", B=37, n=9001, Hq=32, Hkv=8, d=128, rot=64, inter=True, norm=True,
             page=16, layer=True, varlen=True, far=0),
        # the small layer, no norm, positions far into a long document
        dict(name="rope_small", op="rope", B=1, n=2048, Hq=2, Hkv=1, d=64, rot=64, inter=False, norm=False,
             page=16, layer=True, varlen=False, far=1 << 20),
        # smallest attention call: one request of the small layer, one token
        dict(name="tree_one", op="tree", S=1, n=1, Hq=2, Hkv=1, d=64, lo=2047, hi=2047, page=16, mask=False,
             ragged=False),
        # a decode step of the 64-request batch
        dict(name="tree_decode64", op="tree", S=64, n=1, Hq=32, Hkv=8, d=128, lo=1024, hi=16384, page=64, mask=False,
             ragged=False),
        # speculative step: ragged trees of up to 48 drafted tokens, small pages
        dict(name="tree_draft48", op="tree", S=16, n=48, Hq=32, Hkv=8, d=128, lo=4096, hi=32768, page=16, mask=True,
             ragged=True),
        # one 128K document, a tree of 32
        dict(name="tree_128k", op="tree", S=1, n=32, Hq=32, Hkv=8, d=128, lo=131072, hi=131072, page=128, mask=True,
             ragged=False),
        # one document of a million tokens, a chain of five drafted tokens
        dict(name="tree_1m", op="tree", S=1, n=5, Hq=32, Hkv=8, d=128, lo=1048571, hi=1048571, page=64, mask=False,
             ragged=False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope", "tree", "tree"])
    if op == "tables":
        S = _logint(rng, 1, 1024)
        padded = rng.random() < 0.6
        hi = _logint(rng, 64, 16384)
        return dict(op="tables", S=S, lo=max(1, hi // rng.randint(1, 32)), hi=hi,
                    add=_logint(rng, 1, 64) if padded else 0, page=rng.choice([16, 32, 64, 128]), padded=padded,
                    tree=padded and rng.random() < 0.5)
    heads = rng.choice([(2, 1), (32, 8), (8, 8), (16, 2), (5, 5), (12, 4), (7, 1)])
    d = rng.choice([64, 128])
    if op == "rope":
        varlen = rng.random() < 0.4
        B = _logint(rng, 1, 64)
        n = _logint(rng, 1, max(1, 100000 // (B * max(1, heads[0] // 4))))
        rot = rng.choice([d, d, d // 2, 16, 48])
        return dict(op="rope", B=B, n=n, Hq=heads[0], Hkv=heads[1], d=d, rot=rot, inter=rng.random() < 0.4,
                    norm=rng.random() < 0.7, page=rng.choice([16, 32, 64, 128]), layer=varlen or rng.random() < 0.6,
                    varlen=varlen, far=rng.choice([0, 16384, 1 << 20]))
    S = _logint(rng, 1, 64)
    n = _logint(rng, 1, 100)
    most = min(131072, 400000 // S, (1 << 30) // (S * heads[0] * n))
    hi = _logint(rng, 1, max(1, most))
    return dict(op="tree", S=S, n=n, Hq=heads[0], Hkv=heads[1], d=d, lo=max(1, hi // rng.randint(1, 8)), hi=hi,
                page=rng.choice([16, 32, 64, 128]), mask=rng.random() < 0.6, ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _sizes(case):
    """(lengths, new tokens) of the requests of a case: its own, whatever the seed, so that outputs keep their shapes."""
    r = np.random.default_rng(11)
    if case["op"] == "rope":
        B, n = case["B"], case["n"]
        return _lengths(r, B, max(1, n // 16), n) if case["varlen"] else np.full(B, n), None
    S, T = case["S"], case["add"] if case["op"] == "tables" else case["n"]
    lens = _lengths(r, S, case["lo"], case["hi"])
    ragged = case["tree"] if case["op"] == "tables" else case["ragged"]
    return lens, r.integers(_ceil(T, 2), T + 1, S) if ragged else np.full(S, T)


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


def _cu(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(DEV)


def _table(r, lens, page, max_pages, num_pages):
    """A page table whose pages lie anywhere in the pool, and the pages left over."""
    perm = r.permutation(num_pages)
    table = np.full((len(lens), max_pages), -1, np.int64)
    used = 0
    for s, x in enumerate(lens):
        p = _ceil(int(x), page)
        table[s, :p] = perm[used:used + p]
        used += p
    return table, perm[used:]


def _prepare_tables(case, r):
    S, page, T = case["S"], case["page"], case["add"]
    lens, add = _sizes(case)
    if case["padded"]:
        old = lens
        new, cap = old + add, S * T
    else:
        old, new, cap = np.zeros(S, np.int64), lens, int(lens.sum())
    max_pages = _ceil(case["hi"] + T, page)
    need = int(sum(_ceil(int(x), page) for x in new))
    num_pages = need + need // 4 + 8
    table, left = _table(r, old, page, max_pages, num_pages)
    stack = np.full(num_pages, -1, np.int64)
    stack[:len(left)] = left
    depth = _i32(_trees(r, S, T)[1]) if case["tree"] else None
    return dict(page_table=_i32(table), seq_len=_i32(old), free_pages=_i32(stack),
                state=_i32(np.array([len(left), 0, 0, 0])), old=_i32(old), new=_i32(new), depth=depth, page=page,
                T=T if case["padded"] else 0, cap=cap)


def _prepare_rope(case, r, g):
    B, n, Hq, Hkv, d, page = (case[k] for k in ("B", "n", "Hq", "Hkv", "d", "page"))
    lens, _ = _sizes(case)
    tok = int(lens.sum())
    cu = _cu(lens)
    x = torch.randn(tok, (Hq + 2 * Hkv) * d, generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((Hq + 2 * Hkv) * d, generator=g, device=DEV))  # channels of unequal size
    x = x.to(torch.bfloat16)
    start = r.integers(0, case["far"] + 1, B)
    pos = np.repeat(start, lens) + np.arange(tok) - np.repeat(cu[:-1], lens)
    pages = [_ceil(int(v), page) for v in lens]
    num_pages = sum(pages) + 3
    table, _ = _table(r, lens, page, max(pages), num_pages)
    i = np.arange(tok) - np.repeat(cu[:-1], lens)
    slots = table[np.repeat(np.arange(B), lens), i // page] * page + i % page
    w = (1 + 0.3 * torch.randn(2, d, generator=g, device=DEV)).to(torch.bfloat16)
    kp = torch.randn(2, num_pages, Hkv, page, d, generator=g, device=DEV).to(torch.bfloat16)
    return dict(x=x, Hq=Hq, Hkv=Hkv, d=d, B=B, n=n, cu=[int(v) for v in cu], cu_dev=_i32(cu), lens=_i32(lens), tok=tok,
                positions=_i32(pos), slots=_i32(slots), w=w, k_pages=kp[0], v_pages=kp[1], page=page, rot=case["rot"],
                inter=case["inter"], norm=case["norm"], layer=case["layer"], varlen=case["varlen"], theta=500000.0,
                eps=1e-6)


def _prepare_tree(case, r, g):
    S, n, Hq, Hkv, d, page = (case[k] for k in ("S", "n", "Hq", "Hkv", "d", "page"))
    ctx, tl = _sizes(case)
    lens = ctx + tl
    max_pages = _ceil(case["hi"] + n, page)
    num_pages = int(sum(_ceil(int(x), page) for x in lens)) + 3
    table, _ = _table(r, lens, page, max_pages, num_pages)
    u = torch.randn(Hkv, 1, d, generator=g, device=DEV)
    k = torch.randn(num_pages, Hkv, page, d, generator=g, device=DEV)
    k[::7, :, :1] += 2.0 * u  # keys that every query looks at: softmax rows with peaks
    v = torch.randn(num_pages, Hkv, page, d, generator=g, device=DEV)
    q = torch.randn(S, Hkv, Hq // Hkv, n, d, generator=g, device=DEV) + 0.7 * u[:, None]
    mask = _trees(r, S, n)[0] if case["mask"] else None
    return dict(q=q.reshape(S, Hq, n, d).to(torch.bfloat16), k_pages=k.to(torch.bfloat16), v_pages=v.to(torch.bfloat16),
                page_table=_i32(table), seq_len=_i32(lens), tree_len=_i32(tl) if case["ragged"] else None,
                tree_mask=None if mask is None else _i32(mask), o=torch.zeros(S, Hq, n, d, dtype=torch.bfloat16, device=DEV),
                lse=torch.zeros(S, Hq, n, device=DEV), longest=int(lens.max()), page=page)


def prepare(case, seed):
    r = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = {"tables": lambda: _prepare_tables(case, r), "rope": lambda: _prepare_rope(case, r, g),
          "tree": lambda: _prepare_tree(case, r, g)}[case["op"]]()
    st["op"] = case["op"]
    return st


# ------------------------------------------------------------------ plain forms
def _plain_tables(st, new_len, tokens):
    """One resize of every request: pages released and granted in (request, page) order from a stack."""
    table, stack, state, page = st["page_table"], st["free_pages"], st["state"], st["page"]
    S, max_pages = table.shape
    N = stack.shape[0]
    old, new = st["seq_len"].long(), new_len.long()
    valid = (new >= 0) & (new <= max_pages * page)
    if st["T"] and tokens:
        valid &= new - old <= st["T"]
    tok = torch.where(valid, (new - old).clamp(min=0), 0)
    po, pn = (old + page - 1) // page, (new + page - 1) // page
    grow = torch.where(valid, (pn - po).clamp(min=0), 0)
    rel = torch.where(valid, (po - pn).clamp(min=0), 0)
    count, Rl = state[0].long(), rel.sum()
    ok = valid & ((grow == 0) | (grow.cumsum(0) <= count + Rl))
    if tokens and not st["T"]:
        ok &= (tok == 0) | (tok.cumsum(0) <= st["cap"])
    tok = torch.where(ok, tok, 0)
    p = torch.arange(max_pages, device=DEV)[None]
    gm = (ok[:, None] & (p >= po[:, None]) & (p < pn[:, None])).reshape(-1)
    rm = (valid[:, None] & (p >= pn[:, None]) & (p < po[:, None])).reshape(-1)
    gi, ri = gm.long().cumsum(0) - 1, rm.long().cumsum(0) - 1
    G = gm.sum()
    flat = table.reshape(-1)
    freed = torch.full((N + 1,), -1, dtype=torch.int32, device=DEV)
    freed.scatter_(0, torch.where(rm, ri, N), torch.where(rm, flat, -1))
    top = stack[(count - 1 - (gi - Rl)).clamp(0, N - 1)]
    pages = torch.where(gi < Rl, freed[gi.clamp(0, N)], top)
    pushed = torch.cat([stack, stack[:1]])
    pushed.scatter_(0, torch.where(rm & (ri >= G), count + Rl - 1 - ri, N), flat)
    flat.copy_(torch.where(gm, pages, flat))
    stack.copy_(pushed[:N])
    cu = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    cu[1:] = tok.cumsum(0)
    st["seq_len"].copy_(torch.where(ok, new, old))
    state[0] = (count + Rl - G).int()
    state[1] = (~ok).sum().int()
    if not tokens:
        return cu, None, None
    t = torch.arange(st["cap"], device=DEV)
    if st["T"]:
        s, i = t // st["T"], t % st["T"]
        live = i < tok[s]
    else:
        s = torch.searchsorted(cu[1:].contiguous(), t.int(), right=True).clamp(max=S - 1)
        i = t - cu[s]
        live = t < cu[-1]
    at = torch.where(live, old[s] + i, 0)
    slots = torch.where(live, table[s, at // page] * page + at % page, -1).int()
    ahead = i if st["depth"] is None else st["depth"].reshape(-1).long()
    return cu, slots, torch.where(live, old[s] + ahead, -1).int()


def _rms(x, w, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w


def _rotate(x, cos, sin, rot, inter):
    """x [tokens, H, d], cos and sin [tokens, 1, rot/2]."""
    a = x[..., :rot].unflatten(-1, (rot // 2, 2)) if inter else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    y = torch.stack([a[..., 0] * cos - a[..., 1] * sin, a[..., 1] * cos + a[..., 0] * sin], -1)
    y = (y if inter else y.transpose(-1, -2)).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


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


def _norm_rope(st, x, dtype):
    """q, k, v [tokens, H, d] of fused rows x, in `dtype` (not rounded)."""
    Hq, Hkv, d, rot = st["Hq"], st["Hkv"], st["d"], st["rot"]
    q, k, v = x.to(dtype).view(-1, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], 1)
    if st["norm"]:
        q, k = _rms(q, st["w"][0].to(dtype), st["eps"]), _rms(k, st["w"][1].to(dtype), st["eps"])
    f = st["theta"] ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=DEV) / rot)
    ang = st["positions"].double()[:, None, None] * f
    cos, sin = ang.cos().to(dtype), ang.sin().to(dtype)
    return _rotate(q, cos, sin, rot, st["inter"]), _rotate(k, cos, sin, rot, st["inter"]), v


def _plain_rope(st):
    q, k, v = (t.to(torch.bfloat16) for t in _norm_rope(st, st["x"], torch.float32))
    pg, off = st["slots"].long() // st["page"], st["slots"].long() % st["page"]
    st["k_pages"][pg, :, off] = k
    st["v_pages"][pg, :, off] = v
    out = dict(q=_to_layer(st, q), k_pages=st["k_pages"], v_pages=st["v_pages"])
    if st["layer"]:
        out |= dict(k=_to_layer(st, k), v=_to_layer(st, v))
    return out


def _plain_tree(st):
    q, table, page = st["q"], st["page_table"], st["page"]
    S, Hq, n, d = q.shape
    Hkv, L = st["k_pages"].shape[1], st["longest"]
    pages = table[:, :_ceil(L, page)].long().clamp(min=0)
    k = st["k_pages"][pages].transpose(1, 2).reshape(S, Hkv, -1, d)[:, :, :L].float()
    v = st["v_pages"][pages].transpose(1, 2).reshape(S, Hkv, -1, d)[:, :, :L].float()
    lens = st["seq_len"].long()[:, None, None]
    tl = torch.full_like(lens, n) if st["tree_len"] is None else st["tree_len"].long()[:, None, None]
    key = torch.arange(L, device=DEV)[None, None]
    row = torch.arange(n, device=DEV)[None, :, None]
    rel = key - (lens - tl)
    if st["tree_mask"] is None:
        seen = (rel <= row).expand(S, n, L)
    else:
        word = torch.gather(st["tree_mask"], 2, (rel.clamp(0, n - 1) // 32).expand(S, n, L))
        seen = (rel < 0) | ((word >> (rel.clamp(min=0) % 32)) & 1).bool()
    seen = (seen & (key < lens))[:, None, None]
    s = (q.float().view(S, Hkv, -1, d) @ k.transpose(2, 3)).view(S, Hkv, Hq // Hkv, n, L) / math.sqrt(d)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    v = torch.where(key[..., None] < lens[..., None], v, 0.0)
    o = ((e / z).view(S, Hkv, -1, L) @ v).view(S, Hq, n, d).to(torch.bfloat16)
    live = (row < tl)[:, None]
    st["o"].copy_(torch.where(live, o, st["o"]))
    st["lse"].copy_(torch.where(live[..., 0], (m + z.log()).view(S, Hq, n), st["lse"]))
    return dict(o=st["o"], lse=st["lse"])


# ------------------------------------------------------------------ one pass
def _own_tables(st):
    import long_context_prefill_gb300 as msa

    pool = msa.PagePool(st["page_table"], st["seq_len"], st["free_pages"], st["state"], st["page"])
    cu, slots, positions = msa.build_page_tables(pool, st["new"], seq_tokens=st["T"], tok_cap=st["cap"], depth=st["depth"])
    msa.build_page_tables(pool, st["old"])
    return cu, slots, positions


def _own_rope(st):
    import long_context_prefill_gb300 as msa

    Hq, Hkv, d = st["Hq"], st["Hkv"], st["d"]
    cfg = msa.rope_cfg(rot_dim=st["rot"], theta=st["theta"], interleaved=st["inter"], norm=st["norm"], eps=st["eps"],
                       q_weight=st["w"][0], k_weight=st["w"][1])
    q, k, v = st["x"].view(-1, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], 1)
    keep = dict(positions=st["positions"], k_pages=st["k_pages"], v_pages=st["v_pages"], slots=st["slots"],
                layer_kv=st["layer"])
    if st["varlen"]:
        q, k, v = msa.qk_norm_rope_varlen(q, k, v, st["cu"], cfg, **keep)
    else:
        q, k, v = (t.unflatten(0, (st["B"], st["n"])) for t in (q, k, v))
        q, k, v = msa.qk_norm_rope(q, k, v, cfg, **keep)
    out = dict(q=q, k_pages=st["k_pages"], v_pages=st["v_pages"])
    return out | dict(k=k, v=v) if st["layer"] else out


def _own_tree(st):
    import long_context_prefill_gb300 as msa

    msa.attn_tree(st["q"], st["k_pages"], st["v_pages"], st["page_table"], st["seq_len"], tree_len=st["tree_len"],
                  tree_mask=st["tree_mask"], o=st["o"], lse=st["lse"])
    return dict(o=st["o"], lse=st["lse"])


def run(state):
    if state["op"] == "tables":
        if own:
            cu, slots, positions = _own_tables(state)
        else:
            cu, slots, positions = _plain_tables(state, state["new"], True)
            _plain_tables(state, state["old"], False)  # rolled back: the pages return to the stack
        return dict(cu=cu, slots=slots, positions=positions,
                    **{k: state[k] for k in ("page_table", "seq_len", "free_pages", "state")})
    if state["op"] == "rope":
        return _own_rope(state) if own else _plain_rope(state)
    return _own_tree(state) if own else _plain_tree(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    lens, add = _sizes(case)
    if case["op"] == "tables":
        S, page = case["S"], case["page"]
        old, new = (lens, lens + add) if case["padded"] else (0 * lens, lens)
        tok = S * case["add"] if case["padded"] else int(lens.sum())
        pages = int(((new + page - 1) // page - (old + page - 1) // page).sum())
        depth = 4 * tok if case["tree"] else 0
        # lengths, offsets, slots and positions; each page from the stack to the table, and back
        return dict(bytes=2 * 4 * 3 * S + 4 * S + 8 * tok + depth + 2 * 2 * 4 * pages, flops=0)
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        tok = int(lens.sum())
        heads = (Hq + 2 * Hkv) * 2 + (2 * Hkv if case["layer"] else 0)
        return dict(bytes=tok * (heads * d * 2 + 8), flops=tok * (Hq + Hkv) * d * (7 if case["norm"] else 3))
    keys, pairs, rows = int((lens + add).sum()), int(((lens + add) * add).sum()), int(add.sum()) * Hq
    return dict(bytes=keys * Hkv * d * 4 + rows * (d * 4 + 4) + keys // case["page"] * 4, flops=4 * pairs * Hq * d)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    st = prepare(case, seed)
    return _exact_rope(st) if case["op"] == "rope" else _exact_tree(st)


def _exact_rope(st):
    if st["x"].numel() > 1 << 31:
        return None
    Hq, Hkv, d, rot, page = st["Hq"], st["Hkv"], st["d"], st["rot"], st["page"]
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
    out = dict(k_pages=st["k_pages"].double(), v_pages=st["v_pages"].double())
    for name, y in (("k_pages", parts[1]), ("v_pages", parts[2])):
        rows = out[name].transpose(1, 2).reshape(-1, Hkv, d)
        rows[st["slots"].long()] = y
        out[name] = rows.view(-1, page, Hkv, d).transpose(1, 2).contiguous()
    for name, y in (("q", parts[0]), ("k", parts[1]), ("v", parts[2])):
        if name == "q" or st["layer"]:
            seqs = [y[a:b].transpose(0, 1) for a, b in zip(st["cu"][:-1], st["cu"][1:])]
            out[name] = torch.cat([t.reshape(-1) for t in seqs]) if st["varlen"] else torch.stack(seqs)
    return out


def _exact_tree(st):
    S, Hq, n, d = st["q"].shape
    Hkv = st["k_pages"].shape[1]
    g = Hq // Hkv
    lens = st["seq_len"].tolist()
    tls = [n] * S if st["tree_len"] is None else st["tree_len"].tolist()
    if sum(a * b for a, b in zip(lens, tls)) * Hq * d > 1 << 42:
        return None
    o, lse = st["o"].double(), st["lse"].double()
    words = None if st["tree_mask"] is None else st["tree_mask"].cpu().numpy().view(np.uint32)
    for b in range(S):
        L, T = lens[b], tls[b]
        pages = st["page_table"][b, :_ceil(L, st["page"])].long()
        see = torch.ones(T, L, dtype=torch.bool, device=DEV)
        if words is None:
            see[:, L - T:] = torch.ones(T, T, dtype=torch.bool, device=DEV).tril()
        else:
            bits = np.unpackbits(words[b].view(np.uint8).reshape(n, -1), axis=1, bitorder="little")[:T, :T]
            see[:, L - T:] = torch.from_numpy(bits.astype(bool)).to(DEV)
        for h in range(Hkv):
            k = st["k_pages"][pages, h].reshape(-1, d)[:L].double()
            v = st["v_pages"][pages, h].reshape(-1, d)[:L].double()
            s = torch.einsum("gid,jd->gij", st["q"][b, h * g:(h + 1) * g, :T].double(), k) * d ** -0.5
            s = s.masked_fill(~see, -math.inf)
            lse[b, h * g:(h + 1) * g, :T] = torch.logsumexp(s, -1)
            o[b, h * g:(h + 1) * g, :T] = torch.softmax(s, -1) @ v
    return dict(o=o, lse=lse)
