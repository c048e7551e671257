"""Plain references of the paged-cache operators, in 64 bits, and the error
bounds their tests use (test infrastructure only; no library code)."""
import math

import numpy as np
import torch

# Half a step of bf16 (torch.finfo(torch.bfloat16).eps / 2), relative to the value.
BF16_HALF = 2.0 ** -8


# ------------------------------------------------------------------ page tables
def resize(table, seq_len, stack, state, new_len, page, seq_tokens=0, tok_cap=None, depth=None):
    """One call of msa_build_page_tables on int lists, one request after another.
    Updates its arguments; returns (cu, slots, positions), the last two None without token outputs."""
    S, width, N = len(seq_len), len(table[0]), len(stack)
    tokens = bool(seq_tokens) or tok_cap is not None
    pages = lambda x: -(-x // page)  # noqa: E731
    old = list(seq_len)
    valid = [0 <= new_len[s] <= width * page and 0 <= old[s] <= width * page and
             not (seq_tokens and new_len[s] - old[s] > seq_tokens) for s in range(S)]
    released = []
    for s in range(S):
        if valid[s] and new_len[s] < old[s]:
            released += table[s][pages(new_len[s]):pages(old[s])]
    count = state[0]
    fits = count + len(released) <= N
    want_pages = want_tok = granted = refused = 0
    cu, new_pages = [0], {}
    for s in range(S):
        ok = valid[s] and fits
        grow = max(0, pages(new_len[s]) - pages(old[s])) if valid[s] else 0
        tok = max(0, new_len[s] - old[s]) if valid[s] else 0
        want_pages += grow
        want_tok += tok
        if grow and want_pages > count + len(released):
            ok = False
        if tokens and not seq_tokens and tok and want_tok > tok_cap:
            ok = False
        cu.append(cu[-1] + (tok if ok else 0))
        if ok:
            for p in range(pages(old[s]), pages(new_len[s])):
                new_pages[s, p] = released[granted] if granted < len(released) else stack[count - 1 - (granted - len(released))]
                granted += 1
            seq_len[s] = new_len[s]
        else:
            refused += 1
    if fits:
        for r in range(granted, len(released)):
            stack[count + len(released) - 1 - r] = released[r]
        state[0] = count + len(released) - granted
    for (s, p), page_id in new_pages.items():
        table[s][p] = page_id
    state[1] = refused
    if not tokens:
        return cu, None, None
    total = S * seq_tokens if seq_tokens else tok_cap
    slots, positions = [-1] * total, [-1] * total
    for s in range(S):
        for i in range(cu[s + 1] - cu[s]):
            t = s * seq_tokens + i if seq_tokens else cu[s] + i
            at = old[s] + i
            slots[t] = table[s][at // page] * page + at % page
            positions[t] = old[s] + (i if depth is None else depth[t])
    return cu, slots, positions


# ------------------------------------------------------------------ norm and rotation
def norm_rope(x, w, norm, eps, rot, freq, inter, pos, scale=1.0):
    """x [tokens, H, d] (any float type) -> (float64 result, bound on its error before the bf16 rounding)."""
    x = x.double()
    d = x.shape[-1]
    if norm:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
    y = x.clone()
    size = x.abs()
    if rot:
        half = rot // 2
        i = torch.arange(half, device=x.device)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        ang = pos.double()[:, None] * torch.as_tensor(freq, dtype=torch.float64, device=x.device)[None]
        c, s = (torch.cos(ang) * scale)[:, None], (torch.sin(ang) * scale)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        m = (x[..., a].abs() + x[..., b].abs()) * abs(scale)
        size = size.clone()
        size[..., a] = m
        size[..., b] = m
    # fp32: the mean of d squares, a root, a quotient and two products stay below (d/16 + 12) half steps of 2^-24
    # (16 values a lane, then a tree); the angle is exact to pi 2^-25 (an fp32 half turn), sine and cosine to 2 steps,
    # two products and a sum more: 32 half steps of the pair's size cover both
    return y, size * (2.0 ** -24 * 32)


def check_rounded(got, ref, slack, what):
    """got (bf16) is ref, computed within `slack`, rounded once: half a bf16 step of a value within slack of ref."""
    err = (got.double() - ref).abs()
    bound = BF16_HALF * (ref.abs() + slack) + slack + 2.0 ** -133  # smallest bf16 step
    bad = err > bound
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).max()):.3e}"


# ------------------------------------------------------------------ attention over pages
def attend(q, k, v, seen, scale):
    """q [H, rows, d], k / v [L, d] of one KV head, seen [rows, L]: (o, lse) in
    float64 and bounds on the kernel's errors in them.

    Scores: d exact bf16 products summed in fp32, at most d steps of 2^-23 (an
    accumulator that truncates) of the absolute sum; delta, in nats, is that
    and 2^-20 for scaling and exponential.  A weight is off by delta in
    numerator and denominator each and by half a bf16 step (the weights enter
    the second product as bf16); L products summed in fp32 add L steps of 2^-23."""
    q, k, v = q.double(), k.double(), v.double()
    L = k.shape[0]
    s = torch.einsum("hrd,ld->hrl", q, k) * scale
    size = torch.einsum("hrd,ld->hrl", q.abs(), k.abs()) * scale
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    o = torch.einsum("hrl,ld->hrd", p, v)
    a = torch.einsum("hrl,ld->hrd", p, v.abs())
    delta = q.shape[-1] * 2.0 ** -23 * size.masked_fill(~seen, 0.0).amax(-1) + 2.0 ** -20
    o_tol = a * (BF16_HALF + 2 * delta[..., None] + L * 2.0 ** -23) + BF16_HALF * o.abs() + 2.0 ** -100
    lse_tol = delta + L * 2.0 ** -23 + 2.0 ** -21 * (1 + torch.where(torch.isinf(lse), 0.0, lse.abs()))
    return o, lse, o_tol, lse_tol


def unpack_mask(words, n):
    """[.., n, ceil(n/32)] int32 words -> [.., n, n] bool."""
    w = np.ascontiguousarray(words.cpu().numpy()).view(np.uint8)
    bits = np.unpackbits(w, axis=-1, bitorder="little")[..., :n]
    return torch.from_numpy(bits.astype(bool))


def pack_mask(bits):
    """[.., n, n] bool -> [.., n, ceil(n/32)] int32 words."""
    bits = np.asarray(bits, bool)
    n = bits.shape[-1]
    words = -(-n // 32)
    full = np.zeros(bits.shape[:-1] + (words * 32,), bool)
    full[..., :n] = bits
    return torch.from_numpy(np.ascontiguousarray(np.packbits(full, axis=-1, bitorder="little")).view(np.int32).copy())


def tree_bits(rng, n):
    """Ancestor matrix of a random tree of n drafted tokens."""
    anc = np.zeros((n, n), bool)
    for i in range(n):
        par = int(rng.integers(-1, i)) if i else -1
        if par >= 0:
            anc[i] = anc[par]
        anc[i, i] = True
    return anc


def check_tree(q, k_pages, v_pages, table, lens, tls, masks, o, lse, o0, lse0, scale=None, what=""):
    """Every row of msa_attn_tree's outputs; o0 / lse0: what they held before.  masks: [B, n, n] bool or None."""
    B, Hq, n, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    g = Hq // Hkv
    scale = 1 / math.sqrt(d) if scale is None else scale
    for b in range(B):
        L, T = int(lens[b]), int(tls[b])
        assert torch.equal(o[b, :, T:], o0[b, :, T:]) and torch.equal(lse[b, :, T:], lse0[b, :, T:]), f"{what}: rows behind request {b}"
        if T == 0:
            continue
        ids = torch.as_tensor(table[b][:-(-L // page)], dtype=torch.long, device=q.device)
        seen = torch.ones(T, L, dtype=torch.bool, device=q.device)
        tail = torch.ones(T, T, dtype=torch.bool).tril() if masks is None else torch.from_numpy(np.array(masks[b]))[:T, :T]
        seen[:, L - T:] = tail.to(q.device)
        for h in range(Hkv):
            k = k_pages[ids, h].reshape(-1, d)[:L]
            v = v_pages[ids, h].reshape(-1, d)[:L]
            ro, rl, to, tl = attend(q[b, h * g:(h + 1) * g, :T], k, v, seen, scale)
            go, gl = o[b, h * g:(h + 1) * g, :T].double(), lse[b, h * g:(h + 1) * g, :T].double()
            none = torch.isinf(rl)
            assert torch.equal(torch.isneginf(gl), none), f"{what}: rows without keys, request {b} head {h}"
            assert bool((go[none] == 0).all()), f"{what}: output of rows without keys, request {b} head {h}"
            e = (go - ro).abs()
            assert bool((e <= to).all()), f"{what}: request {b} head {h}: o off by {float((e - to).max()):.3e} above {float(to.max()):.3e}"
            e = torch.where(none, 0.0, gl - rl).abs()
            assert bool((e <= tl).all()), f"{what}: request {b} head {h}: lse off by {float(e.max()):.3e}"
