"""Attention of drafted tokens over a paged cache (msa_attn_tree).

CPU: host checks and the reference's own mask handling.  GPU: every row against
the definition in 64 bits within the bounds derived in paged_ref.attend; rows
behind a request's tokens keep their bits; pages hold NaN wherever no live
token lies."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_prefill_gb300 as msa
from paged_ref import check_tree, pack_mask, tree_bits, unpack_mask

BF = torch.bfloat16


def test_mask_words_round_trip():
    rng = np.random.default_rng(0)
    for n in (1, 31, 32, 33, 70):
        bits = np.stack([tree_bits(rng, n) for _ in range(3)])
        words = pack_mask(bits)
        assert words.shape == (3, n, -(-n // 32))
        assert torch.equal(unpack_mask(words, n), torch.from_numpy(bits))
        assert bool(bits[:, np.arange(n), np.arange(n)].all()) and not np.triu(bits, 1).any()


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_gb300 import build
    build.build()
    return msa.load()


def test_refusals(lib):
    inv, uns, small = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_UNSUPPORTED, msa.MSA_ERR_WORKSPACE_TOO_SMALL
    P = ctypes.c_void_p

    def call(shape=None, pages=(0x10000000, 0x20000000, 64, 16), ws_bytes=1 << 40, width=8, stride=0, **kw):
        sh = dict(B=2, Hq=4, Hkv=2, n=3, d_h=128, scale=0.0)
        sh.update(shape or {})
        x = dict(q=P(0x1000), table=P(0x2000), lens=P(0x3000), tl=None, mask=None, o=P(0x4000), lse=None, ws=P(0x5000))
        x.update(kw)
        pg = None if pages is None else ctypes.byref(msa.KVPagesC(*pages))
        return lib.msa_attn_tree(ctypes.byref(msa.Shape(**sh)), x["q"], pg, x["table"], width, x["lens"], x["tl"],
                                 x["mask"], stride, x["o"], x["lse"], x["ws"], ws_bytes, None)

    assert call(shape=dict(d_h=96)) == uns
    assert call(shape=dict(n=1025)) == uns
    assert call(shape=dict(n=0)) == inv
    assert call(shape=dict(Hkv=3)) == inv
    assert call(shape=dict(scale=float("inf"))) == inv
    assert call(shape=dict(B=1 << 19, Hq=32, Hkv=8, n=1024)) == uns
    assert call(pages=None) == inv
    assert call(pages=(0x10000000, None, 64, 16)) == inv
    assert call(pages=(0x10000008, 0x20000000, 64, 16)) == inv
    assert call(pages=(0x10000000, 0x20000000, 0, 16)) == inv
    assert call(pages=(0x10000000, 0x20000000, 64, 8)) == uns
    assert call(pages=(0x10000000, 0x20000000, 1 << 26, 16)) == uns  # Hkv rows of the cache pass 2^31
    assert call(width=0) == inv
    assert call(width=1 << 28) == uns
    for k in ("q", "table", "lens", "o", "ws"):
        assert call(**{k: None}) == inv, k
    assert call(q=P(0x4000)) == inv            # in place
    assert call(o=P(0x4008)) == inv
    assert call(lse=P(0x4002)) == inv
    assert call(mask=P(0x6000), stride=2) == inv
    assert call(ws_bytes=16) == small
    sh = msa.Shape(2, 4, 2, 3, 128, 0.0)
    assert lib.msa_attn_tree_workspace(ctypes.byref(sh)) > 0
    sh.n = 2000
    assert lib.msa_attn_tree_workspace(ctypes.byref(sh)) == 0
    assert lib.msa_attn_tree_workspace(None) == 0


def test_binding_refusals():
    q = torch.zeros(2, 4, 3, 64, dtype=BF)
    kp = torch.zeros(9, 2, 16, 64, dtype=BF)
    i32 = dict(dtype=torch.int32)
    table, lens = torch.zeros(2, 4, **i32), torch.ones(2, **i32)
    for call, what in [
        (lambda: msa.attn_tree(q, kp, kp, table, lens), "q: must be on a CUDA device"),
        (lambda: msa.attn_tree(q[0], kp, kp, table, lens), "q: a 4-d"),
        (lambda: msa.attn_tree(q.transpose(1, 2), kp, kp, table, lens), "q: must be contiguous"),
        (lambda: msa.attn_tree(q, kp[..., :32], kp, table, lens), "k_pages: shape"),
        (lambda: msa.attn_tree(q, kp, kp[:8], table, lens), "v_pages: shape"),
        (lambda: msa.attn_tree(q, kp, kp, table[:1], lens), "page_table: shape"),
        (lambda: msa.attn_tree(q, kp, kp, table.long(), lens), "page_table: dtype"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens[:1]), "seq_len: shape"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens, tree_len=lens.float()), "tree_len: dtype"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens, tree_mask=torch.zeros(2, 2, 1, **i32)), "tree_mask: shape"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens, tree_mask=torch.zeros(3, 2, **i32)), "tree_mask: shape"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens, tree_mask=[[1]] * 3), "tree_mask: a torch.Tensor"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens, lse=torch.zeros(2, 4, 2)), "lse: shape"),
        (lambda: msa.attn_tree(q, kp, kp, table, lens, ws=torch.zeros(8)), "ws: dtype"),
    ]:
        with pytest.raises(ValueError, match=what):
            call()


class Case:
    """A cache with requests of the given lengths, NaN in every row that holds no live token."""

    def __init__(self, Hq, Hkv, n, d, page, lens, seed, tls=None, masks=None, peak=2.0, spare=3, width=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens = [int(x) for x in lens]
        B = len(self.lens)
        self.tls = [n] * B if tls is None else [int(x) for x in tls]
        counts = [-(-x // page) for x in self.lens]
        N = sum(counts) + spare
        perm = rng.permutation(N)
        width = max([width, 1] + counts)
        table = np.full((B, width), -123456, np.int64)  # entries behind a request's pages are not read
        self.k, self.v = (torch.full((N, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
        used = 0
        for b, c in enumerate(counts):
            table[b, :c] = perm[used:used + c]
            used += c
            if not c:
                continue
            for t, f in ((self.k, peak), (self.v, 1.0)):
                rows = torch.full((c * page, Hkv, d), float("nan"), device="cuda")
                rows[:self.lens[b]] = torch.randn(self.lens[b], Hkv, d, generator=g, device="cuda")
                rows[0:self.lens[b]:5] *= f
                t[torch.from_numpy(table[b, :c]).cuda()] = rows.view(c, page, Hkv, d).transpose(1, 2).to(BF)
        self.table = table
        self.table_dev = torch.from_numpy(table.astype(np.int32)).cuda()
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.tls_dev = None if tls is None else torch.tensor(self.tls, dtype=torch.int32, device="cuda")
        self.masks = masks
        self.words = None if masks is None else pack_mask(masks).cuda()
        self.q = torch.randn(B, Hq, n, d, generator=g, device="cuda").to(BF)

    def run(self, **kw):
        B, Hq, n, d = self.q.shape
        o0 = torch.full((B, Hq, n, d), 7.0, dtype=BF, device="cuda")
        l0 = torch.full((B, Hq, n), 5.0, device="cuda")
        o, lse = o0.clone(), l0.clone()
        msa.attn_tree(self.q, self.k, self.v, self.table_dev, self.lens_dev, tree_len=self.tls_dev,
                      tree_mask=self.words, o=o, lse=lse, **kw)
        return o, lse, o0, l0

    def check(self, out, scale=None, what=""):
        o, lse, o0, l0 = out
        masks = self.masks
        if masks is not None and masks.ndim == 2:
            masks = np.broadcast_to(masks, (len(self.lens),) + masks.shape)
        check_tree(self.q, self.k, self.v, self.table, self.lens, self.tls, masks, o, lse, o0, l0, scale, what)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (4, 2, 128), (8, 8, 128), (7, 1, 64)])
def test_single_token(cuda_lib, Hq, Hkv, d, page):
    """Decode: one row per head, lengths around every page and tile border."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000, 2049]
    c = Case(Hq, Hkv, 1, d, page, lens, 100 + page + d)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"decode {Hq}/{Hkv} d{d} page {page}")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,n,d", [(2, 1, 2, 64), (8, 2, 8, 128), (4, 1, 31, 64), (4, 1, 32, 128), (4, 1, 33, 128),
                                        (8, 1, 24, 64), (32, 8, 64, 128), (5, 5, 129, 64), (8, 2, 65, 128), (3, 1, 100, 64),
                                        (16, 2, 100, 128), (1, 1, 1024, 64)])
def test_trees(cuda_lib, Hq, Hkv, n, d):
    """Random trees, ragged, from 4 to 1024 rows a KV group: one and two row tiles, partly filled, and several 256-row blocks."""
    rng = np.random.default_rng(n)
    B = 4
    tls = [n, max(1, n // 2), 1, 0]
    ctx = [0, 700, 128 - 1, 50]
    masks = np.stack([tree_bits(rng, n) for _ in range(B)])
    c = Case(Hq, Hkv, n, d, 16, [a + b for a, b in zip(ctx, tls)], n, tls=tls, masks=masks)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"trees {Hq}/{Hkv} n{n} d{d}")


@pytest.mark.gpu
@pytest.mark.parametrize("n,page", [(1, 16), (5, 128), (40, 32), (70, 64)])
def test_chains_and_scale(cuda_lib, n, page):
    """No mask: drafted token i sees the drafted ones up to itself; a scale of the caller's."""
    c = Case(8, 2, n, 128, page, [n, n + 1, n + 127, n + 1000], 31 + n)
    out = c.run(scale=0.02)
    assert cuda_lib.poll_device_status() == 0
    c.check(out, scale=0.02, what=f"chain n{n}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [6, 40])
def test_rows_without_keys_and_shared_mask(cuda_lib, n):
    """A mask that names nothing for some rows (no context: o = 0, lse = -inf), one mask for all requests."""
    rng = np.random.default_rng(9)
    m = rng.random((n, n)) < 0.3
    m[1] = m[n - 1] = False
    c = Case(8, 2, n, 64, 16, [n, n + 5, n - 2], 77, tls=[n, n, n - 2], masks=m)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    assert bool(torch.isneginf(out[1][0, :, 1]).all())
    c.check(out, what="empty rows")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 1, 1), (4, 1, 17), (4, 1, 50), (6, 2, 100)])
def test_long_contexts_are_cut_and_joined(cuda_lib, Hq, Hkv, n, d):
    """One long request cut over all CTAs beside short ones; the same bits on every run."""
    rng = np.random.default_rng(n)
    lens = [60001, 5, 4097, 130]
    tls = [n, min(n, 5), max(1, n // 3), n]
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Case(Hq, Hkv, n, d, 64, lens, 40 + n, tls=tls, masks=masks, peak=6.0)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="long")
    again = c.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 1), (4, 2, 20), (4, 1, 32), (8, 2, 40)])
def test_items_across_many_cuts(cuda_lib, Hq, Hkv, n, page):
    """Requests of a few to a few hundred tiles, so that parts begin and end anywhere in items: single tiles, items
    cut once, items over many parts, parts over many items; every row layout."""
    rng = np.random.default_rng(7 * n)
    lens = (n + np.exp(rng.uniform(0, math.log(30000), 24))).astype(int)
    tls = rng.integers(1, n + 1, len(lens))
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Case(Hq, Hkv, n, 128, page, lens, 60 + n, tls=tls, masks=masks, peak=4.0)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="cuts")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,n,d,lens", [(16, 2, 100, 128, [12001, 300, 5000]), (4, 1, 200, 64, [9000]),
                                             (4, 1, 200, 128, [5000, 1000]), (3, 1, 100, 64, [200, 7000])])
def test_row_blocks_are_cut_and_joined(cuda_lib, Hq, Hkv, n, d, lens):
    """More than 256 rows a KV group, the last block of them partly filled, each block cut on its own: few long items
    and many; a request whose tree is shorter than its rows."""
    rng = np.random.default_rng(n + d)
    tls = [n, n // 2, n][:len(lens)]
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Case(Hq, Hkv, n, d, 32, lens, 90 + n, tls=tls, masks=masks, peak=4.0)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="row blocks")
    again = c.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.gpu
def test_large_scores_across_tiles(cuda_lib):
    """Scores that grow along the keys (every tile raises the maximum by tens) and fall again."""
    c = Case(4, 2, 3, 128, 32, [900, 4000], 13)
    ramp = torch.linspace(1, 12, 4000, device="cuda")
    ids = torch.from_numpy(c.table[1]).cuda()
    rows = c.k[ids].transpose(1, 2).reshape(-1, 2, 128)
    rows[:4000] = (rows[:4000].float() * torch.where(ramp < 9, ramp, 18 - ramp)[:, None, None]).to(BF)
    c.k[ids] = rows.view(len(ids), 32, 2, 128).transpose(1, 2)
    c.q *= 4
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="ramp")


@pytest.mark.gpu
def test_masked_infinities(cuda_lib):
    """An infinite or NaN key that a row's mask leaves out does not reach that row (values stay finite)."""
    n = 4
    m = np.eye(n, dtype=bool)
    c = Case(4, 1, n, 64, 16, [40], 3, masks=m[None])
    slot = 36 + 2  # key of drafted token 2
    page, off = c.table[0][slot // 16], slot % 16
    good = c.run()
    c.k[page, 0, off, 0] = float("inf")
    bad = c.run()
    assert cuda_lib.poll_device_status() == 0
    keep = [0, 1, 3]
    assert torch.equal(good[0][0, :, keep], bad[0][0, :, keep]) and torch.equal(good[1][0, :, keep], bad[1][0, :, keep])
    c.k[page, 0, off] = float("nan")
    bad = c.run()
    assert torch.equal(good[0][0, :, keep], bad[0][0, :, keep])
    assert bool(bad[0][0, :, 2].isnan().all()) and bool(bad[1][0, :, 2].isnan().all())


@pytest.mark.gpu
def test_shared_pages_and_wide_tables(cuda_lib):
    """Two requests that read the same prefix pages; a table wider than any request needs."""
    c = Case(8, 2, 2, 128, 16, [100, 100], 21, width=600)
    c.table[1, :5] = c.table[0, :5]
    c.table_dev[1, :5] = c.table_dev[0, :5]
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="shared prefix")


@pytest.mark.gpu
def test_empty_batch_and_requests(cuda_lib):
    """No drafted tokens anywhere: nothing is written; requests without any beside one that has some."""
    c = Case(4, 2, 3, 64, 16, [0, 20], 2, tls=[0, 0])
    out = c.run()
    c.check(out, what="nothing")
    c = Case(4, 2, 3, 64, 16, [0, 20, 0, 9, 0], 2, tls=[0, 0, 0, 2, 0])
    out = c.run()
    c.check(out, what="one of five")
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_many_requests(cuda_lib):
    """More requests than threads of a CTA."""
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 200, 900)
    c = Case(2, 1, 1, 64, 16, lens, 8)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="900 requests")


@pytest.mark.gpu
def test_bad_requests_are_reported(cuda_lib):
    """Lengths and page ids that break the contract set the error word; the context goes on."""
    for change in ("short", "long", "negative", "page", "page negative"):
        c = Case(4, 2, 2, 64, 16, [40, 50], 4, tls=[2, 2])
        if change == "short":
            c.lens_dev[0] = 1
        if change == "long":
            c.lens_dev[0] = 16 * c.table.shape[1] + 1
        if change == "negative":
            c.tls_dev[0] = -1
        if change == "page":
            c.table_dev[0, 1] = c.k.shape[0]
        if change == "page negative":
            c.table_dev[0, 1] = -1
        c.run()
        assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX, change
        assert cuda_lib.poll_device_status() == 0
    c = Case(4, 2, 2, 64, 16, [40, 50], 4, tls=[2, 2])
    c.check(c.run(), what="after bad requests")


@pytest.mark.gpu
def test_streams_and_captures(cuda_lib):
    """Two calls at once on two streams; captured calls that follow lengths which change on the device."""
    a = Case(8, 2, 4, 128, 64, [5000, 900, 33], 51)
    b = Case(4, 1, 40, 128, 16, [3000, 77], 52)
    wa, wb = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            x = a.run()
        with torch.cuda.stream(s2):
            y = b.run()
        outs.append((x, y))
    z = a.run(stream=s1)
    torch.cuda.synchronize()
    for x, y in outs + [(z, wb)]:
        assert torch.equal(x[0], wa[0]) and torch.equal(x[1], wa[1])
        assert torch.equal(y[0], wb[0]) and torch.equal(y[1], wb[1])
    o, lse = torch.zeros_like(a.q), torch.zeros(a.q.shape[:3], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.attn_tree(a.q, a.k, a.v, a.table_dev, a.lens_dev, o=o, lse=lse)
    for lens in ([5000, 900, 33], [4, 900, 20], [4999, 100, 4], [129, 128, 5]):
        a.lens = lens
        a.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check_tree(a.q, a.k, a.v, a.table, lens, a.tls, None, o, lse, o, lse, what=f"replay {lens}")
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_cache_beyond_32_bit_offsets(cuda_lib):
    """Pages whose element offsets lie above 2^32."""
    N, Hkv, page, d = 34000, 8, 128, 128
    if torch.cuda.mem_get_info()[0] < 3 * N * Hkv * page * d * 2:
        pytest.skip("needs 27 GB")
    k, v = (torch.empty(N, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    ids = [N - 1, 0, N - 7, 16384 + 3, 32768 + 5]
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k, v):
        for p in ids:
            t[p] = torch.randn(Hkv, page, d, generator=g, device="cuda").to(BF)
    lens, n = [5 * 128 - 9], 3
    table = np.array([ids])
    q = torch.randn(1, 32, n, d, generator=g, device="cuda").to(BF)
    o, lse = torch.zeros_like(q), torch.zeros(1, 32, n, device="cuda")
    msa.attn_tree(q, k, v, torch.from_numpy(table.astype(np.int32)).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  o=o, lse=lse)
    assert cuda_lib.poll_device_status() == 0
    check_tree(q, k, v, table, lens, [n], None, o, lse, o, lse, what="far pages")
    # and written there
    x = torch.randn(4, Hkv * 2 + 32, d, generator=g, device="cuda").to(BF)
    slots = torch.tensor([(N - 2) * page + 5, 3, (N - 3) * page, 32769 * page + 127], dtype=torch.int32, device="cuda")
    msa.qk_norm_rope(x[None, :, :32], x[None, :, 32:40], x[None, :, 40:], msa.rope_cfg(0), k_pages=k, v_pages=v,
                     slots=slots, layer_kv=False)
    assert cuda_lib.poll_device_status() == 0
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(k[s // page, :, s % page], x[t, 32:40]) and torch.equal(v[s // page, :, s % page], x[t, 40:])


@pytest.mark.gpu
def test_prefill_draft_verify_together(cuda_lib):
    """The operators as a server runs them: pages for two prompts, prompts normed and rotated into layer and cache,
    the prefill, a drafted tree into the cache and over it, then the accepted path again as a chain."""
    Hq, Hkv, d, page, theta = 8, 2, 128, 16, 10000.0
    lens, n = [300, 1000], 6
    g = torch.Generator(device="cuda").manual_seed(4)
    pool = msa.PagePool.empty(2, 80, 150, page, "cuda")
    kp, vp = (torch.full((150, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    w = (1 + 0.2 * torch.randn(2, d, generator=g, device="cuda")).to(BF)
    cfg = msa.rope_cfg(d, theta=theta, norm=True, q_weight=w[0], k_weight=w[1])
    i32 = dict(dtype=torch.int32, device="cuda")

    def project(*lead):
        x = torch.randn(*lead, Hq + 2 * Hkv, d, generator=g, device="cuda").to(BF)
        return x, x.split([Hq, Hkv, Hkv], -2)

    # prompts
    xp, (q, k, v) = project(sum(lens))
    cu, slots, pos = msa.build_page_tables(pool, torch.tensor(lens, **i32), tok_cap=sum(lens))
    cul = [0, 300, 1300]
    assert cu.tolist() == cul
    ql, kl, vl = msa.qk_norm_rope_varlen(q, k, v, cul, cfg, positions=pos, k_pages=kp, v_pages=vp, slots=slots)
    table = [dict(pattern="ashape", sink=2000, window=2000)] * Hq  # every key: the prefill's rows are dense attention
    o = msa.prefill_layer_varlen(ql, kl, vl, table, cul, Hq, Hkv, d)
    assert cuda_lib.poll_device_status() == 0

    # the last prompt row again, from the cache
    last = torch.stack([msa.unpack_varlen(ql, Hq, cul, d)[s][:, -1:] for s in range(2)]).contiguous()
    got = msa.attn_tree(last, kp, vp, pool.page_table, pool.seq_len)
    for s in range(2):
        want = msa.unpack_varlen(o, Hq, cul, d)[s][:, -1].float()
        assert float((got[s, :, 0].float() - want).abs().max()) <= 2 * (1.5e-2 + 2.0 ** -8 * float(want.abs().max()))

    # a drafted tree: 0 -> 1 -> 3, 0 -> 2 -> 4 -> 5
    parents = [-1, 0, 0, 1, 2, 4]
    anc, depth = np.zeros((n, n), bool), [0] * n
    for i, p in enumerate(parents):
        if p >= 0:
            anc[i] = anc[p]
            depth[i] = depth[p] + 1
        anc[i, i] = True
    xt, (q, k, v) = project(2, n)
    new = pool.seq_len + n
    _, slots, pos = msa.build_page_tables(pool, new, seq_tokens=n, depth=torch.tensor(depth * 2, **i32))
    assert pos.tolist() == [300 + x for x in depth] + [1000 + x for x in depth]
    qt, _, _ = msa.qk_norm_rope(q, k, v, cfg, positions=pos, k_pages=kp, v_pages=vp, slots=slots, layer_kv=False)
    lse_t = torch.zeros(2, Hq, n, device="cuda")
    ot = msa.attn_tree(qt, kp, vp, pool.page_table, pool.seq_len, tree_mask=pack_mask(anc).cuda(), lse=lse_t)
    assert cuda_lib.poll_device_status() == 0
    check_tree(qt, kp, vp, pool.page_table.cpu().numpy(), [306, 1006], [n, n], np.stack([anc, anc]), ot, lse_t, ot, lse_t,
               what="drafted")

    # path 0, 2, 4, 5 accepted: the pages of the tree go back, the path's tokens come as a chain at the same positions
    msa.build_page_tables(pool, pool.seq_len - n)
    path = [0, 2, 4, 5]
    q, k, v = xt[:, path].split([Hq, Hkv, Hkv], -2)
    _, slots, pos = msa.build_page_tables(pool, pool.seq_len + 4, seq_tokens=4)
    assert pos.tolist() == list(range(300, 304)) + list(range(1000, 1004))
    qc, _, _ = msa.qk_norm_rope(q, k, v, cfg, positions=pos, k_pages=kp, v_pages=vp, slots=slots, layer_kv=False)
    assert torch.equal(qc, qt[:, :, path])  # same rows, same positions: the same bits
    lse_c = torch.zeros(2, Hq, 4, device="cuda")
    oc = msa.attn_tree(qc, kp, vp, pool.page_table, pool.seq_len, lse=lse_c)
    assert cuda_lib.poll_device_status() == 0
    check_tree(qc, kp, vp, pool.page_table.cpu().numpy(), [304, 1004], [4, 4], None, oc, lse_c, oc, lse_c, what="accepted")
    # tree and chain see the same keys: they differ by at most both bounds
    ref = ot[:, :, path].float()
    assert float((oc.float() - ref).abs().max()) <= 2 * (2.0 ** -7 * float(vp.nan_to_num().abs().max()))
    assert float((lse_c - lse_t[:, :, path]).abs().max()) < 2e-3
    # finished: every page is free again
    msa.build_page_tables(pool, torch.zeros(2, **i32))
    assert pool.state.tolist() == [150, 0, 0, 0] and sorted(pool.free_pages.tolist()) == list(range(150))
    assert math.isfinite(float(oc.float().sum()))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tiles", [303, 304, 305, 400, 606, 607, 608])
def test_parts_of_one_and_two_tiles(cuda_lib, tiles, d):
    """65 to 128 rows a KV head over about as many tiles as there are parts: a CTA's first group is done after one tile,
    and joins with the second; one item over all parts, and items that begin inside them."""
    rng = np.random.default_rng(tiles)
    for lens in ([128 * tiles - 5], [128 * (tiles - 7) - 100, 128 * 2, 128 * 5 - 60]):
        n = 20  # 80 rows
        masks = np.stack([tree_bits(rng, n) for _ in lens])
        c = Case(4, 1, n, d, 64, lens, 10 + tiles, tls=[n, 3, n][:len(lens)], masks=masks)
        out = c.run()
        assert cuda_lib.poll_device_status() == 0
        c.check(out, what=f"{tiles} tiles")
        again = c.run()
        assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


def _guarded(nbytes):
    """A workspace of exactly nbytes between guards, all bytes 0xFF (as fp32: NaN; as int32: -1)."""
    whole = torch.full((nbytes + 512,), 255, dtype=torch.uint8, device="cuda")
    return whole, whole[256:256 + nbytes]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 1), (4, 1, 16), (4, 1, 20), (4, 1, 32), (4, 1, 48), (6, 1, 100)])
def test_workspace_of_the_stated_size(cuda_lib, Hq, Hkv, n, d):
    """Every row layout, items cut many times and not at all: the stated bytes suffice, need no value before the call
    and give the bits of a workspace that the call allocates."""
    rng = np.random.default_rng(n + d)
    lens = [50001, n, n + 700, n + 4000]
    tls = [n, n, max(1, n // 2), 1]
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Case(Hq, Hkv, n, d, 32, lens, 5 + n, tls=tls, masks=masks, peak=4.0)
    whole, ws = _guarded(msa.attn_tree_workspace(len(lens), Hq, Hkv, n, d))
    out = c.run(ws=ws)
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="workspace")
    assert bool((whole[:256] == 255).all()) and bool((whole[-256:] == 255).all())
    own = c.run()
    assert torch.equal(out[0], own[0]) and torch.equal(out[1], own[1])


@pytest.mark.gpu
def test_workspace_reused_by_other_shapes(cuda_lib):
    """One workspace for calls of different shapes and row layouts one after another, each after calls that left more
    parts and cuts in it, fewer, and other ones."""
    rng = np.random.default_rng(17)
    cases = []
    for Hq, Hkv, n, d, lens in [(4, 1, 32, 128, [60000, 900]), (4, 1, 32, 128, [200, 129]), (4, 2, 3, 64, [30000, 7, 5000]),
                                (4, 1, 50, 128, [20000] * 3), (8, 8, 1, 128, [40, 300]), (4, 1, 50, 128, [260]),
                                (4, 1, 20, 64, [300] * 40)]:
        masks = np.stack([tree_bits(rng, n) for _ in lens])
        cases.append(Case(Hq, Hkv, n, d, 64, lens, 70 + n, masks=masks))
    need = max(msa.attn_tree_workspace(len(c.lens), *(c.q.shape[1], c.k.shape[1], *c.q.shape[2:])) for c in cases)
    whole, ws = _guarded(need)
    want = [c.run() for c in cases]
    for x in list(range(len(cases))) + rng.permutation(np.repeat(np.arange(len(cases)), 3)).tolist():
        got = cases[x].run(ws=ws)
        assert torch.equal(got[0], want[x][0]) and torch.equal(got[1], want[x][1]), x
    assert cuda_lib.poll_device_status() == 0
    for c, w in zip(cases, want):
        c.check(w, what="reused")
    assert bool((whole[:256] == 255).all()) and bool((whole[-256:] == 255).all())
