"""Attention of drafted tokens through a sliding window that keeps the first
tokens visible, over the bf16 paged cache (msa_attn_tree_window).

Every row against the definition in 64 bits within the bounds derived in
paged_ref.attend; keys that no row of a request sees hold NaN, and pages without
other keys are gone from the table."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_prefill_gb300 as msa
from paged_ref import check_rows, pack_mask, seen_keys, tree_bits

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_gb300 import build
    build.build()
    return msa.load()


def test_reference_windows():
    """The sets of eq. (3), token by token, of a chain over a whole sequence, and a tree's by depth."""
    for L, sink, window in ((40, 3, 7), (40, 0, 1), (10, 20, 2), (9, 0, 50)):
        got = seen_keys(L, L, sink=sink, window=window)
        for i in range(L):
            assert set(np.nonzero(got[i])[0]) == {j for j in range(i + 1) if j < sink or j > i - window}
    mask = np.array([[1, 0, 0], [1, 1, 0], [1, 0, 1]], bool)
    got = seen_keys(10, 3, mask, [0, 1, 1], 1, 3)
    assert [set(np.nonzero(r)[0]) for r in got] == [{0, 5, 6, 7}, {0, 6, 7, 8}, {0, 6, 7, 9}]


def test_refusals(lib):
    inv, uns, small = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_UNSUPPORTED, msa.MSA_ERR_WORKSPACE_TOO_SMALL
    P = ctypes.c_void_p

    def call(shape=None, pages=(0x10000000, 0x20000000, 64, 16), win=(4, 16, None), ws_bytes=1 << 40, width=8, stride=0, **kw):
        sh = dict(B=2, Hq=4, Hkv=2, n=3, d_h=128, scale=0.0)
        sh.update(shape or {})
        x = dict(q=P(0x1000), table=P(0x2000), lens=P(0x3000), tl=None, mask=None, o=P(0x4000), lse=None, ws=P(0x5000))
        x.update(kw)
        pg = None if pages is None else ctypes.byref(msa.KVPagesC(*pages))
        return lib.msa_attn_tree_window(ctypes.byref(msa.Shape(**sh)), x["q"], pg, x["table"], width, x["lens"], x["tl"],
                                        x["mask"], stride, None if win is None else ctypes.byref(msa.TreeWindowC(*win)),
                                        x["o"], x["lse"], x["ws"], ws_bytes, None)

    assert call(win=None) == inv
    assert call(win=(-1, 16, None)) == inv
    assert call(win=(0, 0, None)) == inv
    assert call(win=(0, -5, None)) == inv
    assert call(win=(0, 5, 0x6000)) == inv  # depths without a mask
    assert call(win=(0, 5, 0x6001), mask=P(0x7000)) == inv
    assert call(shape=dict(d_h=96)) == uns
    assert call(shape=dict(n=1025)) == uns
    assert call(pages=None) == inv
    assert call(pages=(0x10000000, None, 64, 16)) == inv
    assert call(pages=(0x10000008, 0x20000000, 64, 16)) == inv
    assert call(pages=(0x10000000, 0x20000000, 64, 8)) == uns
    assert call(pages=(0x10000000, 0x20000000, 1 << 26, 16)) == uns
    assert call(width=0) == inv
    assert call(width=1 << 28) == uns
    for k in ("q", "table", "lens", "o", "ws"):
        assert call(**{k: None}) == inv, k
    assert call(q=P(0x4000)) == inv
    assert call(mask=P(0x7000), stride=2) == inv
    assert call(ws_bytes=16) == small


def test_binding_refusals():
    q = torch.zeros(2, 4, 3, 64, dtype=BF)
    kp = torch.zeros(9, 2, 16, 64, dtype=BF)
    i32 = dict(dtype=torch.int32)
    table, lens = torch.zeros(2, 4, **i32), torch.ones(2, **i32)
    mask = torch.zeros(2, 3, 1, **i32)
    for call, what in [
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, 1, 2), "q: must be on a CUDA device"),
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, -1, 2), "sink: -1"),
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, 1, 0), "window: 0"),
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, 1, 1 << 31), "window: 2147483648"),
        (lambda: msa.attn_tree_window(q, kp, kp[:8], table, lens, 1, 2), "v_pages: shape"),
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, 1, 2, depth=torch.zeros(2, 3, **i32)), "depth: needs"),
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, 1, 2, tree_mask=mask, depth=torch.zeros(2, 4, **i32)), "depth: shape"),
        (lambda: msa.attn_tree_window(q, kp, kp, table, lens, 1, 2, tree_mask=mask, depth=torch.zeros(2, 3)), "depth: dtype"),
    ]:
        with pytest.raises(ValueError, match=what if "CUDA" not in what else "q: must"):
            call()


class Case:
    """A cache with requests of the given lengths; every row of it that no query row sees holds NaN."""

    def __init__(self, Hq, Hkv, n, d, page, lens, sink, window, seed, tls=None, masks=None, depths=None, peak=2.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.sink, self.window = [int(x) for x in lens], sink, window
        B = len(self.lens)
        self.tls = [n] * B if tls is None else [int(x) for x in tls]
        counts = [-(-x // page) for x in self.lens]
        N = sum(counts) + 3
        perm = rng.permutation(N)
        table = np.full((B, max([1] + counts)), -123456, np.int64)
        self.page, self.masks, self.depths = page, masks, depths
        self.k, self.v = (torch.full((N, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
        given = table.copy()
        used = 0
        for b, c in enumerate(counts):
            table[b, :c] = given[b, :c] = perm[used:used + c]
            used += c
            if not c:
                continue
            live = torch.zeros(c * page, dtype=torch.bool)
            live[:self.lens[b]] = True
            end = self.lens[b] - self.tls[b] - window + 1
            if end > sink:
                live[sink:end] = False
            gone = ~live.view(c, page).any(1).numpy()
            given[b, :c][gone] = [-1, 1 << 30][b % 2]
            for t, f in ((self.k, peak), (self.v, 1.0)):
                rows = torch.randn(c * page, Hkv, d, generator=g, device="cuda")
                rows[::5] *= f
                rows[~live.cuda()] = float("nan")
                t[torch.from_numpy(table[b, :c]).cuda()] = rows.view(c, page, Hkv, d).transpose(1, 2).to(BF)
        self.table = table
        i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()  # noqa: E731
        self.table_dev, self.lens_dev = i32(given), i32(self.lens)
        self.tls_dev = None if tls is None else i32(self.tls)
        self.words = None if masks is None else pack_mask(masks).cuda()
        self.depths_dev = None if depths is None else i32(depths)
        self.q = torch.randn(B, Hq, n, d, generator=g, device="cuda").to(BF)

    def run(self, **kw):
        B, Hq, n, d = self.q.shape
        o0 = torch.full((B, Hq, n, d), 7.0, dtype=BF, device="cuda")
        l0 = torch.full((B, Hq, n), 5.0, device="cuda")
        o, lse = o0.clone(), l0.clone()
        msa.attn_tree_window(self.q, self.k, self.v, self.table_dev, self.lens_dev, self.sink, self.window,
                             tree_len=self.tls_dev, tree_mask=self.words, depth=self.depths_dev, o=o, lse=lse, **kw)
        return o, lse, o0, l0

    def check(self, out, scale=None, what="", lens=None):
        lens = self.lens if lens is None else lens

        def part(t):
            def rows(b, h):
                if h is None:
                    return t.shape[1]
                ids = torch.from_numpy(self.table[b, :-(-int(lens[b]) // self.page)]).cuda()
                return t[ids, h].reshape(-1, t.shape[-1])[:int(lens[b])]
            return rows

        def seen(b):
            m = None if self.masks is None else self.masks if self.masks.ndim == 2 else self.masks[b]
            return seen_keys(int(lens[b]), self.tls[b], m, None if self.depths is None else self.depths[b], self.sink, self.window)

        o, lse, o0, l0 = out
        check_rows(self.q, part(self.k), part(self.v), lens, self.tls, seen, o, lse, o0, l0, scale, what)


WINDOWS = [(0, 1), (0, 100), (3, 64), (64, 512), (128, 1024), (130, 100), (5000, 7), (1, 100000)]


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", WINDOWS)
@pytest.mark.parametrize("Hq,Hkv,n,d,page", [(2, 1, 1, 64, 16), (4, 2, 1, 128, 128), (8, 2, 5, 64, 32), (4, 1, 20, 128, 16),
                                             (4, 1, 40, 128, 64), (3, 1, 100, 64, 16)])
def test_windows(cuda_lib, Hq, Hkv, n, d, page, sink, window):
    """Chains and trees of every row layout, windows and sinks that end anywhere in tiles and pages."""
    rng = np.random.default_rng(n + window)
    lens = n + np.array([0, 1, 130, 700, 1500, 6000])
    for masked in (False, True):
        masks = depths = None
        if masked:
            masks = np.stack([tree_bits(rng, n) for _ in lens])
            depths = masks.sum(-1) - 1
        c = Case(Hq, Hkv, n, d, page, lens, sink, window, sink + window, masks=masks, depths=depths)
        out = c.run()
        assert cuda_lib.poll_device_status() == 0
        c.check(out, what=f"window {sink}+{window} masked {masked}")


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", [(0, 60), (16, 200), (128, 1024)])
def test_chunk_of_a_prompt(cuda_lib, sink, window):
    """1024 rows, more than the window: a chunk's early keys are behind its late rows' windows; shorter chunks and a
    chunk at the start of its prompt beside it."""
    n = 1024
    c = Case(8, 2, n, 128, 64, [9000, 1024, 3000], sink, window, 5, tls=[1024, 1024, 700])
    out = c.run(scale=0.2)
    assert cuda_lib.poll_device_status() == 0
    c.check(out, scale=0.2, what="chunk")


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", [(0, 1), (0, 129), (200, 300), (128, 1024), (3, 100000)])
@pytest.mark.parametrize("Hq,n,d,page", [(1, 256, 64, 16), (2, 512, 128, 128), (3, 768, 64, 64), (2, 1024, 128, 32)])
def test_items_have_their_own_windows(cuda_lib, Hq, n, d, page, sink, window):
    """Chains whose items are 256 consecutive tokens: whole and short chunks, at the start of a prompt and far in."""
    lens = [n, 1, n + 77, 700, 5000, n + 4000, 300]
    tls = [n, 1, n, min(n, 600), n, 257 if n > 256 else 255, 0]
    c = Case(Hq, 1, n, d, page, lens, sink, window, n + window, tls=tls)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"items {n} {sink}+{window}")


@pytest.mark.gpu
@pytest.mark.parametrize("n,d", [(1, 128), (12, 64), (30, 128), (60, 128)])
def test_many_requests_cut_anywhere(cuda_lib, n, d):
    """More tiles than CTAs, parts that begin and end in sinks and in windows; the same bits on every run."""
    rng = np.random.default_rng(n)
    lens = (n + np.exp(rng.uniform(0, math.log(30000), 40))).astype(int)
    tls = rng.integers(0, n + 1, len(lens))
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    depths = masks.sum(-1) - 1
    c = Case(4, 1, n, d, 16, lens, 300, 2000, 60 + n, tls=tls, masks=masks, depths=depths, peak=4.0)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="cuts")
    again = c.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 20, 40])
def test_window_over_everything_is_the_whole(cuda_lib, n):
    """A window or a sink that covers every key: the bits of attn_tree."""
    rng = np.random.default_rng(n)
    lens = [n, 5000, 333]
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    for sink, window in ((0, 1 << 30), (6000, 1), (2600, 2600)):
        c = Case(4, 1, n, 128, 32, lens, sink, window, 3, masks=masks)
        o, lse, _, _ = c.run()
        ref_l = torch.empty_like(lse)
        ref = msa.attn_tree(c.q, c.k, c.v, c.table_dev, c.lens_dev, tree_mask=c.words, lse=ref_l)
        assert cuda_lib.poll_device_status() == 0
        assert torch.equal(o, ref) and torch.equal(lse, ref_l), (sink, window)


@pytest.mark.gpu
def test_a_window_agrees_with_the_ashape_prefill(cuda_lib):
    """Every row of a prompt through the cache sees what an A-shape head of the prefill sees."""
    n, Hq, Hkv, d, page, sink, window = 1000, 4, 2, 128, 16, 64, 200
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(1, h, n, d, generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    want = msa.attn_ashape(q, k, v, list(range(Hq)), sink, window)
    P = -(-n // page)
    kp, vp = (torch.zeros(P, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    for t, x in ((kp, k), (vp, v)):
        t.transpose(1, 2).reshape(-1, Hkv, d)[:n] = 0
        rows = torch.zeros(P * page, Hkv, d, dtype=BF, device="cuda")
        rows[:n] = x[0].transpose(0, 1)
        t.copy_(rows.view(P, page, Hkv, d).transpose(1, 2))
    table = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    got = msa.attn_tree_window(q, kp, vp, table, lens, sink, window)
    assert cuda_lib.poll_device_status() == 0
    # each is within half a step for its weights and one for its output of the exact rows, with room for the scores
    assert float((got.float() - want.float()).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())


@pytest.mark.gpu
def test_depths_out_of_range_are_clamped(cuda_lib):
    """A depth below 0 or at n and above counts as 0 or n - 1."""
    n = 5
    masks = np.tril(np.ones((n, n), bool))[None]
    depths = np.array([[-9, 1, 2, 3, 1 << 30]])
    c = Case(4, 2, n, 64, 16, [400], 3, 50, 2, masks=masks, depths=depths)
    out = c.run()
    c.depths = depths.clip(0, n - 1)
    c.check(out, what="clamped")
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_bad_requests_are_reported(cuda_lib):
    for change in ("short", "long", "page", "page negative"):
        c = Case(4, 2, 2, 64, 16, [140, 50], 16, 20, 4, tls=[2, 2])
        if change == "short":
            c.lens_dev[0] = 1
        if change == "long":
            c.lens_dev[0] = 16 * c.table.shape[1] + 1
        if change == "page":
            c.table_dev[0, 8] = c.k.shape[0]
        if change == "page negative":
            c.table_dev[0, 0] = -1
        c.run()
        assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX, change
        assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_streams_capture_and_workspace(cuda_lib):
    """Calls on a given stream; a captured decode step that follows its lengths; a workspace of the stated size."""
    c = Case(8, 2, 1, 128, 16, [3000, 900, 1], 16, 256, 9)
    want = c.run()
    nbytes = msa.attn_tree_workspace(3, 8, 2, 1, 128)
    whole = torch.full((nbytes + 512,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(ws=whole[256:256 + nbytes])
    other = c.run(stream=side)
    torch.cuda.synchronize()
    for x in (got, other):
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])
    assert bool((whole[:256] == 255).all()) and bool((whole[-256:] == 255).all())
    # every key there again, so that shorter lengths see finite ones
    c.table_dev.copy_(torch.from_numpy(c.table.astype(np.int32)))
    c.k.nan_to_num_(0.5)
    c.v.nan_to_num_(0.25)
    o, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:3], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.attn_tree_window(c.q, c.k, c.v, c.table_dev, c.lens_dev, 16, 256, o=o, lse=lse)
    for lens in ([3000, 900, 1], [2999, 1, 1], [129, 300, 1], [40, 512, 1]):
        c.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check((o, lse, o, lse), what=f"replay {lens}", lens=lens)
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", [(0, 100), (3, 64), (200, 300), (128, 1024)])
@pytest.mark.parametrize("Hq,Hkv,n,d,page", [(4, 1, 20, 64, 32), (8, 2, 32, 64, 16), (6, 2, 2, 64, 64), (8, 8, 100, 128, 128),
                                             (4, 1, 16, 128, 16), (5, 1, 27, 64, 16)])
def test_ragged_windows_of_every_row_layout(cuda_lib, Hq, Hkv, n, d, page, sink, window):
    """6 to 135 rows a KV head, both sides of 64 and 128, heads of 64 with 65 to 128 rows among them; requests with
    fewer drafted tokens than rows."""
    rng = np.random.default_rng(n + window)
    lens = n + np.array([0, 1, 130, 700, 1500, 6000])
    tls = [n, 1, n // 2, n, 0, n - 1]
    for masked in (False, True):
        masks = depths = None
        if masked:
            masks = np.stack([tree_bits(rng, n) for _ in lens])
            depths = masks.sum(-1) - 1
        c = Case(Hq, Hkv, n, d, page, lens, sink, window, sink + window + d, tls=tls, masks=masks, depths=depths)
        out = c.run()
        assert cuda_lib.poll_device_status() == 0
        c.check(out, what=f"window {sink}+{window} masked {masked}")
