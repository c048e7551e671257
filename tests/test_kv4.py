"""The 4-bit paged cache: appending (msa_qk_norm_rope_kv4 and its varlen form),
reading back (msa_kv4_gather) and attention of drafted tokens over it
(msa_attn_tree_kv4), with and without a window.

CPU: host checks and the reference's own rounding.  GPU: the cache holds exactly
what the definition gives in 64 bits; every attention row within the bounds that
paged_ref.attend derives, with weights rounded to fp16."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_prefill_gb300 as msa
from paged_ref import (KV4_WEIGHTS, check_rounded, check_rows, kv4_round, kv4_store, kv4_values, norm_rope, pack_mask,
                       seen_keys, tree_bits)

BF = torch.bfloat16
NAN_SCALE = 0x7F  # an e4m3 NaN


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_gb300 import build
    build.build()
    return msa.load()


# ------------------------------------------------------------------ CPU
def test_reference_rounding_and_layout():
    """Borders go to the even code, scales to the even number; what was stored reads back."""
    x = torch.zeros(1, 1, 32, dtype=torch.float64)
    x[..., :16] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.2, 0.26, 0.74, 2.51, 4.99, 5.01])
    x[..., 16] = 6 * 1.0625  # a scale halfway between 1 and 1.125
    v, codes, s = kv4_round(x)
    want = [6, 0, 1, 1, 2, 2, 4, 4, 0, -4, 0, 0.5, 0.5, 3, 4, 6]
    assert v[0, 0, :16].tolist() == want and s[0, 0].tolist() == [0x38, 0x38]
    assert float(v[0, 0, 16]) == 6.0
    tiny = torch.full((1, 1, 32), 6 * 2.0 ** -10, dtype=torch.float64)  # halfway to the smallest scale: zero
    tiny[..., 16:] *= 1.01
    v, _, s = kv4_round(tiny)
    assert not bool(v[..., :16].any()) and s[0, 0].tolist() == [0, 1]
    big = torch.full((1, 1, 16), 1e6, dtype=torch.float64)
    assert float(kv4_round(big)[0].max()) == 448 * 6
    g = torch.Generator().manual_seed(0)
    for page, d, ks, vs in ((16, 64, 1.0, 0.5), (128, 128, 4.0, 1.0)):
        data = torch.zeros(5, 2, msa.kv4_page_bytes(page, d), dtype=torch.uint8)
        slots = torch.randperm(5 * page, generator=g)[:40]
        x = torch.randn(2, 40, 2, d, generator=g, dtype=torch.float64)
        kept = []
        for which, sc in ((0, ks), (1, vs)):
            v, c, s = kv4_round(x[which], sc)
            kv4_store(data, page, d, which, slots, c, s)
            kept.append(v)
        for got, v in zip(kv4_values(data, page, d, ks, vs), kept):
            assert torch.equal(got.transpose(1, 2).reshape(-1, 2, d)[slots], v)


def test_refusals(lib):
    inv, uns, small = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_UNSUPPORTED, msa.MSA_ERR_WORKSPACE_TOO_SMALL
    P = ctypes.c_void_p
    good = (0x10000000, 64, 16, 1.0, 0.5)

    def bad_pages(call):
        assert call(None) == inv
        assert call((None,) + good[1:]) == inv
        assert call((0x10000008,) + good[1:]) == inv
        assert call(good[:1] + (0,) + good[2:]) == inv
        assert call(good[:2] + (24,) + good[3:]) == uns
        assert call(good[:1] + (1 << 27,) + good[2:]) == uns
        for s in (3.0, -1.0, float("nan"), float("inf"), 2.0 ** -41, 2.0 ** 41):
            assert call(good[:3] + (s, 1.0)) == inv, s
            assert call(good[:3] + (1.0, s)) == inv, s

    def attn(pages=good, shape=None, win=None, ws_bytes=1 << 40, width=8, stride=0, **kw):
        sh = dict(B=2, Hq=4, Hkv=2, n=3, d_h=128, scale=0.0)
        sh.update(shape or {})
        x = dict(q=P(0x1000), table=P(0x2000), lens=P(0x3000), tl=None, mask=None, o=P(0x4000), lse=None, ws=P(0x5000))
        x.update(kw)
        pg = None if pages is None else ctypes.byref(msa.KV4PagesC(*pages))
        return lib.msa_attn_tree_kv4(ctypes.byref(msa.Shape(**sh)), x["q"], pg, x["table"], width, x["lens"], x["tl"],
                                     x["mask"], stride, None if win is None else ctypes.byref(msa.TreeWindowC(*win)),
                                     x["o"], x["lse"], x["ws"], ws_bytes, None)

    bad_pages(attn)
    assert attn(shape=dict(d_h=96)) == uns
    assert attn(shape=dict(n=1025)) == uns
    assert attn(shape=dict(n=0)) == inv
    assert attn(shape=dict(Hkv=3)) == inv
    assert attn(width=0) == inv
    assert attn(width=1 << 28) == uns
    for k in ("q", "table", "lens", "o", "ws"):
        assert attn(**{k: None}) == inv, k
    assert attn(q=P(0x4000)) == inv
    assert attn(o=P(0x4008)) == inv
    assert attn(lse=P(0x4002)) == inv
    assert attn(mask=P(0x6000), stride=2) == inv
    assert attn(win=(-1, 4, None)) == inv
    assert attn(win=(0, 0, None)) == inv
    assert attn(win=(0, 4, 0x7000)) == inv           # depths without a mask
    assert attn(win=(0, 4, 0x7002), mask=P(0x6000)) == inv
    assert attn(ws_bytes=8) == small
    sh = msa.Shape(2, 4, 2, 3, 128, 0.0)
    assert lib.msa_attn_tree_kv4_workspace(ctypes.byref(sh)) > 0
    sh.n = 2000
    assert lib.msa_attn_tree_kv4_workspace(ctypes.byref(sh)) == 0
    assert lib.msa_attn_tree_kv4_workspace(None) == 0

    def gather(pages=good, width=8, d=128, **kw):
        x = dict(table=P(0x2000), lens=P(0x3000), k=P(0x4000), v=P(0x5000))
        x.update(kw)
        pg = None if pages is None else ctypes.byref(msa.KV4PagesC(*pages))
        return lib.msa_kv4_gather(ctypes.byref(msa.Shape(2, 2, 2, 9, d, 0.0)), pg, x["table"], width, x["lens"], x["k"],
                                  x["v"], None)

    bad_pages(gather)
    assert gather(d=96) == uns
    assert gather(width=0) == inv
    assert gather(width=1 << 28) == uns
    for k in ("table", "lens", "k", "v"):
        assert gather(**{k: None}) == inv, k
    assert gather(k=P(0x4008)) == inv
    assert gather(k=P(0x5000)) == inv
    assert gather(k=P(0x10000000)) == inv

    c = msa.rope_cfg(128).c

    def append(pages=good, varlen=False, **kw):
        x = dict(q_in=P(0x1000), k_in=P(0x2000), v_in=P(0x3000), q=P(0x4000), k=None, v=None, slots=P(0x5000))
        x.update(kw)
        pg = None if pages is None else ctypes.byref(msa.KV4PagesC(*pages))
        rest = (ctypes.byref(c), x["q_in"], 512, x["k_in"], 256, x["v_in"], 256, None, x["q"], x["k"], x["v"], pg,
                x["slots"], None)
        if varlen:
            return lib.msa_qk_norm_rope_varlen_kv4(ctypes.byref(msa.Shape(1, 4, 2, 1, 128, 0.0)),
                                                   (ctypes.c_int32 * 2)(0, 8), 1, *rest)
        return lib.msa_qk_norm_rope_kv4(ctypes.byref(msa.Shape(1, 4, 2, 8, 128, 0.0)), *rest)

    for varlen in (False, True):
        bad_pages(lambda pages: append(pages, varlen))
        for k in ("q_in", "k_in", "v_in", "q", "slots"):
            assert append(varlen=varlen, **{k: None}) == inv, k
        assert append(varlen=varlen, q=P(0x1000)) == inv
        assert append(varlen=varlen, k=P(0x10000000)) == inv
        assert append(varlen=varlen, q=P(0x10000000)) == inv


def test_binding_refusals():
    i32 = dict(dtype=torch.int32)
    pages = msa.KV4Pages.empty(9, 2, 16, 64, "cpu")
    assert pages.data.shape == (9, 2, 2 * 16 * 36) and msa.kv4_page_bytes(64, 128) == 64 * 144
    q = torch.zeros(2, 4, 3, 64, dtype=BF)
    table, lens = torch.zeros(2, 4, **i32), torch.ones(2, **i32)
    x = torch.zeros(2, 5, 8, 64, dtype=BF)
    qi, ki, vi = x.split([4, 2, 2], 2)
    cfg, slots = msa.rope_cfg(64), torch.zeros(10, **i32)
    other = msa.KV4Pages(torch.zeros(9, 2, 5, dtype=torch.uint8), 16, 64)
    mask = torch.zeros(3, 1, **i32)
    for call, what in [
        (lambda: msa.attn_tree_kv4(q, pages, table, lens), "q: must be on a CUDA device"),
        (lambda: msa.attn_tree_kv4(q, pages.data, table, lens), "pages: KV4Pages"),
        (lambda: msa.attn_tree_kv4(q[0], pages, table, lens), "q: a 4-d"),
        (lambda: msa.attn_tree_kv4(q, other, table, lens), "data: shape"),
        (lambda: msa.attn_tree_kv4(torch.zeros(2, 4, 3, 128, dtype=BF), pages, table, lens), "pages: heads of 64"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens[:1]), "seq_len: shape"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens, sink=3), "need a window"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens, window=-3), "window: -3"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens, sink=-3, window=3), "sink: -3"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens, window=3, depth=torch.zeros(2, 3, **i32)), "depth: needs"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens, window=3, tree_mask=mask, depth=torch.zeros(3, **i32)), "depth: shape"),
        (lambda: msa.attn_tree_kv4(q, pages, table, lens, ws=torch.zeros(8)), "ws: dtype"),
        (lambda: msa.kv4_gather(pages, table, lens, 8), "data: must be on a CUDA device"),
        (lambda: msa.kv4_gather(pages, table, lens, 0), "n: 0"),
        (lambda: msa.kv4_gather(pages, table[0], lens, 8), "page_table: a 2-d"),
        (lambda: msa.kv4_gather(pages, table, lens, 8, k=torch.zeros(2, 2, 7, 64, dtype=BF)), "k: shape"),
        (lambda: msa.qk_norm_rope_kv4(qi, ki, vi, cfg, pages, slots), "q_in: must be on a CUDA device"),
        (lambda: msa.qk_norm_rope_kv4(qi, ki, vi, cfg, pages, None), "slots: a torch.Tensor"),
        (lambda: msa.qk_norm_rope_kv4(qi, ki, None, cfg, pages, slots), "v_in: a torch.Tensor"),
        (lambda: msa.qk_norm_rope_kv4(qi, ki, vi, cfg, pages, slots[:9]), "slots: 9 elements"),
        (lambda: msa.qk_norm_rope_kv4(qi, ki, vi, cfg, (None, None), slots), "pages: KV4Pages"),
        (lambda: msa.qk_norm_rope_kv4(qi, ki[:, :, :1], vi[:, :, :1], cfg, pages, slots), "data: shape"),
        (lambda: msa.qk_norm_rope_varlen_kv4(qi[0], ki[0], vi[0], [0, 4], cfg, pages, slots), "cu_seqlens: must end"),
        (lambda: msa.KV4Pages(torch.zeros(4), 16, 64), "data: a 3-d"),
        (lambda: msa.KV4Pages.empty(1, 1, 16, 64, "cpu", k_scale=-1), "must be positive"),
    ]:
        with pytest.raises(ValueError, match=what):
            call()


# ------------------------------------------------------------------ append
def _inputs(tok, Hq, Hkv, d, seed, pad=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tok, (Hq + 2 * Hkv) * d + pad, generator=g, device="cuda") * 3
    x *= torch.exp(spread * torch.randn(tok, 1, generator=g, device="cuda"))
    x = x.to(BF)
    w = (1 + 0.5 * torch.randn(2, d, generator=g, device="cuda")).to(BF)
    q, k, v = (t.unflatten(1, (-1, d)) for t in x[:, :(Hq + 2 * Hkv) * d].split([Hq * d, Hkv * d, Hkv * d], 1))
    return q, k, v, w


def _freq(rot, theta=10000.0):
    return [theta ** (-2 * i / rot) for i in range(rot // 2)] if rot else []


def _check_held(data, page, d, slots, k, v, before, ks=1.0, vs=1.0):
    """The cache holds fp64 k, v [tokens, Hkv, d] at the slots, exactly, and what it held before elsewhere."""
    good = slots >= 0
    rows = [t.transpose(1, 2).reshape(-1, *t.shape[1:2], d) for t in kv4_values(data, page, d, ks, vs)]
    for got, x, s in ((rows[0], k, ks), (rows[1], v, vs)):
        want = kv4_round(x[good], s)[0]
        assert torch.equal(got[slots[good].long()], want), f"{int((got[slots[good].long()] != want).sum())} values differ"
    other = torch.ones(rows[0].shape[0], dtype=torch.bool, device="cuda")
    other[slots[good].long()] = False
    was = [t.transpose(1, 2).reshape(-1, *t.shape[1:2], d) for t in kv4_values(before, page, d, ks, vs)]
    for got, old in zip(rows, was):
        assert torch.equal(got[other].nan_to_num(), old[other].nan_to_num())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot", [0, 16, 48, None])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_append(cuda_lib, d, rot, inter, norm):
    rot = d if rot is None else rot
    B, n, Hq, Hkv = 3, 37, 6, 2
    page = {0: 16, 16: 32, 48: 64}.get(rot, 128)
    tok = B * n
    q, k, v, w = _inputs(tok, Hq, Hkv, d, d + rot, pad=24)
    rng = np.random.default_rng(rot)
    pos = torch.from_numpy(rng.integers(0, 1 << 20, tok).astype(np.int32)).cuda()
    slots = torch.from_numpy(rng.permutation(tok + 40)[:tok].astype(np.int32)).cuda()
    slots[5] = -1  # a padding token: not stored
    N = -(-(tok + 40) // page)
    ks, vs = (0.25, 8.0) if inter else (1.0, 1.0)
    cfg = msa.rope_cfg(rot, interleaved=inter, norm=norm, eps=1e-5, q_weight=w[0], k_weight=w[1], rot_scale=1.5 if norm else 1.0)
    pages = msa.KV4Pages.empty(N, Hkv, page, d, "cuda", ks, vs)
    pages.data.random_(0, 256)
    before = pages.data.clone()
    shaped = [t.unflatten(0, (B, n)) for t in (q, k, v)]
    qo, ko, vo = msa.qk_norm_rope_kv4(*shaped, cfg, pages, slots, positions=pos, layer_kv=True)
    assert cuda_lib.poll_device_status() == 0
    for a, b in zip((qo, ko, vo), msa.qk_norm_rope(*shaped, cfg, positions=pos)):
        assert torch.equal(a, b)  # the layer's tensors are the bf16 call's
    ref, _ = norm_rope(k, w[1], norm, torch.tensor(1e-5, dtype=torch.float32).double().item(), rot, _freq(rot), inter, pos, 1.5 if norm else 1.0)
    _check_held(pages.data, page, d, slots, ref, v.double(), before, ks, vs)
    only = pages.data.clone()
    pages.data.copy_(before)
    qc, kc, vc = msa.qk_norm_rope_kv4(*shaped, cfg, pages, slots, positions=pos)
    assert kc is None and vc is None and torch.equal(qc, qo) and torch.equal(pages.data, only)


@pytest.mark.gpu
@pytest.mark.parametrize("varlen", [False, True])
def test_append_many_tokens(cuda_lib, varlen):
    """Enough values that some lie within fp32's error of a border: the cache still holds what 64 bits give."""
    Hq, Hkv, d, page = 32, 8, 128, 64
    lens = [4099, 1, 0, 9000, 1903] if varlen else [60003]
    cu = np.concatenate([[0], np.cumsum(lens)])
    tok = int(cu[-1])
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 12)
    rng = np.random.default_rng(12)
    N = -(-tok // page) + 2
    slots = torch.from_numpy(rng.permutation(N * page)[:tok].astype(np.int32)).cuda()
    pages = msa.KV4Pages.empty(N, Hkv, page, d, "cuda")
    before = pages.data.clone()
    cfg = msa.rope_cfg(d, theta=500000.0, norm=True, q_weight=w[0], k_weight=w[1])
    if varlen:
        qo, ko, _ = msa.qk_norm_rope_varlen_kv4(q, k, v, cu, cfg, pages, slots)
        want, _, _ = msa.qk_norm_rope_varlen(q, k, v, cu, cfg)
    else:
        qo, ko, _ = msa.qk_norm_rope_kv4(q[None], k[None], v[None], cfg, pages, slots)
        want, _, _ = msa.qk_norm_rope(q[None], k[None], v[None], cfg)
    assert cuda_lib.poll_device_status() == 0
    assert torch.equal(qo, want) and ko is None
    pos = torch.cat([torch.arange(x) for x in lens]).int().cuda()
    eps = torch.tensor(1e-6, dtype=torch.float32).double().item()
    ref, slack = norm_rope(k, w[1], True, eps, d, _freq(d, 500000.0), False, pos)
    _check_held(pages.data, page, d, slots, ref, v.double(), before)
    # the inputs do hold values within fp32's error of a border (else nothing is shown)
    _, _, s = kv4_round(ref)
    t = ref.abs() / s.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    near = sum(int(((t - b).abs() < 1e-6).sum()) for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0))
    assert near > 10


@pytest.mark.gpu
def test_append_special_blocks(cuda_lib):
    """Blocks of zeros, of the smallest and largest scales, exact borders of codes and scales in V and in unrotated K."""
    d, page, tok = 64, 16, 256
    x = torch.zeros(tok, 1, d, dtype=torch.float64, device="cuda")
    codes = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0, 0.5, 1, 1.5, 2, 3, 4, -5.0], device="cuda").double()
    for t in range(tok):
        scale = torch.tensor([t % 127], dtype=torch.uint8).view(torch.float8_e4m3fn).double().item()
        x[t, 0, :16] = codes * scale                                   # every value a border or a code, every scale
        x[t, 0, 16:32] = 6 * scale * (1 + (t % 17 - 8) / 64) * codes / 6  # scales near and at borders of scales
        x[t, 0, 32:48] = 2.0 ** (t - 140) * codes                      # down to bf16's smallest, up past e4m3's largest
    x[3, 0, 48:] = 0
    x[4, 0, 48] = -0.0
    x[5, 0, 48:] = 1e30
    x = x.to(BF)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = x[torch.randperm(tok, generator=g, device="cuda")]
    pages = msa.KV4Pages.empty(tok // page, 1, page, d, "cuda")
    before = pages.data.clone()
    slots = torch.arange(tok, dtype=torch.int32, device="cuda")
    for rot, norm in ((0, False), (16, False)):
        msa.qk_norm_rope_kv4(x[None], x[None], x[None], msa.rope_cfg(rot, norm=norm), pages, slots,
                             positions=torch.zeros(tok, dtype=torch.int32, device="cuda"))  # position 0: not turned
        assert cuda_lib.poll_device_status() == 0
        _check_held(pages.data, page, d, slots, x.double(), x.double(), before)


@pytest.mark.gpu
def test_append_bad_slots_and_streams(cuda_lib):
    tok, Hq, Hkv, d, page = 24, 4, 2, 64, 16
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 5)
    x = [t[None] for t in (q, k, v)]
    cfg = msa.rope_cfg(d, norm=True)
    pages = msa.KV4Pages.empty(2, Hkv, page, d, "cuda")
    slots = torch.arange(tok, dtype=torch.int32, device="cuda")
    slots[3], slots[4] = 32, 1 << 30
    msa.qk_norm_rope_kv4(*x, cfg, pages, slots)
    assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX and cuda_lib.poll_device_status() == 0
    ref, _ = norm_rope(k, None, True, torch.tensor(1e-6, dtype=torch.float32).double().item(), d, _freq(d), False, torch.arange(tok, device="cuda"))
    keep = slots.clone()
    keep[3:5] = -1
    _check_held(pages.data, page, d, keep, ref, v.double(), torch.zeros_like(pages.data))
    want = pages.data.clone()
    slots = keep
    side, again = torch.cuda.Stream(), msa.KV4Pages.empty(2, Hkv, page, d, "cuda")
    side.wait_stream(torch.cuda.current_stream())
    msa.qk_norm_rope_kv4(*x, cfg, again, slots, stream=side)
    side.synchronize()
    assert torch.equal(again.data, want)
    again.data = torch.zeros_like(want)  # another tensor in its place is followed
    qo = torch.empty(1, Hq, tok, d, dtype=BF, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.qk_norm_rope_kv4(*x, cfg, again, slots, q=qo)
    for _ in range(2):
        again.data.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(again.data, want)


# ------------------------------------------------------------------ a cache with requests
class Cache:
    """Requests of the given lengths in a random 4-bit cache; scales of rows that hold no live token are NaN."""

    def __init__(self, Hq, Hkv, n, d, page, lens, seed, tls=None, masks=None, depths=None, sink=0, window=0, peak=4.0,
                 spare=3, width=0, k_scale=1.0, v_scale=1.0):
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
        data = torch.randint(0, 256, (N, Hkv, msa.kv4_page_bytes(page, d)), generator=g, device="cuda", dtype=torch.uint8)
        self.page, self.d, self.Hkv, self.sink, self.window = page, d, Hkv, sink, window
        for s in self._scales(data):
            s.fill_(NAN_SCALE)
        used = 0
        for b, c in enumerate(counts):
            table[b, :c] = perm[used:used + c]
            used += c
            if not c:
                continue
            ids = torch.from_numpy(table[b, :c]).cuda()
            for s, f in zip(self._scales(data), (peak, 1.0)):
                rows = torch.full((c * page, Hkv, d // 16), float("nan"), device="cuda")
                x = 0.35 * torch.exp(0.5 * torch.randn(self.lens[b], Hkv, d // 16, generator=g, device="cuda"))
                x[::5] *= f
                rows[:self.lens[b]] = x
                s[ids] = rows.to(torch.float8_e4m3fn).view(torch.uint8).view(c, page, Hkv, d // 16).transpose(1, 2)
        self.pages = msa.KV4Pages(data, page, d, k_scale, v_scale)
        self.table = table
        self.table_dev = torch.from_numpy(table.astype(np.int32)).cuda()
        self.lens_dev = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.tls_dev = None if tls is None else torch.tensor(self.tls, dtype=torch.int32, device="cuda")
        self.masks = masks
        self.words = None if masks is None else pack_mask(masks).cuda()
        self.depths = depths
        self.depths_dev = None if depths is None else torch.from_numpy(np.asarray(depths, np.int32)).cuda()
        self.q = torch.randn(B, Hq, n, d, generator=g, device="cuda").to(BF)
        if window:  # keys that no row sees: NaN, and pages without others are gone
            for b in range(B):
                lo, hi = sink, self.lens[b] - self.tls[b] - window + 1
                self.forget(b, lo, hi)

    def _scales(self, data):
        half, size = self.page * self.d // 2, self.page * (self.d // 2 + self.d // 16)
        return [data[..., w * size + half:(w + 1) * size].unflatten(-1, (self.page, self.d // 16)) for w in (0, 1)]

    def forget(self, b, lo, hi):
        """Tokens lo .. hi - 1 of request b."""
        P = self.page
        scales = self._scales(self.pages.data)
        for p in range(lo // P, -(-max(hi, 0) // P)):
            a, e = max(lo, p * P), min(hi, (p + 1) * P)
            if e <= a:
                continue
            for s in scales:
                s[self.table[b, p], :, a - p * P:e - p * P] = NAN_SCALE
            if a == p * P and e == (p + 1) * P:
                self.table_dev[b, p] = -7

    def run(self, **kw):
        B, Hq, n, d = self.q.shape
        o0 = torch.full((B, Hq, n, d), 7.0, dtype=BF, device="cuda")
        l0 = torch.full((B, Hq, n), 5.0, device="cuda")
        o, lse = o0.clone(), l0.clone()
        if self.window:
            kw.update(sink=self.sink, window=self.window, depth=self.depths_dev)
        msa.attn_tree_kv4(self.q, self.pages, self.table_dev, self.lens_dev, tree_len=self.tls_dev,
                          tree_mask=self.words, o=o, lse=lse, **kw)
        return o, lse, o0, l0

    def check(self, out, scale=None, what="", lens=None):
        lens = self.lens if lens is None else lens
        held = [None, None]

        def part(which):
            def rows(b, h):
                if h is None:
                    return self.Hkv
                if held[0] != b:
                    ids = torch.from_numpy(self.table[b, :-(-int(lens[b]) // self.page)]).cuda()
                    held[:] = b, kv4_values(self.pages.data[ids], self.page, self.d, self.pages.k_scale, self.pages.v_scale)
                return held[1][which][:, h].reshape(-1, self.d)[:int(lens[b])]
            return rows

        def seen(b):
            m = None if self.masks is None else self.masks if self.masks.ndim == 2 else self.masks[b]
            return seen_keys(int(lens[b]), self.tls[b], m, None if self.depths is None else self.depths[b], self.sink, self.window)

        o, lse, o0, l0 = out
        check_rows(self.q, part(0), part(1), lens, self.tls, seen, o, lse, o0, l0, scale, what, **KV4_WEIGHTS)


# ------------------------------------------------------------------ reading back
@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hkv,d", [(1, 64), (3, 64), (1, 128), (8, 128)])
def test_gather(cuda_lib, page, Hkv, d):
    lens = [0, 1, 15, 16, 17, 100, 127, 128, 129, 700]
    c = Cache(Hkv, Hkv, 1, d, page, lens, page + d, tls=[0] * len(lens), k_scale=4.0, v_scale=0.125)
    for n in (1, 130, 700, 1000):
        k0, v0 = (torch.full((len(lens), Hkv, n, d), 9.0, dtype=BF, device="cuda") for _ in range(2))
        k, v = msa.kv4_gather(c.pages, c.table_dev, c.lens_dev, n, k=k0.clone(), v=v0.clone())
        assert cuda_lib.poll_device_status() == 0
        for b, L in enumerate(lens):
            m = min(L, n)
            ids = torch.from_numpy(c.table[b, :-(-L // page)]).cuda()
            for got, ref, old in zip((k, v), kv4_values(c.pages.data[ids], page, d, 4.0, 0.125), (k0, v0)):
                ref = ref.transpose(0, 1).reshape(Hkv, -1, d)[:, :m]
                assert torch.equal(got[b, :, :m].double(), ref)  # bf16 holds every value exactly
                assert torch.equal(got[b, :, m:], old[b, :, m:])
    k, v = msa.kv4_gather(c.pages, c.table_dev, c.lens_dev, 50)
    assert not bool(k[0].any()) and not bool(v[1, :, 1:].any())  # what it allocates is zero behind a request's tokens


@pytest.mark.gpu
def test_gather_bad_requests_streams_and_capture(cuda_lib):
    c = Cache(2, 2, 1, 128, 16, [40, 50], 4)
    want = msa.kv4_gather(c.pages, c.table_dev, c.lens_dev, 64)
    assert cuda_lib.poll_device_status() == 0
    for change in ("long", "negative", "page", "page negative"):
        lens, table = c.lens_dev.clone(), c.table_dev.clone()
        if change == "long":
            lens[0] = 16 * table.shape[1] + 1
        if change == "negative":
            lens[0] = -1
        if change == "page":
            table[0, 1] = c.pages.data.shape[0]
        if change == "page negative":
            table[0, 1] = -1
        k, _ = msa.kv4_gather(c.pages, table, lens, 64)
        assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX, change
        assert torch.equal(k[1], want[0][1])  # the other request
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msa.kv4_gather(c.pages, c.table_dev, c.lens_dev, 64, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.kv4_gather(c.pages, c.table_dev, c.lens_dev, 64, k=out[0], v=out[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]) and cuda_lib.poll_device_status() == 0


# ------------------------------------------------------------------ attention
@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 1, 64), (4, 2, 128), (8, 8, 128), (7, 1, 64)])
def test_single_token(cuda_lib, Hq, Hkv, d, page):
    """Decode: one row per head, lengths around every page and tile border."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000, 2049]
    c = Cache(Hq, Hkv, 1, d, page, lens, 100 + page + d)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"decode {Hq}/{Hkv} d{d} page {page}")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,n,d", [(2, 1, 2, 64), (8, 2, 4, 128), (17, 1, 1, 128), (8, 2, 8, 128), (4, 1, 8, 64),
                                        (4, 1, 9, 128), (4, 1, 16, 64), (4, 1, 17, 128), (4, 1, 33, 128), (8, 1, 24, 64),
                                        (32, 8, 64, 128), (5, 5, 129, 64), (3, 1, 100, 64), (16, 2, 100, 128), (1, 1, 1024, 64)])
def test_trees(cuda_lib, Hq, Hkv, n, d):
    """Random trees, ragged, from 4 to 1024 rows a KV group."""
    rng = np.random.default_rng(n)
    B = 4
    tls = [n, max(1, n // 2), 1, 0]
    ctx = [0, 700, 128 - 1, 50]
    masks = np.stack([tree_bits(rng, n) for _ in range(B)])
    c = Cache(Hq, Hkv, n, d, 16, [a + b for a, b in zip(ctx, tls)], n, tls=tls, masks=masks)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"trees {Hq}/{Hkv} n{n} d{d}")


@pytest.mark.gpu
@pytest.mark.parametrize("n,page", [(1, 16), (5, 128), (40, 32), (70, 64)])
def test_chains_and_scales(cuda_lib, n, page):
    """No mask: drafted token i sees the drafted ones up to itself; scales of the caller's and of the tensors."""
    c = Cache(8, 2, n, 128, page, [n, n + 1, n + 127, n + 1000], 31 + n, k_scale=2.0 ** -6, v_scale=2.0 ** 11)
    out = c.run(scale=0.9)
    assert cuda_lib.poll_device_status() == 0
    c.check(out, scale=0.9, what=f"chain n{n}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [6, 40])
def test_rows_without_keys_and_shared_mask(cuda_lib, n):
    """A mask that names nothing for some rows (no context: o = 0, lse = -inf), one mask for all requests."""
    rng = np.random.default_rng(9)
    m = rng.random((n, n)) < 0.3
    m[1] = m[n - 1] = False
    c = Cache(8, 2, n, 64, 16, [n, n + 5, n - 2], 77, tls=[n, n, n - 2], masks=m)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    assert bool(torch.isneginf(out[1][0, :, 1]).all())
    c.check(out, what="empty rows")


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", [(0, 1), (0, 100), (3, 64), (64, 512), (128, 1024), (130, 100), (5000, 7), (1, 100000)])
@pytest.mark.parametrize("Hq,Hkv,n,d,page", [(4, 2, 1, 128, 16), (8, 2, 5, 64, 128), (4, 1, 40, 128, 32)])
def test_windows(cuda_lib, Hq, Hkv, n, d, page, sink, window):
    """Chains and trees through windows and sinks that end anywhere in tiles and pages; keys outside hold NaN, pages
    outside are gone."""
    rng = np.random.default_rng(n + window)
    lens = n + np.array([0, 1, 130, 700, 1500, 6000])
    for masked in (False, True):
        masks = depths = None
        if masked:
            masks = np.stack([tree_bits(rng, n) for _ in lens])
            depths = masks.sum(-1) - 1
        c = Cache(Hq, Hkv, n, d, page, lens, sink + window, masks=masks, depths=depths, sink=sink, window=window)
        out = c.run()
        assert cuda_lib.poll_device_status() == 0
        c.check(out, what=f"window {sink}+{window} masked {masked}")


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", [(0, 1), (0, 129), (200, 300), (3, 100000)])
@pytest.mark.parametrize("Hq,n,d,page", [(1, 64, 64, 16), (2, 128, 128, 128), (3, 192, 64, 64), (2, 512, 128, 32)])
def test_items_have_their_own_windows(cuda_lib, Hq, n, d, page, sink, window):
    """Chains whose items are 64 consecutive tokens: whole and short chunks, at the start of a prompt and far in."""
    lens = [n, 1, n + 77, 700, 5000, n + 4000, 300]
    tls = [n, 1, n, min(n, 600), n, 65 if n > 64 else 63, 0]
    c = Cache(Hq, 1, n, d, page, lens, n + window, tls=tls, sink=sink, window=window)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"items {n} {sink}+{window}")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 1, 1), (4, 1, 7), (4, 1, 17), (4, 1, 50), (6, 2, 100)])
def test_long_contexts_are_cut_and_joined(cuda_lib, Hq, Hkv, n, d):
    """One long request cut over all CTAs beside short ones; the same bits on every run."""
    rng = np.random.default_rng(n)
    lens = [60001, 5, 4097, 130]
    tls = [n, min(n, 5), max(1, n // 3), n]
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Cache(Hq, Hkv, n, d, 64, lens, 40 + n, tls=tls, masks=masks, peak=8.0)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="long")
    again = c.run()
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 1), (4, 2, 20), (4, 1, 8), (8, 2, 40)])
def test_items_across_many_cuts(cuda_lib, Hq, Hkv, n, page):
    """Requests of a few to a few hundred tiles, so that parts begin and end anywhere in items."""
    rng = np.random.default_rng(7 * n)
    lens = (n + np.exp(rng.uniform(0, math.log(30000), 24))).astype(int)
    tls = rng.integers(1, n + 1, len(lens))
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Cache(Hq, Hkv, n, 128, page, lens, 60 + n, tls=tls, masks=masks)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="cuts")


@pytest.mark.gpu
def test_large_scores_across_tiles(cuda_lib):
    """Scores that grow along the keys by tens from tile to tile and fall again, and all far below zero."""
    c = Cache(4, 2, 3, 128, 32, [900, 4000], 13, peak=1.0)
    ids = torch.from_numpy(c.table[1]).cuda()
    s = c._scales(c.pages.data)[0]
    ramp = torch.linspace(0, 12, len(ids) * 32, device="cuda")
    ramp = torch.where(ramp < 9, ramp, 18 - ramp)
    rows = (0.2 * (1 + ramp))[:, None, None].expand(-1, 2, 8).to(torch.float8_e4m3fn).view(torch.uint8)
    rows = rows.contiguous()
    rows[4000:] = NAN_SCALE
    s[ids] = rows.view(len(ids), 32, 2, 8).transpose(1, 2)
    c.q *= 4
    for sign in (1, -1):
        c.q *= sign
        out = c.run()
        assert cuda_lib.poll_device_status() == 0
        c.check(out, what=f"ramp {sign}")


@pytest.mark.gpu
def test_queries_of_any_size(cuda_lib):
    """Rows of q from bf16's smallest to sizes whose scores are thousands, zero rows, values far apart in one row: q's
    exponents are not the fp16 product's."""
    c = Cache(4, 1, 7, 64, 16, [300, 40], 17)
    size = torch.tensor([0.0, 1e-38, 1e-20, 1e-4, 1.0, 40.0, 900.0], device="cuda")
    c.q = (c.q.float() * size[:, None]).to(BF)
    c.q[0, 0, 4, 0] = 3e4
    c.q[0, 1, 4, 0] = 1e-30
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="sizes")
    c.q = (c.q.float() * 1e30).to(BF)  # scores that overflow the exponential's range, not fp32's
    c.q[..., 4:, :] = 0
    out = c.run(scale=1e-30)
    assert cuda_lib.poll_device_status() == 0
    c.check(out, scale=1e-30, what="large")


@pytest.mark.gpu
def test_masked_nan_keys(cuda_lib):
    """A NaN key that a row's mask leaves out does not reach that row (values stay finite)."""
    n = 4
    m = np.eye(n, dtype=bool)
    c = Cache(4, 1, n, 64, 16, [40], 3, masks=m[None])
    good = c.run()
    slot = 36 + 2  # key of drafted token 2
    c._scales(c.pages.data)[0][c.table[0][slot // 16], 0, slot % 16] = NAN_SCALE
    bad = c.run()
    assert cuda_lib.poll_device_status() == 0
    keep = [0, 1, 3]
    assert torch.equal(good[0][0, :, keep], bad[0][0, :, keep]) and torch.equal(good[1][0, :, keep], bad[1][0, :, keep])
    assert bool(bad[0][0, :, 2].isnan().all()) and bool(bad[1][0, :, 2].isnan().all())


@pytest.mark.gpu
def test_rows_not_drafted_hold_anything(cuda_lib):
    """NaN and infinities in rows of q behind a request's tokens change no bit of the others."""
    n = 6
    c = Cache(8, 2, n, 128, 16, [3000, 70], 23, tls=[2, 5])
    want = c.run()
    c.q[0, :, 2:] = float("nan")
    c.q[1, :, 5] = float("inf")
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.gpu
def test_empty_batch_and_many_requests(cuda_lib):
    """No drafted tokens anywhere; requests without any beside one that has some; more requests than threads of a CTA;
    two requests that read the same pages, a table wider than any needs."""
    c = Cache(4, 2, 3, 64, 16, [0, 20], 2, tls=[0, 0])
    c.check(c.run(), what="nothing")
    c = Cache(4, 2, 3, 64, 16, [0, 20, 0, 9, 0], 2, tls=[0, 0, 0, 2, 0])
    c.check(c.run(), what="one of five")
    rng = np.random.default_rng(8)
    c = Cache(2, 1, 1, 64, 16, rng.integers(1, 200, 900), 8)
    c.check(c.run(), what="900 requests")
    c = Cache(8, 2, 2, 128, 16, [100, 100], 21, width=600)
    c.table[1, :5] = c.table[0, :5]
    c.table_dev[1, :5] = c.table_dev[0, :5]
    c.check(c.run(), what="shared prefix")
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_bad_requests_are_reported(cuda_lib):
    """Lengths and page ids that break the contract set the error word; the context goes on."""
    for change in ("short", "long", "negative", "page", "page negative"):
        c = Cache(4, 2, 2, 64, 16, [40, 50], 4, tls=[2, 2])
        if change == "short":
            c.lens_dev[0] = 1
        if change == "long":
            c.lens_dev[0] = 16 * c.table.shape[1] + 1
        if change == "negative":
            c.tls_dev[0] = -1
        if change == "page":
            c.table_dev[0, 1] = c.pages.data.shape[0]
        if change == "page negative":
            c.table_dev[0, 1] = -1
        c.run()
        assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX, change
        assert cuda_lib.poll_device_status() == 0
    c = Cache(4, 2, 2, 64, 16, [40, 50], 4, tls=[2, 2])
    c.check(c.run(), what="after bad requests")


@pytest.mark.gpu
def test_streams_and_captures(cuda_lib):
    """Two calls at once on two streams; captured calls that follow lengths which change on the device."""
    a = Cache(8, 2, 4, 128, 64, [5000, 900, 33], 51)
    b = Cache(4, 1, 40, 128, 16, [3000, 77], 52)
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
        msa.attn_tree_kv4(a.q, a.pages, a.table_dev, a.lens_dev, o=o, lse=lse)
    for lens in ([5000, 900, 33], [4, 900, 20], [4999, 100, 4], [129, 128, 5]):
        a.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        a.check((o, lse, o, lse), what=f"replay {lens}", lens=lens)
    assert cuda_lib.poll_device_status() == 0


def _guarded(nbytes):
    whole = torch.full((nbytes + 512,), 255, dtype=torch.uint8, device="cuda")
    return whole, whole[256:256 + nbytes]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 1), (4, 1, 8), (4, 1, 16), (4, 1, 20), (4, 1, 48), (6, 1, 100)])
def test_workspace_of_the_stated_size(cuda_lib, Hq, Hkv, n, d):
    """Items cut many times and not at all: the stated bytes suffice, need no value before the call and give the bits of
    a workspace that the call allocates."""
    rng = np.random.default_rng(n + d)
    lens = [50001, n, n + 700, n + 4000]
    tls = [n, n, max(1, n // 2), 1]
    masks = np.stack([tree_bits(rng, n) for _ in lens])
    c = Cache(Hq, Hkv, n, d, 32, lens, 5 + n, tls=tls, masks=masks)
    whole, ws = _guarded(msa.attn_tree_kv4_workspace(len(lens), Hq, Hkv, n, d))
    out = c.run(ws=ws)
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="workspace")
    assert bool((whole[:256] == 255).all()) and bool((whole[-256:] == 255).all())
    own = c.run()
    assert torch.equal(out[0], own[0]) and torch.equal(out[1], own[1])


@pytest.mark.gpu
def test_workspace_reused_by_other_shapes(cuda_lib):
    """One workspace for calls of different shapes one after another."""
    rng = np.random.default_rng(17)
    cases = []
    for Hq, Hkv, n, d, lens in [(4, 1, 32, 128, [60000, 900]), (4, 1, 32, 128, [200, 129]), (4, 2, 3, 64, [30000, 7, 5000]),
                                (4, 1, 50, 128, [20000] * 3), (8, 8, 1, 128, [40, 300]), (4, 1, 50, 128, [260])]:
        masks = np.stack([tree_bits(rng, n) for _ in lens])
        cases.append(Cache(Hq, Hkv, n, d, 64, lens, 70 + n, masks=masks))
    need = max(msa.attn_tree_kv4_workspace(len(c.lens), *(c.q.shape[1], c.Hkv, *c.q.shape[2:])) for c in cases)
    whole, ws = _guarded(need)
    want = [c.run() for c in cases]
    for x in list(range(len(cases))) + rng.permutation(np.repeat(np.arange(len(cases)), 3)).tolist():
        got = cases[x].run(ws=ws)
        assert torch.equal(got[0], want[x][0]) and torch.equal(got[1], want[x][1]), x
    assert cuda_lib.poll_device_status() == 0
    for c, w in zip(cases, want):
        c.check(w, what="reused")
    assert bool((whole[:256] == 255).all()) and bool((whole[-256:] == 255).all())


@pytest.mark.gpu
def test_cache_beyond_32_bit_offsets(cuda_lib):
    """Pages whose byte offsets lie above 2^32: appended to, read back, attended to."""
    N, Hkv, page, d, Hq = 60000, 8, 64, 128, 32
    if torch.cuda.mem_get_info()[0] < 2 * N * Hkv * msa.kv4_page_bytes(page, d):
        pytest.skip("needs 9 GB")
    pages = msa.KV4Pages(torch.empty(N, Hkv, msa.kv4_page_bytes(page, d), dtype=torch.uint8, device="cuda"), page, d)
    ids = [N - 1, 0, N - 7, 58300, 32768 + 5]
    L = 5 * page - 9
    q, k, v, _ = _inputs(L, Hq, Hkv, d, 2)
    slots = torch.tensor([ids[t // page] * page + t % page for t in range(L)], dtype=torch.int32, device="cuda")
    qo, _, _ = msa.qk_norm_rope_kv4(q[None], k[None], v[None], msa.rope_cfg(0), pages, slots)
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    hk, hv = msa.kv4_gather(pages, table, lens, L)
    assert cuda_lib.poll_device_status() == 0
    for got, x in ((hk, k), (hv, v)):
        assert torch.equal(got[0].transpose(0, 1).double(), kv4_round(x.double())[0])
    rows = qo[:, :, -3:].contiguous()
    o, lse = torch.zeros_like(rows), torch.zeros(1, Hq, 3, device="cuda")
    msa.attn_tree_kv4(rows, pages, table, lens, o=o, lse=lse)
    assert cuda_lib.poll_device_status() == 0
    keys = lambda b, h: Hkv if h is None else hk[0, h]  # noqa: E731
    check_rows(rows, keys, lambda b, h: hv[0, h], [L], [3], lambda b: seen_keys(L, 3), o, lse, o, lse, what="far pages",
               **KV4_WEIGHTS)


@pytest.mark.gpu
def test_prompt_decode_and_continuation_together(cuda_lib):
    """As a server runs them: pages for two prompts, prompts into layer and 4-bit cache, decode steps through and
    without a window, then a second turn that continues a cached prompt with the prefill's kernels."""
    Hq, Hkv, d, page = 8, 2, 128, 16
    lens = [300, 1000]
    g = torch.Generator(device="cuda").manual_seed(4)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool = msa.PagePool.empty(2, 90, 170, page, "cuda")
    pages = msa.KV4Pages.empty(170, Hkv, page, d, "cuda")
    pages.data.fill_(NAN_SCALE)
    w = (1 + 0.2 * torch.randn(2, d, generator=g, device="cuda")).to(BF)
    cfg = msa.rope_cfg(d, norm=True, q_weight=w[0], k_weight=w[1])

    def project(*lead):
        x = torch.randn(*lead, Hq + 2 * Hkv, d, generator=g, device="cuda").to(BF)
        return x.split([Hq, Hkv, Hkv], -2)

    q, k, v = project(sum(lens))
    _, slots, pos = msa.build_page_tables(pool, torch.tensor(lens, **i32), tok_cap=sum(lens))
    ql, kl, vl = msa.qk_norm_rope_varlen_kv4(q, k, v, [0, 300, 1300], cfg, pages, slots, positions=pos, layer_kv=True)
    exact = [torch.cat([s.transpose(0, 1) for s in msa.unpack_varlen(t, Hkv, [0, 300, 1300], d)]) for t in (kl, vl)]
    for step in range(3):
        q, k, v = project(2, 1)
        _, slots, pos = msa.build_page_tables(pool, pool.seq_len + 1, seq_tokens=1)
        qd, _, _ = msa.qk_norm_rope_kv4(q, k, v, cfg, pages, slots, positions=pos)
        lse = torch.zeros(2, Hq, 1, device="cuda")
        held = msa.kv4_gather(pages, pool.page_table, pool.seq_len, 1003)
        now = pool.seq_len.tolist()
        assert now == [301 + step, 1001 + step]
        for sink, window in ((0, 0), (16, 200)):
            o = msa.attn_tree_kv4(qd, pages, pool.page_table, pool.seq_len, sink=sink, window=window, lse=lse)
            assert cuda_lib.poll_device_status() == 0
            part = lambda t: lambda b, h: Hkv if h is None else t[b, h, :now[b]]  # noqa: E731
            check_rows(qd, part(held[0]), part(held[1]), now, [1, 1], lambda b: seen_keys(now[b], 1, sink=sink, window=window),
                       o, lse, o, lse, what=f"step {step}", **KV4_WEIGHTS)
    # the cache is near the exact keys and values (a value is off by a sixth of its block's largest at most, and the
    # scale's rounding by 1/16 of it)
    for t, x in zip(held, exact):
        for b, (a, e) in enumerate(((0, 300), (300, 1300))):
            got, ref = t[b, :, :e - a].transpose(0, 1).float(), x[a:e].float()
            big = ref.unflatten(-1, (-1, 16)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 16).flatten(-2)
            assert bool(((got - ref).abs() <= big * (1 / 6 + 1 / 16) * 1.01).all())
    # a second turn of request 1: 128 tokens behind its cached prefix, through the prefill's kernel
    n = 128
    L = now[1]
    q, k, v = project(1, n)
    _, slots, pos = msa.build_page_tables(pool, pool.seq_len + torch.tensor([0, n], **i32), tok_cap=n)
    qc, kc, vc = msa.qk_norm_rope_kv4(q, k, v, cfg, pages, slots, positions=pos, layer_kv=True)
    K, V = msa.kv4_gather(pages, pool.page_table[1:], pool.seq_len[1:], L + n)
    Q = torch.zeros(1, Hq, L + n, d, dtype=BF, device="cuda")
    Q[:, :, L:] = qc
    want = msa.attn_dense(Q, K, V, list(range(Hq)))[:, :, L:]
    got = msa.attn_tree_kv4(qc, pages, pool.page_table[1:].contiguous(), pool.seq_len[1:].contiguous())
    assert cuda_lib.poll_device_status() == 0
    assert float((got.float() - want.float()).abs().max()) <= 1.5e-2 + 2.0 ** -7 * float(V.float().abs().max())
    check_rounded(kc[0].transpose(0, 1), *norm_rope(k[0], w[1], True, 1e-6, d, _freq(d), False, pos), "layer keys")


def _fill_shared_memory(word):
    """Leave the 16-bit `word` in the shared memory that holds keys and values of msa_attn_tree, on every SM."""
    Hkv, page, d, pages = 8, 128, 128, 128
    kv = torch.full((pages, Hkv, page, d), word, dtype=torch.int16, device="cuda").view(BF)
    q = torch.zeros(1, Hkv, 1, d, dtype=BF, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    msa.attn_tree(q, kv, kv, table, torch.tensor([pages * page], dtype=torch.int32, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n", [(4, 2, 3), (4, 1, 4), (4, 1, 8), (2, 1, 32), (4, 1, 40)])
def test_bits_do_not_depend_on_what_ran_before(cuda_lib, Hq, Hkv, n, d):
    """Rows that are not drafted have no say in the others' references, whatever shared memory holds in their place: fp16
    numbers, NaN or infinities.  Their windows begin behind a group's first tile."""
    rng = np.random.default_rng(n)
    window = 2000  # items of 17 tiles, parts of several tiles
    lens = [128 * int(rng.integers(8, 40)) + window + 127 - x % 4 for x in range(80)]  # the first row sees a few keys of its first tile
    tls = [1 + x % min(n, 3) for x in range(80)]
    for w in (0, window):
        c = Cache(Hq, Hkv, n, d, 16, lens, n + d, tls=tls, window=w)
        outs = []
        for word in (0x3C00, 0x7C01, 0x7C00, -0x0400, 0):  # fp16: 1, NaN, infinity, -infinity, 0
            _fill_shared_memory(word)
            outs.append(c.run())
        assert cuda_lib.poll_device_status() == 0
        c.check(outs[0], what=f"window {w}")
        for word, out in enumerate(outs):
            assert torch.equal(out[0], outs[0][0]) and torch.equal(out[1], outs[0][1]), (w, word)


def _check_held_with_nan(data, page, d, slots, k, v, ks=1.0, vs=1.0):
    """As _check_held for the tokens' own slots; a NaN value makes its block NaN, by its scale."""
    rows = [t.transpose(1, 2).reshape(-1, *t.shape[1:2], d) for t in kv4_values(data, page, d, ks, vs)]
    for got, x, s, what in ((rows[0], k, ks, "K"), (rows[1], v, vs, "V")):
        got, want = got[slots.long()], kv4_round(x, s)[0]
        assert torch.equal(got.isnan(), want.isnan()), f"{what}: {int((got.isnan() != want.isnan()).sum())} NaN differ"
        assert torch.equal(got.nan_to_num(), want.nan_to_num()), f"{what}: {int((got != want).sum())} values differ"


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot,inter,norm", [(0, False, False), (None, False, False), (48, True, False), (None, False, True),
                                            (16, True, True)])
def test_append_keeps_nan(cuda_lib, d, rot, inter, norm):
    """A NaN in a key or value, and what the norm makes of a head that holds one or (eps 0) of zeros alone, stays one in
    the cache, where reading back and attention find it; other blocks and heads are as without."""
    rot = d if rot is None else rot
    tok, Hq, Hkv, page = 12, 4, 2, 16
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 41 + d)
    nan = float("nan")
    k[1, 0, 3] = k[2, 1, d - 1] = v[3, 0, 17] = v[4, 1, 0] = nan
    k[5, 0] = 0
    k[6, 1, :20] = nan
    k[7], v[8] = nan, nan
    cfg = msa.rope_cfg(rot, interleaved=inter, norm=norm, eps=0.0, q_weight=w[0], k_weight=w[1])
    pages = msa.KV4Pages.empty(1, Hkv, page, d, "cuda")
    slots = torch.arange(tok, dtype=torch.int32, device="cuda")
    pos = torch.arange(5, 5 + tok, dtype=torch.int32, device="cuda")
    qo, _, _ = msa.qk_norm_rope_kv4(q[None], k[None], v[None], cfg, pages, slots, positions=pos)
    assert cuda_lib.poll_device_status() == 0
    ref, _ = norm_rope(k, w[1], norm, 0.0, rot, _freq(rot), inter, pos)
    assert bool(ref[1, 0].isnan().any()) and bool(ref[5, 0].isnan().all()) == norm
    _check_held_with_nan(pages.data, page, d, slots, ref, v.double())
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens = torch.zeros(1, 1, **i32), torch.tensor([tok], **i32)
    hk, hv = msa.kv4_gather(pages, table, lens, tok)
    assert bool(hk[0, 0, 1].isnan().any()) and bool(hv[0, 0, 3, 16:32].isnan().all()) and not bool(hv[0, 0, 3, :16].isnan().any())
    o = msa.attn_tree_kv4(qo[:, :, :1].contiguous(), pages, table, lens)
    assert bool(o[0, :2].isnan().all())  # a NaN key of their KV head
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("ks,vs", [(1.0, 1.0), (2.0 ** -40, 2.0 ** -40), (2.0 ** 40, 2.0 ** 40)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot,inter", [(0, False), (None, False), (48, False), (None, True), (16, True)])
def test_append_infinities_and_values_past_any_scale(cuda_lib, d, rot, inter, ks, vs):
    """Infinities, and finite values that the tensor's scale takes past fp32, are held as the largest number; the others
    of their block by the largest scale, other blocks as without them."""
    rot = d if rot is None else rot
    tok, Hq, Hkv, page = 16, 4, 2, 16
    q, k, v, _ = _inputs(tok, Hq, Hkv, d, 43 + d)
    k[4:8] *= 100 * ks if ks > 1 else 300
    v[4:8] *= 100 * vs if vs > 1 else 300
    inf = float("inf")
    for x in (k, v):
        x[1, 0, 3], x[2, 1, d - 1], x[3, 0, 17] = inf, -inf, 3e38
        x[4, 0, 9], x[5, 1, 30], x[6, 0, 0] = -3e38, inf, 2e30
        x[6, 1, 31], x[7, 0, 2], x[7, 0, 3] = -1e27, inf, -inf
        x[8, 0], x[9, 1] = inf, -1e38
    cfg = msa.rope_cfg(rot, interleaved=inter)
    pages = msa.KV4Pages.empty(1, Hkv, page, d, "cuda", ks, vs)
    slots = torch.arange(tok, dtype=torch.int32, device="cuda")
    pos = torch.arange(3, 3 + tok, dtype=torch.int32, device="cuda")
    msa.qk_norm_rope_kv4(q[None], k[None], v[None], cfg, pages, slots, positions=pos)
    assert cuda_lib.poll_device_status() == 0
    ref, _ = norm_rope(k, None, False, 0.0, rot, _freq(rot), inter, pos)
    _check_held_with_nan(pages.data, page, d, slots, ref, v.double(), ks, vs)


def test_replaced_data_is_checked_by_every_call():
    """KV4Pages.data in whose place something else was put: a ValueError that names it, from each of the calls."""
    i32 = dict(dtype=torch.int32)
    q, x = torch.zeros(2, 4, 3, 64, dtype=BF), torch.zeros(2, 5, 8, 64, dtype=BF)
    qi, ki, vi = x.split([4, 2, 2], 2)
    table, lens = torch.zeros(2, 4, **i32), torch.ones(2, **i32)
    cfg, slots = msa.rope_cfg(64), torch.zeros(10, **i32)
    pages = msa.KV4Pages.empty(9, 2, 16, 64, "cpu")
    for data, what in ((None, "data: a 3-d"), (torch.zeros(9, dtype=torch.uint8), "data: a 3-d"),
                       (torch.zeros(9, 2, 16 * 72), "data: dtype"), (torch.zeros(9, 2, 7, dtype=torch.uint8), "data: shape")):
        pages.data = data
        for call in (lambda: msa.kv4_gather(pages, table, lens, 8), lambda: msa.attn_tree_kv4(q, pages, table, lens),
                     lambda: msa.qk_norm_rope_kv4(qi, ki, vi, cfg, pages, slots)):
            with pytest.raises(ValueError, match=what):
                call()


@pytest.mark.gpu
@pytest.mark.parametrize("inter,norm", [(False, True), (True, False)])
def test_append_at_far_positions(cuda_lib, inter, norm):
    """Positions up to 2^31 - 1 and negative ones.  An angle is off by |position| 2^-60 (its frequency by two units of
    2^-64 turns: 2 pi 2^-63 < 2^-60), the sums by 2^-40 of a pair's size: codes and scales are those of a value that near
    the exact one, and nearly all are the exact one's."""
    tok, Hq, Hkv, d, page = 512, 4, 4, 128, 64
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 91)
    rng = np.random.default_rng(9)
    p = rng.integers(-(1 << 31), 1 << 31, tok)
    p[:4] = [0, (1 << 31) - 1, -(1 << 31), -1]
    pos = torch.from_numpy(p.astype(np.int32)).cuda()
    # multiples of 2^-20: position * f is exact in 64 bits, so the reference has the true angle (as have its sines)
    freq = (rng.integers(-(1 << 20), 1 << 20, d // 2) / 2.0 ** 20).tolist()
    eps = torch.tensor(1e-6, dtype=torch.float32).double().item()
    cfg = msa.rope_cfg(d, norm=norm, interleaved=inter, inv_freq=freq, k_weight=w[1] if norm else None)
    pages = msa.KV4Pages.empty(tok // page, Hkv, page, d, "cuda")
    slots = torch.arange(tok, dtype=torch.int32, device="cuda")
    msa.qk_norm_rope_kv4(q[None], k[None], v[None], cfg, pages, slots, positions=pos)
    assert cuda_lib.poll_device_status() == 0
    y, slack = norm_rope(k, w[1] if norm else None, norm, eps, d, freq, inter, pos)
    size = slack / (2.0 ** -24 * 32)  # of the value's pair
    e = size * (2.0 ** -40 + pos.double().abs()[:, None, None] * 2.0 ** -60)
    held = kv4_values(pages.data, page, d)[0].transpose(1, 2).reshape(tok, Hkv, d)
    scales = pages.data[..., page * d // 2:page * (d // 2 + d // 16)].unflatten(-1, (page, d // 16)).transpose(1, 2)
    scales = scales.contiguous().view(torch.float8_e4m3fn).double().reshape(tok, Hkv, d // 16)
    # a block's scale lies between those of its values less and more what they may be off
    low, high = (kv4_round(torch.copysign((y.abs() + x).clamp(min=0), y))[2].view(torch.float8_e4m3fn).double() for x in (-e, e))
    assert bool((low <= scales).all()) and bool((scales <= high).all())
    s = scales.repeat_interleave(16, -1)

    def code(x):  # the e2m1 number nearest x / s
        t = (x / s).clamp(-6, 6)
        unit = torch.where(t.abs() < 2, 0.5, torch.where(t.abs() < 4, 1.0, 2.0))
        return torch.round(t / unit) * unit

    assert bool((s > 0).all()) and bool((code(y - e) <= held / s).all()) and bool((held / s <= code(y + e)).all())
    assert float((held == kv4_round(y)[0]).double().mean()) > 0.9999


@pytest.mark.gpu
@pytest.mark.parametrize("sink,window", [(0, 100), (3, 64), (200, 300), (128, 1024)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,n,page", [(6, 2, 2, 32), (8, 2, 3, 16), (4, 1, 4, 64), (4, 1, 5, 128), (4, 1, 8, 16), (4, 1, 12, 32)])
def test_windows_of_every_row_width(cuda_lib, Hq, Hkv, n, page, d, sink, window):
    """6, 12, 16, 20, 32 and 48 rows a KV head, whole and ragged, in products of 8, 16, 32 and 64 rows."""
    rng = np.random.default_rng(n + window)
    lens = n + np.array([0, 1, 130, 700, 1500, 6000])
    for masked in (False, True):
        masks = depths = None
        if masked:
            masks = np.stack([tree_bits(rng, n) for _ in lens])
            depths = masks.sum(-1) - 1
        tls = [n, 1, max(1, n // 2), n, 0, n - 1]
        c = Cache(Hq, Hkv, n, d, page, lens, sink + window + d, tls=tls, masks=masks, depths=depths, sink=sink, window=window)
        out = c.run()
        assert cuda_lib.poll_device_status() == 0
        c.check(out, what=f"window {sink}+{window} masked {masked}")


@pytest.mark.gpu
@pytest.mark.parametrize("n,d", [(128, 128), (1024, 64), (200, 128)])
def test_the_next_chunk_of_a_prompt(cuda_lib, n, d):
    """Many tokens behind a cached prefix, without a window: every row against the definition over what the cache holds,
    and the chunk read back and attended to by the prefill's dense kernel."""
    Hq, Hkv, page = 4, 2, 32
    L = 1003
    c = Cache(Hq, Hkv, n, d, page, [L + n, n], n + d)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what="chunk")
    K, V = msa.kv4_gather(c.pages, c.table_dev, c.lens_dev, L + n)
    Q = torch.zeros(1, Hq, L + n, d, dtype=BF, device="cuda")
    Q[:, :, L:] = c.q[:1]
    dense_lse = torch.zeros(1, Hq, L + n, device="cuda")
    dense = msa.attn_dense(Q, K[:1], V[:1], list(range(Hq)), lse=dense_lse)
    assert cuda_lib.poll_device_status() == 0
    # the same rows by the prefill's kernel, whose weights are bf16
    rows, lse = dense[:, :, L:].contiguous(), dense_lse[:, :, L:].contiguous()
    check_rows(c.q[:1], lambda b, h: Hkv if h is None else K[0, h], lambda b, h: V[0, h], [L + n], [n],
               lambda b: seen_keys(L + n, n), rows, lse, rows, lse, what="dense")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,n,B", [(2, 1, 1, 2600), (4, 1, 12, 1700)])
@pytest.mark.parametrize("window", [0, 150])
def test_more_requests_than_threads(cuda_lib, Hq, Hkv, n, B, window):
    """Several requests for each thread that adds up the tiles, some of them empty."""
    rng = np.random.default_rng(B + window)
    tls = rng.integers(0, n + 1, B) if n > 1 else (rng.random(B) < 0.9).astype(int)
    c = Cache(Hq, Hkv, n, 64, 16, tls + rng.integers(0, 300, B), B, tls=tls, sink=5 if window else 0, window=window)
    out = c.run()
    assert cuda_lib.poll_device_status() == 0
    c.check(out, what=f"{B} requests")


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,n,d", [(4, 2, 6, 128), (2, 1, 40, 64)])
def test_masks_of_windows(cuda_lib, Hq, Hkv, n, d):
    """One mask for all requests, depths with it and without (a row's index stands in), rows whose mask names nothing
    and whose window holds nothing."""
    rng = np.random.default_rng(3)
    m = rng.random((n, n)) < 0.3
    m[1] = m[n - 1] = False
    lens = [n, n + 1, n + 5, n + 700, n + 130, n + 2000]
    tls = [n, n, n - 1, n, n // 2, n]
    for depths in (None, np.tile(rng.integers(0, n, n), (len(lens), 1))):
        for sink, window in ((0, 1), (2, 3), (0, 300), (130, 200)):
            c = Cache(Hq, Hkv, n, d, 16, lens, 7, tls=tls, masks=m, depths=depths, sink=sink, window=window)
            out = c.run()
            assert cuda_lib.poll_device_status() == 0
            c.check(out, what=f"masks {sink}+{window}")
    assert bool(torch.isneginf(out[1][0, :, 1]).all())  # no context, no drafted key


@pytest.mark.gpu
def test_two_graphs_of_one_workspace(cuda_lib):
    """Captured calls of different shapes that share a workspace, replayed in turn, and an eager one between."""
    a = Cache(4, 1, 8, 128, 64, [40000, 300], 1)
    b = Cache(8, 2, 20, 64, 16, [3000, 9000, 21], 2, sink=16, window=600)
    want = [c.run() for c in (a, b)]
    ws = torch.empty(max(msa.attn_tree_kv4_workspace(len(c.lens), *c.q.shape[1:2], c.Hkv, *c.q.shape[2:]) for c in (a, b)),
                     dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in (a, b):
        graph = torch.cuda.CUDAGraph()
        c.run(ws=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs.append(c.run(ws=ws))
        graphs.append(graph)
    for x in (0, 1, 1, 0, 0, 1, 0):
        for t in outs[x][:2]:
            t.zero_()
        graphs[x].replay()
        y = (a, b)[x ^ 1].run(ws=ws)
        torch.cuda.synchronize()
        for got, ref in ((outs[x], want[x]), (y, want[x ^ 1])):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), x
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_append_many_sequences(cuda_lib):
    """More packed sequences than one launch takes, empty ones among them, positions given and not."""
    Hq, Hkv, d, page = 2, 1, 64, 16
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 6, 2500)
    cu = np.concatenate([[0], np.cumsum(lens)])
    tok = int(cu[-1])
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 8)
    N = -(-tok // page) + 1
    slots = torch.from_numpy(rng.permutation(N * page)[:tok].astype(np.int32)).cuda()
    cfg = msa.rope_cfg(d, norm=True, q_weight=w[0], k_weight=w[1])
    eps = torch.tensor(1e-6, dtype=torch.float32).double().item()
    own = torch.from_numpy((np.arange(tok) - np.repeat(cu[:-1], lens)).astype(np.int32)).cuda()
    for pos in (None, torch.from_numpy(rng.integers(0, 100000, tok).astype(np.int32)).cuda()):
        pages = msa.KV4Pages.empty(N, Hkv, page, d, "cuda")
        before = pages.data.clone()
        qo, _, _ = msa.qk_norm_rope_varlen_kv4(q, k, v, cu, cfg, pages, slots, positions=pos)
        want, _, _ = msa.qk_norm_rope_varlen(q, k, v, cu, cfg, positions=pos)
        assert cuda_lib.poll_device_status() == 0
        assert torch.equal(qo, want)
        ref, _ = norm_rope(k, w[1], True, eps, d, _freq(d), False, own if pos is None else pos)
        _check_held(pages.data, page, d, slots, ref, v.double(), before)
