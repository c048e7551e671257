"""Per-head norms of queries and keys with the rotation (msa_qk_norm_rope).

CPU: host checks.  GPU: every value against the formula in 64 bits, within the
fp32 bound of paged_ref.norm_rope and one bf16 rounding; V and the cache's
other rows bit for bit."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_prefill_gb300 as msa
from paged_ref import check_rounded, norm_rope

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_gb300 import build
    build.build()
    return msa.load()


def test_refusals(lib):
    P = ctypes.c_void_p
    inv, uns = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_UNSUPPORTED
    a = {k: P(0x100000 * (x + 1)) for x, k in enumerate(("q_in", "k_in", "v_in", "pos", "q", "k", "v", "slots"))}

    def call(shape=None, cfg=None, qs=512, ks=256, vs=256, pages=None, **kw):
        sh = dict(B=1, Hq=4, Hkv=2, n=8, d_h=128, scale=0.0)
        sh.update(shape or {})
        c = dict(norm=1, eps=1e-6, q_weight=None, k_weight=None, rot_dim=128, interleaved=0, theta=1e4, inv_freq=None,
                 rot_scale=1.0)
        c.update(cfg or {})
        x = dict(a, slots=None)
        x.update(kw)
        return lib.msa_qk_norm_rope(ctypes.byref(msa.Shape(**sh)), ctypes.byref(msa.RopeCfgC(**c)), x["q_in"], qs,
                                    x["k_in"], ks, x["v_in"], vs, x["pos"], x["q"], x["k"], x["v"],
                                    None if pages is None else ctypes.byref(pages), x["slots"], None)

    assert call(shape=dict(d_h=96)) == uns
    assert call(shape=dict(Hq=3)) == inv
    assert call(cfg=dict(rot_dim=24)) == uns
    assert call(cfg=dict(rot_dim=144)) == inv
    assert call(cfg=dict(rot_dim=-16)) == inv
    assert call(cfg=dict(norm=2)) == inv
    assert call(cfg=dict(eps=-1.0)) == inv
    assert call(cfg=dict(eps=float("nan"))) == inv
    assert call(cfg=dict(theta=float("inf"))) == inv
    assert call(cfg=dict(theta=float("nan"))) == inv
    assert call(cfg=dict(rot_scale=float("nan"))) == inv
    bad = (ctypes.c_double * 64)(*([float("nan")] * 64))
    assert call(cfg=dict(inv_freq=bad)) == inv
    assert call(qs=504) == inv
    assert call(ks=260) == inv  # not a multiple of 8 elements
    assert call(q_in=P(0x100008)) == inv
    assert call(q_in=None) == inv
    assert call(k=None, v=None) == inv                     # no destination
    assert call(v=None) == inv                             # values read and dropped
    assert call(v_in=None) == inv                          # values written from nothing
    assert call(q=a["q_in"]) == inv                        # in place
    assert call(slots=a["slots"]) == inv                   # slots without pages
    pages = msa.KVPagesC(0x10000000, 0x20000000, 8, 16)
    assert call(pages=pages) == inv                        # pages without slots
    assert call(pages=msa.KVPagesC(0x10000000, 0x20000000, 8, 24), slots=a["slots"]) == uns
    assert call(pages=msa.KVPagesC(0x10000000, None, 8, 16), slots=a["slots"]) == inv
    sh, c = msa.Shape(1, 4, 2, 1, 128, 0.0), msa.rope_cfg(128).c

    def varlen(cu):
        arr = (ctypes.c_int32 * len(cu))(*cu)
        return lib.msa_qk_norm_rope_varlen(ctypes.byref(sh), arr, len(cu) - 1, ctypes.byref(c), a["q_in"], 512,
                                           a["k_in"], 256, a["v_in"], 256, None, a["q"], a["k"], a["v"], None, None,
                                           None)
    assert varlen([1, 5]) == inv
    assert varlen([0, 5, 4]) == inv
    assert varlen([0, 0, 0]) == msa.MSA_OK  # nothing to do
    a = dict.fromkeys(a)
    assert varlen([0, 0, 0]) == msa.MSA_OK  # empty tensors have no address
    assert varlen([0, 5]) == inv


def test_binding_refusals():
    x = torch.zeros(2, 5, 8, 64, dtype=BF)
    q, k, v = x.split([4, 2, 2], 2)
    cfg = msa.rope_cfg(64, norm=True, q_weight=torch.ones(64, dtype=BF))
    for call, what in [
        (lambda: msa.qk_norm_rope(q, k, v, cfg), "q_in: must be on a CUDA device"),
        (lambda: msa.qk_norm_rope(q[0], k, v, cfg), "q_in: a 4-d"),
        (lambda: msa.qk_norm_rope(q, k[:, :4], v, cfg), "k_in: leading"),
        (lambda: msa.qk_norm_rope(q, k, v[..., :1, :], cfg), "v_in: heads"),
        (lambda: msa.qk_norm_rope(q.float(), k, v, cfg), "q_in: dtype"),
        (lambda: msa.qk_norm_rope(q[..., ::2, :], k, v, cfg), "q_in: the heads"),
        (lambda: msa.qk_norm_rope(q[:, ::2], k[:, ::2], v[:, :3], cfg), "tokens must lie at one stride"),
        (lambda: msa.qk_norm_rope(q, k, v, msa.rope_cfg(64, norm=True, q_weight=torch.ones(32, dtype=BF))), "q_weight: shape"),
        (lambda: msa.qk_norm_rope(q, k, v, cfg, positions=torch.zeros(9, dtype=torch.int32)), "positions: 9 elements"),
        (lambda: msa.qk_norm_rope(q, k, v, cfg, q=torch.zeros(2, 4, 4, 64, dtype=BF)), "q: shape"),
        (lambda: msa.qk_norm_rope(q, k, v, cfg, k_pages=torch.zeros(3, 2, 16, 64, dtype=BF)), "v_pages: a torch"),
        (lambda: msa.qk_norm_rope(q, k, v, cfg, v_pages=torch.zeros(3, 2, 16, 64, dtype=BF)), "k_pages: a 4-d"),
        (lambda: msa.qk_norm_rope_varlen(q[0], k[0], v[0], [0, 4], cfg), "cu_seqlens: must end"),
        (lambda: msa.rope_cfg(64, inv_freq=[1.0] * 31), "inv_freq: 31 values"),
    ]:
        with pytest.raises(ValueError, match=what):
            call()


def _freq(rot, theta=10000.0):
    return [theta ** (-2 * i / rot) for i in range(rot // 2)] if rot else []


def _inputs(tok, Hq, Hkv, d, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tok, (Hq + 2 * Hkv) * d + pad, generator=g, device="cuda") * 3
    x = x.to(BF)
    w = (1 + 0.5 * torch.randn(2, d, generator=g, device="cuda")).to(BF)
    q, k, v = (t.unflatten(1, (-1, d)) for t in x[:, :(Hq + 2 * Hkv) * d].split([Hq * d, Hkv * d, Hkv * d], 1))
    return q, k, v, w


def _check(got, x, w, cfgd, pos, what):
    y, slack = norm_rope(x, w, cfgd["norm"], cfgd["eps"], cfgd["rot"], cfgd["freq"], cfgd["inter"], pos,
                         cfgd.get("scale", 1.0))
    check_rounded(got, y, slack, what)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rot", [0, 16, 48, None])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_layer_and_cache(cuda_lib, d, rot, inter, norm):
    rot = d if rot is None else rot
    B, n, Hq, Hkv, page = 3, 37, 6, 2, 16
    tok = B * n
    q, k, v, w = _inputs(tok, Hq, Hkv, d, d + rot, pad=24)
    rng = np.random.default_rng(rot)
    pos = torch.from_numpy(rng.integers(0, 1 << 20, tok).astype(np.int32)).cuda()
    slots = torch.from_numpy(rng.permutation(tok + 40)[:tok].astype(np.int32)).cuda()
    slots[5] = -1  # a padding token: not stored
    N = -(-(tok + 40) // page)
    cfg = msa.rope_cfg(rot, interleaved=inter, norm=norm, eps=1e-5, q_weight=w[0], k_weight=w[1])
    kp, vp = (torch.full((N, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    shaped = [t.unflatten(0, (B, n)) for t in (q, k, v)]
    qo, ko, vo = msa.qk_norm_rope(*shaped, cfg, positions=pos, k_pages=kp, v_pages=vp, slots=slots)
    assert cuda_lib.poll_device_status() == 0
    c = dict(norm=norm, eps=1e-5, rot=rot, freq=_freq(rot), inter=inter)
    back = lambda t: t.transpose(1, 2).reshape(tok, -1, d)  # noqa: E731
    _check(back(qo), q, w[0], c, pos, "q")
    _check(back(ko), k, w[1], c, pos, "k")
    assert torch.equal(back(vo), v)
    keep = torch.arange(tok, device="cuda") != 5
    rows = lambda t: t.transpose(1, 2).reshape(-1, Hkv, d)  # noqa: E731
    assert torch.equal(rows(kp)[slots[keep].long()], back(ko)[keep])
    assert torch.equal(rows(vp)[slots[keep].long()], v[keep])
    other = torch.ones(N * page, dtype=torch.bool, device="cuda")
    other[slots[keep].long()] = False
    assert bool(rows(kp)[other].isnan().all()) and bool(rows(vp)[other].isnan().all())  # left as they were


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,lens", [(5, 1, 64, [1]), (8, 8, 128, [3, 0, 130, 1, 64]), (4, 2, 128, [700, 0, 0, 1]),
                                           (32, 8, 128, [257, 1000])])
def test_varlen_layout(cuda_lib, Hq, Hkv, d, lens):
    cu = np.concatenate([[0], np.cumsum(lens)])
    tok = int(cu[-1])
    q, k, v, w = _inputs(tok, Hq, Hkv, d, tok)
    cfg = msa.rope_cfg(d, theta=500000.0, norm=True, q_weight=w[0])  # k: no weight
    qo, ko, vo = msa.qk_norm_rope_varlen(q, k, v, cu, cfg)
    pos = torch.cat([torch.arange(x) for x in lens]).int().cuda()
    c = dict(norm=True, eps=1e-6, rot=d, freq=_freq(d, 500000.0), inter=False)
    for t, x, ww, H in ((qo, q, w[0], Hq), (ko, k, None, Hkv)):
        seqs = msa.unpack_varlen(t, H, cu, d)
        _check(torch.cat([s.transpose(0, 1) for s in seqs]), x, ww, c, pos, "varlen")
    assert torch.equal(torch.cat([s.transpose(0, 1) for s in msa.unpack_varlen(vo, Hkv, cu, d)]), v)


@pytest.mark.gpu
def test_many_sequences(cuda_lib):
    """More sequences than one launch's table holds."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 4, 2500)
    cu = np.concatenate([[0], np.cumsum(lens)])
    tok = int(cu[-1])
    q, k, v, w = _inputs(tok, 2, 1, 64, 9)
    qo, ko, vo = msa.qk_norm_rope_varlen(q, k, v, cu, msa.rope_cfg(64))
    pos = torch.from_numpy(np.concatenate([np.arange(x) for x in lens]).astype(np.int32)).cuda()
    c = dict(norm=False, eps=0.0, rot=64, freq=_freq(64), inter=False)
    _check(torch.cat([s.transpose(0, 1) for s in msa.unpack_varlen(qo, 2, cu, 64)]), q, None, c, pos, "q")


@pytest.mark.gpu
def test_far_positions_given_angles_and_factor(cuda_lib):
    """Angles of positions up to 2^31 - 1, negative ones, angles above a turn, a factor on the rotation."""
    tok, Hq, Hkv, d = 64, 4, 2, 128
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 77)
    rng = np.random.default_rng(7)
    p = rng.integers(-(1 << 31), 1 << 31, tok)
    p[:4] = [0, (1 << 31) - 1, -(1 << 31), -1]
    pos = torch.from_numpy(p.astype(np.int32)).cuda()
    # multiples of 2^-20: position * f is exact in 64 bits, so the reference has the true angle
    freq = (rng.integers(-(1 << 22), 1 << 22, d // 2) / 2.0 ** 20).tolist()
    cfg = msa.rope_cfg(d, inv_freq=freq, rot_scale=1.25)
    qo, _, _ = msa.qk_norm_rope(*(t[None] for t in (q, k, v)), cfg, positions=pos)
    # the reference's cos reduces an angle of up to 2^33 by pi in 64 bits: exact to its last bit
    y, slack = norm_rope(q, None, False, 0.0, d, freq, False, pos, 1.25)
    # f / (2 pi): two roundings of 2^-53, so position * f is off by at most 4 * 2^-52 * 2^31 = 2^-19 rad
    slack = 2 * slack  # which was the pair's size times 2^-19 (32 * 2^-24) already
    check_rounded(qo[0].transpose(0, 1), y, slack, "far")


@pytest.mark.gpu
def test_zeros_infinities_and_bad_slots(cuda_lib):
    tok, Hq, Hkv, d, page = 8, 2, 1, 64, 16
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 5)
    q[0, 0] = 0
    q[1, 1, 3] = float("inf")
    q[2, 0, 9] = float("nan")
    cfg = msa.rope_cfg(d, norm=True, eps=0.0)
    kp, vp = (torch.zeros(2, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    slots = torch.arange(tok, dtype=torch.int32, device="cuda")
    slots[3], slots[4] = 32, 1 << 30  # behind the pool
    qo, ko, _ = msa.qk_norm_rope(*(t[None] for t in (q, k, v)), cfg, k_pages=kp, v_pages=vp, slots=slots)
    assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX
    assert cuda_lib.poll_device_status() == 0
    assert torch.equal(kp[0, 0, 5:8], ko[0, 0, 5:8]) and not bool(kp[0, 0, 3:5].any()) and not bool(kp[1].any())
    assert bool(qo[0, 0, 0].isnan().all())     # 0 / 0: a zero row without eps
    assert bool(qo[0, 1, 1].isnan().any()) and bool(qo[0, 0, 2].isnan().all())
    good = torch.ones(Hq, tok, dtype=torch.bool, device="cuda")
    good[0, 0] = good[1, 1] = good[0, 2] = False
    assert bool(qo[0][good].isfinite().all())  # a bad row stays its own


@pytest.mark.gpu
def test_streams_and_capture(cuda_lib):
    tok, Hq, Hkv, d = 19, 4, 2, 128
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 6)
    x = [t[None] for t in (q, k, v)]
    cfg = msa.rope_cfg(d, norm=True, q_weight=w[0], k_weight=w[1])
    want = msa.qk_norm_rope(*x, cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msa.qk_norm_rope(*x, cfg, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        msa.qk_norm_rope(*x, cfg, q=out[0], k=out[1], v=out[2])
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_weights_replaced_in_a_config(cuda_lib):
    """A config follows its weights: another tensor in their place, new storage of the same tensor."""
    q, k, v, w = _inputs(9, 4, 2, 128, 8)
    x = [t[None] for t in (q, k, v)]
    cfg = msa.rope_cfg(128, norm=True, q_weight=w[0].clone(), k_weight=w[1].clone())
    first = (cfg.q_weight, cfg.k_weight.detach())  # keeps the storages
    cfg.q_weight = 2 * w[0]
    cfg.k_weight.data = 4 * w[1]
    got = msa.qk_norm_rope(*x, cfg)
    want = msa.qk_norm_rope(*x, msa.rope_cfg(128, norm=True, q_weight=2 * w[0], k_weight=4 * w[1]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    cfg.q_weight = None
    got = msa.qk_norm_rope(*x, cfg)
    want = msa.qk_norm_rope(*x, msa.rope_cfg(128, norm=True, k_weight=4 * w[1]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    cfg.k_weight.data = torch.ones(64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="k_weight: shape"):
        msa.qk_norm_rope(*x, cfg)
    assert first[0].shape == first[1].shape


def _inverse_two_pi(bits):
    """2^bits / (2 pi), rounded down (Machin's formula in integers)."""
    one = 1 << (bits + 80)

    def atan_inverse(x):
        term, total, k = one // x, one // x, 1
        while term:
            term //= -x * x
            k += 2
            total += term // k
        return total

    pi = 4 * (4 * atan_inverse(5) - atan_inverse(239))  # pi 2^(bits + 80)
    return (one << bits) // (2 * pi)


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [-8, 0, 18])
def test_angles_near_whole_turns_at_far_positions(cuda_lib, size, sign):
    """The angle itself at positions up to 2^31, where it lies within 2^-18 turns of a whole turn, so that the sine that
    comes out is the angle: the reference is position * f / (2 pi) in exact integers."""
    d, tok = 128, 64
    rng = np.random.default_rng(size + 50)
    unit = _inverse_two_pi(64 + 200)
    # unrounded doubles of about 2^size
    freq = [sign * float(x) * 2.0 ** size for x in rng.uniform(0.5, 1.0, d // 2)]
    turn = []  # f / (2 pi) in 2^-64 turns
    for f in freq:
        num, den = f.as_integer_ratio()
        turn.append((num * unit // (den << 200)) % (1 << 64))
    turn = np.array(turn, np.uint64)
    pos = np.zeros(tok, np.int64)
    for t in range(tok):  # token t: a position where pair t comes close to a whole turn
        p = rng.integers(1 << 30, 1 << 31, 1 << 20) * rng.choice([-1, 1], 1 << 20)
        near = np.abs((p.astype(np.uint64) * turn[t]).view(np.int64).astype(np.float64))
        pos[t] = p[np.argmin(np.where(near < 2.0 ** 41, np.inf, near))]
    x = torch.zeros(1, tok, 1, d, dtype=BF, device="cuda")
    x[..., d // 2:] = 1  # (0, 1) -> (-sin, cos)
    cfg = msa.rope_cfg(d, inv_freq=freq)
    q, _, _ = msa.qk_norm_rope(x, x, x, cfg, positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    u = (pos.astype(np.uint64)[:, None] * turn[None]).view(np.int64) / 2.0 ** 63  # half turns in [-1, 1)
    u = torch.from_numpy(u).cuda()
    ref = torch.cat([-torch.sin(math.pi * u), torch.cos(math.pi * u)], 1)
    near = torch.diagonal(u).abs()
    assert bool((near < 2.0 ** -17).all())
    # 32 bits of a turn, cut off (2^-31 half turns; the 64-bit product: 2^31 units of 2^-64 turns, 2^-32 half turns), then rounded to fp32; the
    # sine or cosine of that to 2 steps
    slack = math.pi * (1.5 * 2.0 ** -31 + u.abs() * 2.0 ** -24)
    check_rounded(q[0, 0], ref, torch.cat([slack, slack], 1) + ref.abs() * 2.0 ** -22, "far angles")


def test_outputs_in_one_place_are_refused(lib):
    """Two outputs, or an output and an input, at one address: which value stays would be chance."""
    P = ctypes.c_void_p
    names = ("q_in", "k_in", "v_in", "q", "k", "v", "k_pages", "v_pages")
    sh, c = msa.Shape(1, 4, 4, 8, 128, 0.0), msa.rope_cfg(128).c

    def call(**same):
        a = {k: 0x100000 * (x + 1) for x, k in enumerate(names)}
        a.update({k: a[v] for k, v in same.items()})
        pages = msa.KVPagesC(a["k_pages"], a["v_pages"], 8, 16)
        return lib.msa_qk_norm_rope(ctypes.byref(sh), ctypes.byref(c), P(a["q_in"]), 512, P(a["k_in"]), 512, P(a["v_in"]),
                                    512, None, P(a["q"]), P(a["k"]), P(a["v"]), ctypes.byref(pages), P(0x1000), None)

    outs = names[3:]
    for x, out in enumerate(outs):
        for other in names[:3] + outs[:x]:
            assert call(**{out: other}) == msa.MSA_ERR_INVALID_ARG, (out, other)


@pytest.mark.gpu
@pytest.mark.parametrize("varlen", [False, True])
def test_many_tokens_of_full_heads(cuda_lib, varlen):
    """32 / 8 heads of 128 and enough tokens that a CTA takes eight, the last one fewer: into layer and cache."""
    Hq, Hkv, d, page = 32, 8, 128, 64
    lens = [4099, 1, 0, 6000, 903] if varlen else [10003]
    cu = np.concatenate([[0], np.cumsum(lens)])
    tok = int(cu[-1])
    q, k, v, w = _inputs(tok, Hq, Hkv, d, 12)
    rng = np.random.default_rng(12)
    N = -(-tok // page) + 2
    slots = torch.from_numpy(rng.permutation(N * page)[:tok].astype(np.int32)).cuda()
    kp, vp = (torch.full((N, Hkv, page, d), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    cfg = msa.rope_cfg(d, theta=500000.0, norm=True, q_weight=w[0], k_weight=w[1])
    where = dict(k_pages=kp, v_pages=vp, slots=slots)
    if varlen:
        outs = msa.qk_norm_rope_varlen(q, k, v, cu, cfg, **where)
        outs = [torch.cat([s.transpose(0, 1) for s in msa.unpack_varlen(t, H, cu, d)])
                for t, H in zip(outs, (Hq, Hkv, Hkv))]
    else:
        outs = [t[0].transpose(0, 1) for t in msa.qk_norm_rope(*(t[None] for t in (q, k, v)), cfg, **where)]
    assert cuda_lib.poll_device_status() == 0
    pos = torch.cat([torch.arange(x) for x in lens]).int().cuda()
    c = dict(norm=True, eps=1e-6, rot=d, freq=_freq(d, 500000.0), inter=False)
    _check(outs[0], q, w[0], c, pos, "q")
    _check(outs[1], k, w[1], c, pos, "k")
    assert torch.equal(outs[2], v)
    rows = lambda t: t.transpose(1, 2).reshape(-1, Hkv, d)  # noqa: E731
    assert torch.equal(rows(kp)[slots.long()], outs[1]) and torch.equal(rows(vp)[slots.long()], v)
    other = torch.ones(N * page, dtype=torch.bool, device="cuda")
    other[slots.long()] = False
    assert bool(rows(kp)[other].isnan().all()) and bool(rows(vp)[other].isnan().all())


@pytest.mark.gpu
def test_packed_tokens_on_a_given_stream(cuda_lib):
    lens = [5, 0, 300, 17]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v, w = _inputs(int(cu[-1]), 4, 2, 64, 14)
    cfg = msa.rope_cfg(64, norm=True, q_weight=w[0], k_weight=w[1])
    want = msa.qk_norm_rope_varlen(q, k, v, cu, cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = msa.qk_norm_rope_varlen(q, k, v, cu, cfg, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
