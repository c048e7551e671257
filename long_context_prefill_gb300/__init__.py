"""Python binding of libmsa (MInference-style dynamic sparse prefill attention
on sm_103a).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  There is no fallback:
if ``libmsa.so`` is missing or cannot be loaded, every call raises.

Function names mirror the C ABI in ``include/msa.h`` without the ``msa_``
prefix.  Tensors: Q/O [B,Hq,n,d] bf16, K/V [B,Hkv,n,d] bf16 (contiguous, on
the current CUDA device); ``heads`` is a list of query-head indices.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmsa.so")

MSA_OK, MSA_ERR_INVALID_ARG, MSA_ERR_UNSUPPORTED, MSA_ERR_WORKSPACE_TOO_SMALL = 0, 1, 2, 3
MSA_ERR_CUDA, MSA_ERR_DEVICE_TIMEOUT, MSA_ERR_INDEX = 4, 5, 6
ASHAPE, VS, BLOCK = 0, 1, 2
PATTERNS = {"ashape": ASHAPE, "vs": VS, "block": BLOCK}

EXPORTS = ("msa_status_string", "msa_vs_index_workspace", "msa_block_index_workspace", "msa_layer_workspace",
           "msa_build_vs_index", "msa_build_block_index", "msa_attn_ashape", "msa_attn_vs", "msa_attn_block",
           "msa_prefill_layer", "msa_layer_index", "msa_layer_attend", "msa_kernel_launches", "msa_layer_indices",
           "msa_vs_expand", "msa_poll_device_status", "msa_build_block_index_static",
           "msa_check_wait_timeout", "msa_attn_dense", "msa_layer_varlen_workspace", "msa_prefill_layer_varlen",
           "msa_layer_attend_rows", "msa_merge_attention", "msa_captured_mass", "msa_layer_varlen_indices",
           "msa_layer_attend_stats", "msa_build_page_tables", "msa_qk_norm_rope", "msa_qk_norm_rope_varlen",
           "msa_attn_tree_workspace", "msa_attn_tree", "msa_attn_tree_window", "msa_qk_norm_rope_kv4",
           "msa_qk_norm_rope_varlen_kv4", "msa_kv4_gather", "msa_attn_tree_kv4_workspace", "msa_attn_tree_kv4")


class MsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("n", ctypes.c_int32),
                ("d_h", ctypes.c_int32), ("scale", ctypes.c_float)]


class HeadCfg(ctypes.Structure):
    _fields_ = [("pattern", ctypes.c_int32), ("sink", ctypes.c_int32), ("window", ctypes.c_int32),
                ("last_q", ctypes.c_int32), ("n_vertical", ctypes.c_int32), ("n_slash", ctypes.c_int32),
                ("block", ctypes.c_int32), ("topk", ctypes.c_int32), ("proxy", ctypes.c_int32)]


class VSIndexC(ctypes.Structure):
    _fields_ = [("vertical", ctypes.c_void_p), ("vertical_cnt", ctypes.c_void_p), ("slash", ctypes.c_void_p),
                ("slash_cnt", ctypes.c_void_p), ("vertical_bits", ctypes.c_void_p), ("slash_bits", ctypes.c_void_p),
                ("slash_cover", ctypes.c_void_p), ("v_cap", ctypes.c_int32), ("s_cap", ctypes.c_int32)]


class KVPagesC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class PagePoolC(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("state", ctypes.c_void_p)]


class TreeWindowC(ctypes.Structure):
    _fields_ = [("sink", ctypes.c_int32), ("window", ctypes.c_int32), ("depth", ctypes.c_void_p)]


class KV4PagesC(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class RopeCfgC(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("theta", ctypes.c_double), ("inv_freq", ctypes.POINTER(ctypes.c_double)),
                ("rot_scale", ctypes.c_float)]


_lib = None
_lock = threading.Lock()


def load(path: str = LIB_PATH):
    """Load libmsa.so (raises if it is missing: there is no CPU fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libmsa.so not built ({path}); run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
            st = ctypes.c_int
            lib.msa_status_string.restype = ctypes.c_char_p
            lib.msa_status_string.argtypes = [st]
            lib.msa_vs_index_workspace.restype = sz
            lib.msa_vs_index_workspace.argtypes = [P, P, i32]
            lib.msa_block_index_workspace.restype = sz
            lib.msa_block_index_workspace.argtypes = [P, i32, i32]
            lib.msa_layer_workspace.restype = sz
            lib.msa_layer_workspace.argtypes = [P, P]
            lib.msa_build_vs_index.restype = st
            lib.msa_build_vs_index.argtypes = [P, P, P, P, i32, P, P, P, sz, P]
            lib.msa_build_block_index.restype = st
            lib.msa_build_block_index.argtypes = [P, P, P, P, i32, i32, i32, P, P, P, sz, P]
            lib.msa_attn_ashape.restype = st
            lib.msa_attn_ashape.argtypes = [P, P, P, P, P, i32, i32, i32, P, P, P, P]
            lib.msa_attn_vs.restype = st
            lib.msa_attn_vs.argtypes = [P, P, P, P, P, i32, i32, P, P, P, P, P]
            lib.msa_attn_block.restype = st
            lib.msa_attn_block.argtypes = [P, P, P, P, P, i32, i32, i32, P, P, P, P, P, P]
            lib.msa_prefill_layer.restype = st
            lib.msa_prefill_layer.argtypes = [P, P, P, P, P, P, P, P, P, sz, P]
            lib.msa_layer_index.restype = st
            lib.msa_layer_index.argtypes = [P, P, P, P, P, sz, P]
            lib.msa_layer_attend.restype = st
            lib.msa_layer_attend.argtypes = [P, P, P, P, P, P, P, P, P, sz, P]
            lib.msa_kernel_launches.restype = ctypes.c_uint64
            lib.msa_kernel_launches.argtypes = []
            lib.msa_layer_indices.restype = st
            lib.msa_layer_indices.argtypes = [P, P, P, P, P, P]
            lib.msa_vs_expand.restype = st
            lib.msa_vs_expand.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P, P, P]
            lib.msa_poll_device_status.restype = st
            lib.msa_poll_device_status.argtypes = [P]
            lib.msa_attn_dense.restype = st
            lib.msa_attn_dense.argtypes = [P, P, P, P, P, i32, P, P, P, P]
            lib.msa_check_wait_timeout.restype = st
            lib.msa_check_wait_timeout.argtypes = [i32, P]
            lib.msa_layer_varlen_workspace.restype = sz
            lib.msa_layer_varlen_workspace.argtypes = [P, P, P, i32]
            lib.msa_prefill_layer_varlen.restype = st
            lib.msa_prefill_layer_varlen.argtypes = [P, P, i32, P, P, P, P, P, P, P, P, sz, P]
            lib.msa_layer_attend_stats.restype = st
            lib.msa_layer_attend_stats.argtypes = [P, P, P, P, P, P, P, P, P, P, sz, P]
            lib.msa_layer_varlen_indices.restype = st
            lib.msa_layer_varlen_indices.argtypes = [P, P, P, i32, P, i32, P, P, P]
            lib.msa_layer_attend_rows.restype = st
            lib.msa_layer_attend_rows.argtypes = [P, P, P, P, P, P, P, P, P, sz, i32, i32, P]
            lib.msa_merge_attention.restype = st
            lib.msa_merge_attention.argtypes = [ctypes.c_int64, i32, P, P, P, P, P, P, P]
            lib.msa_captured_mass.restype = st
            lib.msa_captured_mass.argtypes = [ctypes.c_int64, ctypes.c_int64, P, P, P, P]
            lib.msa_build_block_index_static.restype = st
            lib.msa_build_block_index_static.argtypes = [P, P, P, P, i32, i32, i32, P, P, P]
            i64 = ctypes.c_int64
            lib.msa_build_page_tables.restype = st
            lib.msa_build_page_tables.argtypes = [P, P, P, i32, i32, P, P, P, P]
            lib.msa_qk_norm_rope.restype = st
            lib.msa_qk_norm_rope.argtypes = [P, P, P, i64, P, i64, P, i64, P, P, P, P, P, P, P]
            lib.msa_qk_norm_rope_varlen.restype = st
            lib.msa_qk_norm_rope_varlen.argtypes = [P, P, i32, P, P, i64, P, i64, P, i64, P, P, P, P, P, P, P]
            lib.msa_attn_tree_workspace.restype = sz
            lib.msa_attn_tree_workspace.argtypes = [P]
            lib.msa_attn_tree.restype = st
            lib.msa_attn_tree.argtypes = [P, P, P, P, i32, P, P, P, i64, P, P, P, sz, P]
            lib.msa_attn_tree_window.restype = st
            lib.msa_attn_tree_window.argtypes = [P, P, P, P, i32, P, P, P, i64, P, P, P, P, sz, P]
            lib.msa_qk_norm_rope_kv4.restype = st
            lib.msa_qk_norm_rope_kv4.argtypes = lib.msa_qk_norm_rope.argtypes
            lib.msa_qk_norm_rope_varlen_kv4.restype = st
            lib.msa_qk_norm_rope_varlen_kv4.argtypes = lib.msa_qk_norm_rope_varlen.argtypes
            lib.msa_kv4_gather.restype = st
            lib.msa_kv4_gather.argtypes = [P, P, P, i32, P, P, P, P]
            lib.msa_attn_tree_kv4_workspace.restype = sz
            lib.msa_attn_tree_kv4_workspace.argtypes = [P]
            lib.msa_attn_tree_kv4.restype = st
            lib.msa_attn_tree_kv4.argtypes = [P, P, P, P, i32, P, P, P, i64, P, P, P, P, sz, P]
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().msa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != MSA_OK:
        raise MsaError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _heads(heads):
    arr = (ctypes.c_int32 * len(heads))(*[int(h) for h in heads])
    return arr, len(heads)


def make_shape(q: torch.Tensor, k: torch.Tensor, scale: float | None = None) -> Shape:
    B, Hq, n, d = q.shape
    return Shape(B, Hq, k.shape[1], n, d, float(scale) if scale else 0.0)


def head_cfg(entry: dict) -> HeadCfg:
    """A config-table entry from a dict: pattern 'ashape' | 'vs' | 'block' plus its budgets."""
    pat = entry["pattern"]
    pat = PATTERNS[pat] if isinstance(pat, str) else int(pat)
    return HeadCfg(pat, int(entry.get("sink", 0)), int(entry.get("window", 1)), int(entry.get("last_q", 64)),
                   int(entry.get("n_vertical", 0)), int(entry.get("n_slash", 0)), int(entry.get("block", 64)),
                   int(entry.get("topk", 1)), int(entry.get("proxy", 0)))


def table_array(table):
    arr = (HeadCfg * len(table))()
    for h, e in enumerate(table):
        arr[h] = head_cfg(e)
    return arr


def _out_like(q, o):
    return torch.empty_like(q) if o is None else o


def _want(t, what, dtype, shape=None, min_numel=None, device=None):
    """Raise ValueError unless t (None passes) is a contiguous tensor of this
    dtype and shape (on `device` if given): the library sees only a pointer,
    so a smaller or strided buffer would be read or written out of bounds."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: a torch.Tensor is required")
    if t.dtype != dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{what}: {t.numel()} elements, at least {min_numel} needed")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")


def _cuda(**tensors):
    """Raise ValueError for the first given tensor (None passes) not on a CUDA device."""
    for what, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{what}: must be on a CUDA device")


def _check_attn(q, k, v=None, o=None, lse=None, edges=None, dims=None):
    """Q/O [B,Hq,n,d], K/V [B,Hkv,n,d] bf16, LSE [B,Hq,n] fp32, edges >= B*Hq int64.
    dims: (B, Hq, Hkv, n, d) the tensors must have (a layer's shape), else taken from q and k."""
    for t, what in ((q, "q"), (k, "k")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{what}: a 4-d tensor [B, H, n, d] is required")
    if dims:
        B, Hq, Hkv, n, d = dims
    else:
        B, Hq, n, d = q.shape
        Hkv = k.shape[1]
    dev = q.device
    _want(q, "q", torch.bfloat16, (B, Hq, n, d), device=dev)
    _want(k, "k", torch.bfloat16, (B, Hkv, n, d), device=dev)
    _want(v, "v", torch.bfloat16, (B, Hkv, n, d), device=dev)
    _want(o, "o", torch.bfloat16, (B, Hq, n, d), device=dev)
    _want(lse, "lse", torch.float32, (B, Hq, n), device=dev)
    _want(edges, "edges", torch.int64, min_numel=B * Hq, device=dev)
    _cuda(q=q, k=k, v=v, o=o, lse=lse, edges=edges)


# ----------------------------------------------------------------- attention
def attn_ashape(q, k, v, heads, sink, window, o=None, lse=None, edges=None, scale=None, stream=None):
    """A-shape heads (sink g, window w); returns o."""
    _check_attn(q, k, v, o, lse, edges)
    lib = load()
    o = _out_like(q, o)
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    _check(lib.msa_attn_ashape(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), hp, nh, int(sink), int(window), _ptr(o),
                               _ptr(lse), _ptr(edges), _stream(stream)), "msa_attn_ashape")
    return o


def attn_dense(q, k, v, heads, o=None, lse=None, edges=None, scale=None, stream=None):
    """Dense causal attention of the listed heads on the same engine; returns o."""
    _check_attn(q, k, v, o, lse, edges)
    lib = load()
    o = _out_like(q, o)
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    _check(lib.msa_attn_dense(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), hp, nh, _ptr(o), _ptr(lse), _ptr(edges),
                              _stream(stream)), "msa_attn_dense")
    return o


class VSIndex:
    """Device buffers of a Vertical-Slash index (see msa_vs_index in msa.h)."""

    def __init__(self, slots: int, n: int, n_vertical: int, n_slash: int, device):
        self.slots, self.n = int(slots), int(n)
        self.v_cap = max(min(int(n_vertical), n), 0)
        self.s_cap = max(min(int(n_slash), n), 0)
        words = (n + 31) // 32
        self.vertical = torch.empty(slots, max(self.v_cap, 1), dtype=torch.int32, device=device)
        self.vertical_cnt = torch.empty(slots, dtype=torch.int32, device=device)
        self.slash = torch.empty(slots, max(self.s_cap, 1), dtype=torch.int32, device=device)
        self.slash_cnt = torch.empty(slots, dtype=torch.int32, device=device)
        self.vertical_bits = torch.zeros(slots, words, dtype=torch.int32, device=device)
        self.slash_bits = torch.zeros(slots, words, dtype=torch.int32, device=device)
        self.slash_cover = torch.zeros(slots, (n + 63 + 31) // 32, dtype=torch.int32, device=device)

    def check(self, slots: int, n: int, device=None):
        """Raise ValueError unless the buffers hold `slots` slots of an n-token index (on `device`)."""
        if self.n != n or self.slots < slots:
            raise ValueError(f"VSIndex: {self.slots} slots for n = {self.n}, need {slots} for n = {n}")
        if device is not None and self.vertical_bits.device != device:
            raise ValueError(f"VSIndex: on {self.vertical_bits.device}, expected {device}")

    def c(self) -> VSIndexC:
        return VSIndexC(self.vertical.data_ptr(), self.vertical_cnt.data_ptr(), self.slash.data_ptr(),
                        self.slash_cnt.data_ptr(), self.vertical_bits.data_ptr(), self.slash_bits.data_ptr(),
                        self.slash_cover.data_ptr(), self.v_cap, self.s_cap)

    @staticmethod
    def from_c(c: VSIndexC, slots: int, n: int, ws: torch.Tensor):
        """View of an index that lives in the layer workspace `ws` (the views keep it alive)."""
        ix = VSIndex.__new__(VSIndex)
        ix.slots, ix.n = int(slots), int(n)
        ix.v_cap, ix.s_cap = c.v_cap, c.s_cap
        words = (n + 31) // 32
        ix.vertical = _view_i32(ws, c.vertical, slots * max(c.v_cap, 1)).view(slots, max(c.v_cap, 1))
        ix.vertical_cnt = _view_i32(ws, c.vertical_cnt, slots)
        ix.slash = _view_i32(ws, c.slash, slots * max(c.s_cap, 1)).view(slots, max(c.s_cap, 1))
        ix.slash_cnt = _view_i32(ws, c.slash_cnt, slots)
        ix.vertical_bits = _view_i32(ws, c.vertical_bits, slots * words).view(slots, words)
        ix.slash_bits = _view_i32(ws, c.slash_bits, slots * words).view(slots, words)
        cw = (n + 63 + 31) // 32
        ix.slash_cover = _view_i32(ws, c.slash_cover, slots * cw).view(slots, cw)
        return ix


def _view_i32(base: torch.Tensor, ptr: int, count: int) -> torch.Tensor:
    """A torch int32 view of `count` elements at device address `ptr` inside the uint8 workspace `base`."""
    off = ptr - base.data_ptr()
    assert off % 4 == 0 and 0 <= off and off + 4 * count <= base.numel()
    return base[off:off + 4 * count].view(torch.int32)


def attn_vs(q, k, v, heads, index: VSIndex, o=None, lse=None, edges=None, scale=None, stream=None):
    _check_attn(q, k, v, o, lse, edges)
    index.check(q.shape[0] * len(heads), q.shape[2], q.device)
    lib = load()
    o = _out_like(q, o)
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    ic = index.c()
    _check(lib.msa_attn_vs(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), hp, nh, 64, ctypes.byref(ic), _ptr(o),
                           _ptr(lse), _ptr(edges), _stream(stream)), "msa_attn_vs")
    return o


def attn_block(q, k, v, heads, topk, block_idx, block_cnt, o=None, lse=None, edges=None, scale=None, stream=None):
    _check_attn(q, k, v, o, lse, edges)
    B, nb = q.shape[0], (q.shape[2] + 63) // 64
    _want(block_idx, "block_idx", torch.int32, (B, len(heads), nb, int(topk)), device=q.device)
    _want(block_cnt, "block_cnt", torch.int32, (B, len(heads), nb), device=q.device)
    lib = load()
    o = _out_like(q, o)
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    _check(lib.msa_attn_block(ctypes.byref(sh), _ptr(q), _ptr(k), _ptr(v), hp, nh, 64, int(topk), _ptr(block_idx),
                              _ptr(block_cnt), _ptr(o), _ptr(lse), _ptr(edges), _stream(stream)), "msa_attn_block")
    return o


# ----------------------------------------------------------------- indices
def build_vs_index(q, k, heads, last_q, n_vertical, n_slash, index: VSIndex | None = None, scale=None, stream=None,
                   proxy: int = 0):
    _check_attn(q, k)
    lib = load()
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    cfg = HeadCfg(VS, 0, 1, int(last_q), int(n_vertical), int(n_slash), 64, 1, int(proxy))
    if index is None:
        index = VSIndex(q.shape[0] * nh, q.shape[2], n_vertical, n_slash, q.device)
    index.check(q.shape[0] * nh, q.shape[2], q.device)
    if index.v_cap < min(int(n_vertical), q.shape[2]) or index.s_cap < min(int(n_slash), q.shape[2]):
        raise ValueError("VSIndex: list capacity below the requested budgets")
    ws_bytes = lib.msa_vs_index_workspace(ctypes.byref(sh), ctypes.byref(cfg), nh)
    ws = torch.empty(max(int(ws_bytes), 1), dtype=torch.uint8, device=q.device)
    ic = index.c()
    _check(lib.msa_build_vs_index(ctypes.byref(sh), _ptr(q), _ptr(k), hp, nh, ctypes.byref(cfg), ctypes.byref(ic),
                                  _ptr(ws), int(ws_bytes), _stream(stream)), "msa_build_vs_index")
    index._ws = ws  # keep the scratch alive until the stream has used it
    return index


def build_block_index(q, k, heads, topk, block_idx=None, block_cnt=None, scale=None, stream=None):
    _check_attn(q, k)
    lib = load()
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    B, n = q.shape[0], q.shape[2]
    nb = (n + 63) // 64
    if block_idx is None:
        block_idx = torch.empty(B, nh, nb, int(topk), dtype=torch.int32, device=q.device)
    if block_cnt is None:
        block_cnt = torch.empty(B, nh, nb, dtype=torch.int32, device=q.device)
    _want(block_idx, "block_idx", torch.int32, (B, nh, nb, int(topk)), device=q.device)
    _want(block_cnt, "block_cnt", torch.int32, (B, nh, nb), device=q.device)
    ws_bytes = lib.msa_block_index_workspace(ctypes.byref(sh), 64, nh)
    ws = torch.empty(max(int(ws_bytes), 1), dtype=torch.uint8, device=q.device)
    _check(lib.msa_build_block_index(ctypes.byref(sh), _ptr(q), _ptr(k), hp, nh, 64, int(topk), _ptr(block_idx),
                                     _ptr(block_cnt), _ptr(ws), int(ws_bytes), _stream(stream)),
           "msa_build_block_index")
    block_idx._ws = ws
    return block_idx, block_cnt


def build_block_index_static(q, k, heads, topk, block_idx=None, block_cnt=None, scale=None, stream=None):
    """msa_build_block_index_static: the Block-Sparse index built in the
    library's own scratch (no workspace); outputs as build_block_index."""
    _check_attn(q, k)
    lib = load()
    sh = make_shape(q, k, scale)
    hp, nh = _heads(heads)
    B, n = q.shape[0], q.shape[2]
    nb = (n + 63) // 64
    if block_idx is None:
        block_idx = torch.empty(B, nh, nb, int(topk), dtype=torch.int32, device=q.device)
    if block_cnt is None:
        block_cnt = torch.empty(B, nh, nb, dtype=torch.int32, device=q.device)
    _want(block_idx, "block_idx", torch.int32, (B, nh, nb, int(topk)), device=q.device)
    _want(block_cnt, "block_cnt", torch.int32, (B, nh, nb), device=q.device)
    _check(lib.msa_build_block_index_static(ctypes.byref(sh), _ptr(q), _ptr(k), hp, nh, 64, int(topk),
                                            _ptr(block_idx), _ptr(block_cnt), _stream(stream)),
           "msa_build_block_index_static")
    return block_idx, block_cnt


def vs_expand(q_shape, index: VSIndex, slot, u_begin, u_count, range_cap, col_cap, stream=None):
    """Explicit per-block ranges and columns of one slot (device tensors)."""
    lib = load()
    B, Hq, n, d = q_shape
    sh = Shape(B, Hq, 1, n, d, 0.0)
    dev = index.vertical.device
    rc = torch.empty(u_count, dtype=torch.int32, device=dev)
    rg = torch.empty(u_count, max(range_cap, 1), 2, dtype=torch.int32, device=dev)
    cc = torch.empty(u_count, dtype=torch.int32, device=dev)
    cl = torch.empty(u_count, max(col_cap, 1), dtype=torch.int32, device=dev)
    ic = index.c()
    _check(lib.msa_vs_expand(ctypes.byref(sh), ctypes.byref(ic), int(slot), int(u_begin), int(u_count), int(range_cap),
                             int(col_cap), _ptr(rc), _ptr(rg), _ptr(cc), _ptr(cl), _stream(stream)), "msa_vs_expand")
    return rc, rg, cc, cl


# ----------------------------------------------------------------- layer
class Layer:
    """One layer's config table plus its workspace; call() runs msa_prefill_layer."""

    def __init__(self, table, B, Hq, Hkv, n, d, device, scale=None):
        self.table = list(table)
        assert len(self.table) == Hq
        self.tarr = table_array(self.table)
        self.shape = Shape(B, Hq, Hkv, n, d, float(scale) if scale else 0.0)
        lib = load()
        self.ws_bytes = int(lib.msa_layer_workspace(ctypes.byref(self.shape), self.tarr))
        if self.ws_bytes == 0:
            raise MsaError(MSA_ERR_INVALID_ARG, "msa_layer_workspace")
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def _dims(self):
        s = self.shape
        return (s.B, s.Hq, s.Hkv, s.n, s.d_h)

    def __call__(self, q, k, v, o=None, lse=None, edges=None, stream=None):
        _check_attn(q, k, v, o, lse, edges, self._dims())
        lib = load()
        o = _out_like(q, o)
        _check(lib.msa_prefill_layer(ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), self.tarr, _ptr(o), _ptr(lse),
                                     _ptr(edges), _ptr(self.ws), self.ws_bytes, _stream(stream)), "msa_prefill_layer")
        return o

    def index(self, q, k, stream=None):
        """First half of the layer (T_index): build every online index into the workspace."""
        _check_attn(q, k, dims=self._dims())
        _check(load().msa_layer_index(ctypes.byref(self.shape), _ptr(q), _ptr(k), self.tarr, _ptr(self.ws),
                                      self.ws_bytes, _stream(stream)), "msa_layer_index")

    def attend(self, q, k, v, o, lse=None, edges=None, stream=None):
        """Second half (T_sparse): the single attention launch over the indices in the workspace."""
        _check_attn(q, k, v, o, lse, edges, self._dims())
        _check(load().msa_layer_attend(ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), self.tarr, _ptr(o),
                                       _ptr(lse), _ptr(edges), _ptr(self.ws), self.ws_bytes, _stream(stream)),
               "msa_layer_attend")
        return o

    def attend_stats(self, q, k, v, o, lse=None, edges=None, tiles=None, stream=None):
        """attend() with work counters: edges (E_h) and tiles (64-row x 128-key tiles per query head),
        both [B*Hq] int64 device tensors that are ADDED to."""
        _check_attn(q, k, v, o, lse, edges, self._dims())
        if tiles is not None:
            _want(tiles, "tiles", torch.int64, (self.shape.B * self.shape.Hq,), device=q.device)
        _check(load().msa_layer_attend_stats(ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), self.tarr, _ptr(o),
                                             _ptr(lse), _ptr(edges), _ptr(tiles), _ptr(self.ws), self.ws_bytes,
                                             _stream(stream)), "msa_layer_attend_stats")
        return o

    def attend_rows(self, q, k, v, o, row_begin, row_end, lse=None, edges=None, stream=None):
        """Chunked T_sparse: the attention of query rows [row_begin, row_end) only (indices from index())."""
        _check_attn(q, k, v, o, lse, edges, self._dims())
        _check(load().msa_layer_attend_rows(ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), self.tarr, _ptr(o),
                                            _ptr(lse), _ptr(edges), _ptr(self.ws), self.ws_bytes, int(row_begin),
                                            int(row_end), _stream(stream)), "msa_layer_attend_rows")
        return o

    def indices(self):
        """(VSIndex view, block_idx, block_cnt) left in the workspace by the last call."""
        lib = load()
        vc = VSIndexC()
        bi = ctypes.c_void_p()
        bc = ctypes.c_void_p()
        _check(lib.msa_layer_indices(ctypes.byref(self.shape), self.tarr, _ptr(self.ws), ctypes.byref(vc),
                                     ctypes.byref(bi), ctypes.byref(bc)), "msa_layer_indices")
        B, n = self.shape.B, self.shape.n
        nvs = sum(1 for e in self.table if head_cfg(e).pattern == VS)
        nbs = [e for e in self.table if head_cfg(e).pattern == BLOCK]
        vs = VSIndex.from_c(vc, B * nvs, n, self.ws) if nvs else None
        blk = cnt = None
        if nbs:
            nb = (n + 63) // 64
            topk = head_cfg(nbs[0]).topk
            blk = _view_i32(self.ws, bi.value, B * len(nbs) * nb * topk).view(B, len(nbs), nb, topk)
            cnt = _view_i32(self.ws, bc.value, B * len(nbs) * nb).view(B, len(nbs), nb)
        return vs, blk, cnt


# ----------------------------------------------------------------- varlen
def pack_varlen(seqs) -> torch.Tensor:
    """Pack per-sequence [H, n_s, d] tensors back to back (the varlen layout)."""
    return torch.cat([x.contiguous().reshape(-1) for x in seqs])


def unpack_varlen(flat: torch.Tensor, H: int, cu_seqlens, d: int):
    """Split a packed varlen buffer into per-sequence [H, n_s, d] views."""
    out = []
    for s in range(len(cu_seqlens) - 1):
        a, b = int(cu_seqlens[s]), int(cu_seqlens[s + 1])
        out.append(flat[H * a * d:H * b * d].view(H, b - a, d))
    return out


class VarlenLayer:
    """A varlen batch (cumulative lengths cu_seqlens) of one layer's table plus
    its workspace; call() runs msa_prefill_layer_varlen on packed buffers (see
    pack_varlen) and indices(seq) views what it left for one sequence."""

    def __init__(self, table, cu_seqlens, Hq, Hkv, d, device, scale=None):
        self.table = list(table)
        if len(self.table) != int(Hq):
            raise ValueError(f"table: {len(self.table)} entries, expected Hq = {int(Hq)}")
        self.cu_list = [int(x) for x in cu_seqlens]
        self.n_seqs = len(self.cu_list) - 1
        self.cu = (ctypes.c_int32 * len(self.cu_list))(*self.cu_list)
        lens = [self.cu_list[s + 1] - self.cu_list[s] for s in range(self.n_seqs)]
        self.Hq, self.Hkv, self.d = int(Hq), int(Hkv), int(d)
        self.shape = Shape(1, self.Hq, self.Hkv, max([1] + lens), self.d, float(scale) if scale else 0.0)
        self.tarr = table_array(self.table)
        lib = load()
        self.ws_bytes = int(lib.msa_layer_varlen_workspace(ctypes.byref(self.shape), self.tarr, self.cu, self.n_seqs))
        if self.ws_bytes == 0:
            raise MsaError(MSA_ERR_INVALID_ARG, "msa_layer_varlen_workspace")
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)

    def __call__(self, q, k, v, o=None, lse=None, edges=None, stream=None):
        _check_varlen(q, k, v, o, lse, edges, self.cu_list, self.Hq, self.Hkv, self.d)
        o = torch.empty_like(q) if o is None else o
        _check(load().msa_prefill_layer_varlen(ctypes.byref(self.shape), self.cu, self.n_seqs, _ptr(q), _ptr(k),
                                               _ptr(v), self.tarr, _ptr(o), _ptr(lse), _ptr(edges), _ptr(self.ws),
                                               self.ws_bytes, _stream(stream)), "msa_prefill_layer_varlen")
        return o

    def indices(self, seq: int):
        """(VSIndex view, block_idx [n_bs, N_b, topk], block_cnt [n_bs, N_b]) of sequence seq."""
        lib = load()
        vc = VSIndexC()
        bi = ctypes.c_void_p()
        bc = ctypes.c_void_p()
        _check(lib.msa_layer_varlen_indices(ctypes.byref(self.shape), self.tarr, self.cu, self.n_seqs,
                                            _ptr(self.ws), int(seq), ctypes.byref(vc), ctypes.byref(bi),
                                            ctypes.byref(bc)), "msa_layer_varlen_indices")
        n = self.cu_list[seq + 1] - self.cu_list[seq]
        nvs = sum(1 for e in self.table if head_cfg(e).pattern == VS)
        nbs = [e for e in self.table if head_cfg(e).pattern == BLOCK]
        vs = VSIndex.from_c(vc, nvs, n, self.ws) if nvs else None
        blk = cnt = None
        if nbs:
            nb = (n + 63) // 64
            topk = head_cfg(nbs[0]).topk
            blk = _view_i32(self.ws, bi.value, len(nbs) * nb * topk).view(len(nbs), nb, topk)
            cnt = _view_i32(self.ws, bc.value, len(nbs) * nb).view(len(nbs), nb)
        return vs, blk, cnt


def _check_varlen(q, k, v, o, lse, edges, cu_seqlens, Hq, Hkv, d):
    total = int(cu_seqlens[-1]) if len(cu_seqlens) else 0
    _want(q, "q", torch.bfloat16, min_numel=Hq * total * d)
    _want(k, "k", torch.bfloat16, min_numel=Hkv * total * d, device=q.device)
    _want(v, "v", torch.bfloat16, min_numel=Hkv * total * d, device=q.device)
    _want(o, "o", torch.bfloat16, tuple(q.shape), device=q.device)
    _want(lse, "lse", torch.float32, min_numel=Hq * total, device=q.device)
    _want(edges, "edges", torch.int64, min_numel=(len(cu_seqlens) - 1) * Hq, device=q.device)
    _cuda(q=q)


def prefill_layer_varlen(q, k, v, table, cu_seqlens, Hq, Hkv, d, o=None, lse=None, edges=None, scale=None,
                         stream=None):
    """msa_prefill_layer_varlen on packed buffers (see pack_varlen); returns o."""
    _check_varlen(q, k, v, o, lse, edges, cu_seqlens, Hq, Hkv, d)
    layer = VarlenLayer(table, cu_seqlens, Hq, Hkv, d, q.device, scale=scale)
    return layer(q, k, v, o=o, lse=lse, edges=edges, stream=stream)


def merge_attention(o_a, lse_a, o_b, lse_b, o=None, lse=None, stream=None):
    """Combine two attention results over disjoint key sets (msa_merge_attention); returns (o, lse)."""
    if not isinstance(o_a, torch.Tensor) or o_a.dim() < 1:
        raise ValueError("o_a: a tensor [..., d] is required")
    d = o_a.shape[-1]
    rows = o_a.numel() // d
    for t, what in ((o_a, "o_a"), (o_b, "o_b"), (o, "o")):
        _want(t, what, torch.bfloat16, tuple(o_a.shape), device=o_a.device)
    for t, what in ((lse_a, "lse_a"), (lse_b, "lse_b"), (lse, "lse")):
        _want(t, what, torch.float32, tuple(o_a.shape[:-1]), device=o_a.device)
    _cuda(o_a=o_a)
    o = torch.empty_like(o_a) if o is None else o
    lse = torch.empty_like(lse_a) if lse is None else lse
    _check(load().msa_merge_attention(rows, d, _ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(o), _ptr(lse),
                                      _stream(stream)), "msa_merge_attention")
    return o, lse


def captured_mass(lse_sparse, lse_dense, stream=None):
    """Per-head share of the dense softmax mass kept by the sparse sets (msa_captured_mass).
    lse_*: [..., n] with the leading dims flattened into heads; returns [heads] fp32."""
    if not isinstance(lse_sparse, torch.Tensor) or lse_sparse.dim() < 1:
        raise ValueError("lse_sparse: a tensor [..., n] is required")
    _want(lse_sparse, "lse_sparse", torch.float32, device=lse_sparse.device)
    _want(lse_dense, "lse_dense", torch.float32, tuple(lse_sparse.shape), device=lse_sparse.device)
    _cuda(lse_sparse=lse_sparse)
    n = lse_sparse.shape[-1]
    heads = lse_sparse.numel() // n
    mass = torch.empty(heads, dtype=torch.float32, device=lse_sparse.device)
    _check(load().msa_captured_mass(heads, n, _ptr(lse_sparse), _ptr(lse_dense), _ptr(mass), _stream(stream)),
           "msa_captured_mass")
    return mass


# ----------------------------------------------------------------- paged KV cache
# These run once per decode step: their checks take a fast path (one test per
# tensor) and call _want only to name what is wrong.
def _elsewhere(device, stream) -> bool:
    """The call is not for the current stream of the current device."""
    return stream is not None or device.index != torch._C._cuda_getDevice()


class _on:
    """`device` current, on `stream` (None: the device's current one); what is allocated inside belongs to that stream."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"stream: on {stream.device}, expected {device}")
        self.device, self.stream = torch.cuda.device(device), torch.cuda.stream(stream)

    def __enter__(self):
        self.device.__enter__()
        self.stream.__enter__()

    def __exit__(self, *exc):
        self.stream.__exit__(*exc)
        self.device.__exit__(*exc)


def _same(t, what, dtype, shape, device):
    """_want for a tensor that is mostly right."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous()):
        if t is None:
            raise ValueError(f"{what}: a torch.Tensor is required")
        _want(t, what, dtype, shape, device=device)


def _at(t):
    return None if t is None else t.data_ptr()


def _pages(k_pages, v_pages, Hkv, d, device):
    """Check the two page tensors [num_pages, Hkv, page_size, d] (Hkv None: any); returns their C view."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages: a 4-d tensor [num_pages, Hkv, page_size, d] is required")
    N, H, P, _ = k_pages.shape
    want = (N, H if Hkv is None else Hkv, P, d)
    _same(k_pages, "k_pages", torch.bfloat16, want, device)
    _same(v_pages, "v_pages", torch.bfloat16, want, device)
    return KVPagesC(k_pages.data_ptr(), v_pages.data_ptr(), N, P)


class PagePool:
    """The requests that share a pool of cache pages (msa_page_pool): page_table
    [n_seqs, max_pages], seq_len [n_seqs], free_pages [num_pages] (a stack) and
    state [4], int32 tensors that build_page_tables updates in place.  They may
    be replaced: each call checks and uses the ones that are there."""

    def __init__(self, page_table, seq_len, free_pages, state, page_size: int):
        self.__dict__.update(page_table=page_table, seq_len=seq_len, free_pages=free_pages, state=state,
                             page_size=int(page_size), _held=None)
        self.view()

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__["_held"] = None

    def view(self):
        """The tensors' C view."""
        return self._hold()[0]

    def _hold(self):
        """(C view, n_seqs, device, addresses, storages), checked anew when a tensor was replaced or its memory was.
        The storages are held so that an address which was checked is not another tensor's."""
        held = self._held
        if held is not None and held[3] == (self.page_table.data_ptr(), self.seq_len.data_ptr(),
                                            self.free_pages.data_ptr(), self.state.data_ptr()):
            return held
        table, lens, stack, state = self.page_table, self.seq_len, self.free_pages, self.state
        if not isinstance(table, torch.Tensor) or table.dim() != 2:
            raise ValueError("page_table: a 2-d tensor [n_seqs, max_pages] is required")
        if not isinstance(stack, torch.Tensor) or stack.dim() != 1:
            raise ValueError("free_pages: a 1-d tensor [num_pages] is required")
        S, width = table.shape
        N, dev = stack.shape[0], table.device
        _same(table, "page_table", torch.int32, (S, width), dev)
        _same(lens, "seq_len", torch.int32, (S,), dev)
        _same(stack, "free_pages", torch.int32, (N,), dev)
        _same(state, "state", torch.int32, (4,), dev)
        if not 0 < self.page_size < 1 << 31:
            raise ValueError(f"page_size: {self.page_size}")
        at = (table.data_ptr(), lens.data_ptr(), stack.data_ptr(), state.data_ptr())
        held = (PagePoolC(S, N, self.page_size, width, *at), S, dev, at, table.untyped_storage(), lens.untyped_storage(),
                stack.untyped_storage(), state.untyped_storage())
        self.__dict__["_held"] = held
        return held

    @staticmethod
    def empty(n_seqs: int, max_pages: int, num_pages: int, page_size: int, device) -> "PagePool":
        """A pool of num_pages free pages and n_seqs requests without tokens."""
        i32 = dict(dtype=torch.int32, device=device)
        state = torch.zeros(4, **i32)
        state[0] = num_pages
        return PagePool(torch.full((n_seqs, max_pages), -1, **i32), torch.zeros(n_seqs, **i32),
                        torch.arange(num_pages - 1, -1, -1, **i32), state, page_size)


def build_page_tables(pool: PagePool, new_len, seq_tokens: int = 0, tok_cap: int = 0, depth=None, cu_new=None,
                      slots=None, positions=None, stream=None):
    """msa_build_page_tables: every request of the pool from its length to
    new_len [n_seqs].  Returns (cu_new, slots, positions): with seq_tokens = T
    [n_seqs * T] padded, with tok_cap [tok_cap] packed token outputs, with
    neither None (a call that only resizes)."""
    c, S, dev = pool._hold()[:3]
    _same(new_len, "new_len", torch.int32, (S,), dev)
    if seq_tokens < 0 or tok_cap < 0:
        raise ValueError("seq_tokens, tok_cap: must not be negative")
    total = S * seq_tokens if seq_tokens else tok_cap
    if total >> 31 or tok_cap >> 31:
        raise ValueError("seq_tokens, tok_cap: more than 2^31 - 1 token outputs")
    if not total and not (slots is None and positions is None and depth is None):
        raise ValueError("slots, positions, depth: need seq_tokens or tok_cap")
    if depth is not None:
        _per_token(depth, "depth", total, dev)
    if cu_new is not None:
        _same(cu_new, "cu_new", torch.int32, (S + 1,), dev)
    if slots is not None:
        _same(slots, "slots", torch.int32, (total,), dev)
    if positions is not None:
        _same(positions, "positions", torch.int32, (total,), dev)
    if not new_len.is_cuda:
        _cuda(page_table=pool.page_table)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return build_page_tables(pool, new_len, seq_tokens, tok_cap, depth, cu_new, slots, positions)
    if cu_new is None:
        cu_new = torch.empty(S + 1, dtype=torch.int32, device=dev)
    if total:
        if slots is None:
            slots = torch.empty(total, dtype=torch.int32, device=dev)
        if positions is None:
            positions = torch.empty(total, dtype=torch.int32, device=dev)
    st = load().msa_build_page_tables(ctypes.byref(c), new_len.data_ptr(), _at(depth), int(seq_tokens),
                                      int(tok_cap), cu_new.data_ptr(), _at(slots), _at(positions),
                                      torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, "msa_build_page_tables")
    return cu_new, slots, positions


class RopeCfg:
    """How qk_norm_rope treats a head (msa_rope_cfg); see rope_cfg().  q_weight and k_weight may be replaced: each call
    checks and uses the ones that are there."""

    def __init__(self, c, q_weight, k_weight, inv_freq):
        self.c, self.q_weight, self.k_weight, self.inv_freq = c, q_weight, k_weight, inv_freq

    def check(self, d, device):
        q, k, c = self.q_weight, self.k_weight, self.c
        if q is not None:
            _same(q, "q_weight", torch.bfloat16, (d,), device)
        if k is not None:
            _same(k, "k_weight", torch.bfloat16, (d,), device)
        c.q_weight, c.k_weight = _at(q), _at(k)


def rope_cfg(rot_dim: int, theta: float = 10000.0, interleaved: bool = False, norm: bool = False, eps: float = 1e-6,
             q_weight=None, k_weight=None, inv_freq=None, rot_scale: float = 1.0) -> RopeCfg:
    """Rotation of the first rot_dim columns by position * theta^(-2i / rot_dim)
    (or by the rot_dim / 2 angles per position of the sequence inv_freq), after
    an RMS norm with weights [d] (None: ones) when norm is set."""
    arr = None
    if inv_freq is not None:
        vals = [float(x) for x in inv_freq]
        if len(vals) != int(rot_dim) // 2:
            raise ValueError(f"inv_freq: {len(vals)} values, expected {int(rot_dim) // 2}")
        arr = (ctypes.c_double * len(vals))(*vals)
    c = RopeCfgC(1 if norm else 0, float(eps), None, None, int(rot_dim), 1 if interleaved else 0,
                 float(theta), arr, float(rot_scale))
    return RopeCfg(c, q_weight, k_weight, arr)


def _token_rows(t, what, lead, H, d, device):
    """Token stride (elements) of a token-major tensor [*lead, H, d] whose heads are contiguous within a token."""
    want = (*lead, H, d)
    if not (isinstance(t, torch.Tensor) and t.shape == want and t.dtype is torch.bfloat16 and t.device == device):
        if not isinstance(t, torch.Tensor) or t.dim() != len(want):
            raise ValueError(f"{what}: a {len(want)}-d tensor [..., H, d] is required")
        if t.dtype is not torch.bfloat16:
            raise ValueError(f"{what}: dtype {t.dtype}, expected {torch.bfloat16}")
        if t.shape[:-2] != lead:
            raise ValueError(f"{what}: leading dimensions {tuple(t.shape[:-2])}, expected {tuple(lead)}")
        if t.shape != want:
            raise ValueError(f"{what}: heads {tuple(t.shape[-2:])}, expected {(H, d)}")
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    st = t.stride()
    if (d > 1 and st[-1] != 1) or (H > 1 and st[-2] != d):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    if len(lead) == 1:
        return st[0] if lead[0] > 1 else H * d
    B, n = lead
    if n > 1:
        if B > 1 and st[0] != n * st[1]:
            raise ValueError(f"{what}: tokens must lie at one stride")
        return st[1]
    return st[0] if B > 1 else H * d


def _per_token(t, what, tokens, device):
    """One int32 per token, in any shape."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.numel() == tokens and t.device == device
            and t.is_contiguous()):
        if isinstance(t, torch.Tensor) and t.numel() != tokens:
            raise ValueError(f"{what}: {t.numel()} elements, expected {tokens}")
        _want(t, what, torch.int32, device=device)


def _rope_args(lead, out, dims, q_in, k_in, v_in, cfg, positions, q, k, v, pages, slots):
    """Check everything; returns (token strides of q_in, k_in and v_in, C view of the pages or None).  pages: KV4Pages,
    or the pair k_pages, v_pages."""
    Hq, Hkv, d = dims
    dev = q_in.device
    qs = _token_rows(q_in, "q_in", lead, Hq, d, dev)
    ks = _token_rows(k_in, "k_in", lead, Hkv, d, dev)
    vs = 0 if v_in is None else _token_rows(v_in, "v_in", lead, Hkv, d, dev)
    cfg.check(d, dev)
    if isinstance(pages, KV4Pages):
        if slots is None or v_in is None:
            raise ValueError(f"{'slots' if slots is None else 'v_in'}: a torch.Tensor is required")
        pages = pages.view(Hkv, d, dev)
    else:
        pages = None if pages[0] is None and pages[1] is None else _pages(*pages, Hkv, d, dev)
    tokens = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    if positions is not None:
        _per_token(positions, "positions", tokens, dev)
    if slots is not None:
        _per_token(slots, "slots", tokens, dev)
    if q is not None:
        _same(q, "q", torch.bfloat16, out[0], dev)
    if k is not None:
        _same(k, "k", torch.bfloat16, out[1], dev)
    if v is not None:
        _same(v, "v", torch.bfloat16, out[1], dev)
    if not q_in.is_cuda:
        _cuda(q_in=q_in)
    return qs, ks, vs, pages


def _norm_rope(name, q_in, k_in, v_in, cfg, positions, q, k, v, pages, slots, layer_kv, stream):
    """qk_norm_rope and qk_norm_rope_kv4, of which `name` is the C name."""
    for t, what in ((q_in, "q_in"), (k_in, "k_in")):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{what}: a 4-d tensor [B, n, H, d] is required")
    B, n, Hq, d = q_in.shape
    Hkv, dev = k_in.shape[2], q_in.device
    kv = (B, Hkv, n, d)
    qs, ks, vs, held = _rope_args((B, n), ((B, Hq, n, d), kv), (Hq, Hkv, d), q_in, k_in, v_in, cfg, positions, q, k, v,
                                  pages, slots)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return _norm_rope(name, q_in, k_in, v_in, cfg, positions, q, k, v, pages, slots, layer_kv, None)
    if q is None:
        q = torch.empty((B, Hq, n, d), dtype=torch.bfloat16, device=dev)
    if layer_kv:
        if k is None:
            k = torch.empty(kv, dtype=torch.bfloat16, device=dev)
        if v is None and v_in is not None:
            v = torch.empty(kv, dtype=torch.bfloat16, device=dev)
    st = getattr(load(), name)(ctypes.byref(Shape(B, Hq, Hkv, n, d, 0.0)), ctypes.byref(cfg.c), q_in.data_ptr(), qs,
                               k_in.data_ptr(), ks, _at(v_in), vs, _at(positions), q.data_ptr(), _at(k), _at(v),
                               None if held is None else ctypes.byref(held), _at(slots),
                               torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, name)
    return q, k, v


def _norm_rope_varlen(name, q_in, k_in, v_in, cu, cfg, positions, q, k, v, pages, slots, layer_kv, stream):
    """The packed forms, of which `name` is the C name."""
    for t, what in ((q_in, "q_in"), (k_in, "k_in")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{what}: a 3-d tensor [tokens, H, d] is required")
    cu = [int(x) for x in cu]
    tokens, Hq, d = q_in.shape
    Hkv, dev = k_in.shape[1], q_in.device
    if len(cu) < 2 or cu[-1] != tokens:
        raise ValueError(f"cu_seqlens: must end at the {tokens} tokens of q_in")
    qn, kn = tokens * Hq * d, tokens * Hkv * d
    qs, ks, vs, held = _rope_args((tokens,), ((qn,), (kn,)), (Hq, Hkv, d), q_in, k_in, v_in, cfg, positions, q, k, v,
                                  pages, slots)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return _norm_rope_varlen(name, q_in, k_in, v_in, cu, cfg, positions, q, k, v, pages, slots, layer_kv, None)
    if q is None:
        q = torch.empty(qn, dtype=torch.bfloat16, device=dev)
    if layer_kv:
        if k is None:
            k = torch.empty(kn, dtype=torch.bfloat16, device=dev)
        if v is None and v_in is not None:
            v = torch.empty(kn, dtype=torch.bfloat16, device=dev)
    st = getattr(load(), name)(ctypes.byref(Shape(1, Hq, Hkv, 1, d, 0.0)), (ctypes.c_int32 * len(cu))(*cu),
                               len(cu) - 1, ctypes.byref(cfg.c), q_in.data_ptr(), qs, k_in.data_ptr(), ks,
                               _at(v_in), vs, _at(positions), q.data_ptr(), _at(k), _at(v),
                               None if held is None else ctypes.byref(held), _at(slots),
                               torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, name)
    return q, k, v


def qk_norm_rope(q_in, k_in, v_in, cfg: RopeCfg, positions=None, q=None, k=None, v=None, k_pages=None, v_pages=None,
                 slots=None, layer_kv: bool = True, stream=None):
    """msa_qk_norm_rope: q_in [B, n, Hq, d], k_in / v_in [B, n, Hkv, d] (views
    of the projection's rows) to (q [B, Hq, n, d], k, v [B, Hkv, n, d]) and,
    with k_pages / v_pages and slots, into the cache.  layer_kv=False leaves k
    and v to the cache alone (returned as given, or None)."""
    return _norm_rope("msa_qk_norm_rope", q_in, k_in, v_in, cfg, positions, q, k, v, (k_pages, v_pages), slots,
                      layer_kv, stream)


def qk_norm_rope_varlen(q_in, k_in, v_in, cu_seqlens, cfg: RopeCfg, positions=None, q=None, k=None, v=None,
                        k_pages=None, v_pages=None, slots=None, layer_kv: bool = True, stream=None):
    """msa_qk_norm_rope_varlen: packed q_in [tokens, Hq, d], k_in / v_in
    [tokens, Hkv, d] to flat buffers in the varlen layout (see pack_varlen)
    and, as for qk_norm_rope, the cache."""
    return _norm_rope_varlen("msa_qk_norm_rope_varlen", q_in, k_in, v_in, cu_seqlens, cfg, positions, q, k, v,
                             (k_pages, v_pages), slots, layer_kv, stream)


class KV4Pages:
    """A pool of 4-bit cache pages (msa_kv4_pages): data, uint8 [num_pages, Hkv,
    kv4_page_bytes(page_size, d)], for heads of d channels, and the tensors'
    scales, powers of two.  data may be replaced: each call checks and uses the
    tensor that is there."""

    def __init__(self, data, page_size: int, d: int, k_scale: float = 1.0, v_scale: float = 1.0):
        self.data, self.page_size, self.d = data, int(page_size), int(d)
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        if not self.k_scale > 0 or not self.v_scale > 0:
            raise ValueError("k_scale, v_scale: must be positive")
        if not isinstance(data, torch.Tensor) or data.dim() != 3:
            raise ValueError("data: a 3-d tensor [num_pages, Hkv, bytes] is required")

    @staticmethod
    def empty(num_pages: int, Hkv: int, page_size: int, d: int, device, k_scale: float = 1.0,
              v_scale: float = 1.0) -> "KV4Pages":
        """A pool whose values are all zero."""
        data = torch.zeros(num_pages, Hkv, kv4_page_bytes(page_size, d), dtype=torch.uint8, device=device)
        return KV4Pages(data, page_size, d, k_scale, v_scale)

    def view(self, Hkv, d, device):
        """C view of the pages, checked against Hkv heads (None: any) of d channels on `device`."""
        t = self.data
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError("data: a 3-d tensor [num_pages, Hkv, bytes] is required")
        if d != self.d:
            raise ValueError(f"pages: heads of {self.d} channels, expected {d}")
        N, H, _ = t.shape
        _same(t, "data", torch.uint8, (N, H if Hkv is None else Hkv, kv4_page_bytes(self.page_size, d)), device)
        return KV4PagesC(t.data_ptr(), N, self.page_size, self.k_scale, self.v_scale)


def kv4_page_bytes(page_size: int, d: int) -> int:
    """Bytes that the K and V of one page and head take in a 4-bit cache."""
    return 2 * int(page_size) * (int(d) // 2 + int(d) // 16)


def _kv4(pages):
    if not isinstance(pages, KV4Pages):
        raise ValueError("pages: KV4Pages are required")
    return pages


def qk_norm_rope_kv4(q_in, k_in, v_in, cfg: RopeCfg, pages: KV4Pages, slots, positions=None, q=None, k=None, v=None,
                     layer_kv: bool = False, stream=None):
    """msa_qk_norm_rope_kv4: as qk_norm_rope, K and V into the slots of a 4-bit
    cache.  layer_kv=True also returns them in bf16 in the layer's layout (not
    the cached values: see kv4_gather)."""
    return _norm_rope("msa_qk_norm_rope_kv4", q_in, k_in, v_in, cfg, positions, q, k, v, _kv4(pages), slots, layer_kv,
                      stream)


def qk_norm_rope_varlen_kv4(q_in, k_in, v_in, cu_seqlens, cfg: RopeCfg, pages: KV4Pages, slots, positions=None, q=None,
                            k=None, v=None, layer_kv: bool = False, stream=None):
    """msa_qk_norm_rope_varlen_kv4: the packed form of qk_norm_rope_kv4."""
    return _norm_rope_varlen("msa_qk_norm_rope_varlen_kv4", q_in, k_in, v_in, cu_seqlens, cfg, positions, q, k, v,
                             _kv4(pages), slots, layer_kv, stream)


def kv4_gather(pages: KV4Pages, page_table, seq_len, n: int, k=None, v=None, stream=None):
    """msa_kv4_gather: the first min(seq_len[b], n) cached tokens of every
    request to (k, v) [B, Hkv, n, d] bf16; the rows behind them keep what a
    given k and v hold, and are zero otherwise."""
    data, d, n = _kv4(pages).data, pages.d, int(n)
    c = pages.view(None, d, getattr(data, "device", None))
    dev, H = data.device, data.shape[1]
    if n < 1 or n >> 31:
        raise ValueError(f"n: {n}")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table: a 2-d tensor [B, max_pages] is required")
    B, width = page_table.shape
    _same(page_table, "page_table", torch.int32, (B, width), dev)
    _same(seq_len, "seq_len", torch.int32, (B,), dev)
    if k is not None:
        _same(k, "k", torch.bfloat16, (B, H, n, d), dev)
    if v is not None:
        _same(v, "v", torch.bfloat16, (B, H, n, d), dev)
    if not data.is_cuda:
        _cuda(data=data)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return kv4_gather(pages, page_table, seq_len, n, k, v)
    if k is None:
        k = torch.zeros(B, H, n, d, dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.zeros(B, H, n, d, dtype=torch.bfloat16, device=dev)
    st = load().msa_kv4_gather(ctypes.byref(Shape(B, H, H, n, d, 0.0)), ctypes.byref(c), page_table.data_ptr(), width,
                               seq_len.data_ptr(), k.data_ptr(), v.data_ptr(),
                               torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, "msa_kv4_gather")
    return k, v


def _query(q):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q: a 4-d tensor [B, Hq, n, d] is required")
    _want(q, "q", torch.bfloat16)


def _tree_args(q, page_table, seq_len, tree_len, tree_mask, depth, o, lse, ws):
    """Check what the attentions of drafted tokens share; returns (columns of the page table, stride of the masks)."""
    B, Hq, n, d = q.shape
    dev = q.device
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table: a 2-d tensor [B, max_pages] is required")
    width = page_table.shape[1]
    _same(page_table, "page_table", torch.int32, (B, width), dev)
    _same(seq_len, "seq_len", torch.int32, (B,), dev)
    if tree_len is not None:
        _same(tree_len, "tree_len", torch.int32, (B,), dev)
    stride = 0
    if tree_mask is not None:
        words = (n + 31) // 32
        shared = isinstance(tree_mask, torch.Tensor) and tree_mask.dim() == 2
        _same(tree_mask, "tree_mask", torch.int32, (n, words) if shared else (B, n, words), dev)
        stride = 0 if shared else n * words
    if depth is not None:
        _same(depth, "depth", torch.int32, (B, n), dev)
    if o is not None:
        _same(o, "o", torch.bfloat16, (B, Hq, n, d), dev)
    if lse is not None:
        _same(lse, "lse", torch.float32, (B, Hq, n), dev)
    if ws is not None:
        _want(ws, "ws", torch.uint8, device=dev)
    if not q.is_cuda:
        _cuda(q=q)
    return width, stride


def _window(sink, window, depth, tree_mask):
    """Check a window (its depth needs a mask); returns (sink, window)."""
    sink, window = int(sink), int(window)
    if sink < 0 or sink >> 31:
        raise ValueError(f"sink: {sink}")
    if window < 1 or window >> 31:
        raise ValueError(f"window: {window}")
    if depth is not None and tree_mask is None:
        raise ValueError("depth: needs a tree_mask")
    return sink, window


def attn_tree(q, k_pages, v_pages, page_table, seq_len, tree_len=None, tree_mask=None, o=None, lse=None, scale=None,
              ws=None, stream=None):
    """msa_attn_tree: drafted tokens (n = 1: a decode step) q [B, Hq, n, d] over
    the paged cache; seq_len [B] counts the drafted tokens.  tree_len [B];
    tree_mask [B, n, ceil(n/32)] or, for all requests, [n, ceil(n/32)] int32
    words (None: a chain).  Returns o.  ws: a uint8 workspace of at least
    attn_tree_workspace(...) bytes (None: one is allocated for the call)."""
    _query(q)
    B, Hq, n, d = q.shape
    dev = q.device
    pages = _pages(k_pages, v_pages, None, d, dev)
    width, stride = _tree_args(q, page_table, seq_len, tree_len, tree_mask, None, o, lse, ws)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_tree(q, k_pages, v_pages, page_table, seq_len, tree_len, tree_mask, o, lse, scale, ws)
    lib = load()
    sh = ctypes.byref(Shape(B, Hq, k_pages.shape[1], n, d, float(scale) if scale else 0.0))
    if o is None:
        o = torch.empty_like(q)
    if ws is None:
        ws = torch.empty(lib.msa_attn_tree_workspace(sh) or 1, dtype=torch.uint8, device=dev)
    st = lib.msa_attn_tree(sh, q.data_ptr(), ctypes.byref(pages), page_table.data_ptr(), width, seq_len.data_ptr(),
                           _at(tree_len), _at(tree_mask), stride, o.data_ptr(), _at(lse), ws.data_ptr(), ws.numel(),
                           torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, "msa_attn_tree")
    return o


def attn_tree_window(q, k_pages, v_pages, page_table, seq_len, sink: int, window: int, tree_len=None, tree_mask=None,
                     depth=None, o=None, lse=None, scale=None, ws=None, stream=None):
    """msa_attn_tree_window: attn_tree through a sliding window of `window`
    keys that keeps the first `sink` tokens visible.  depth [B, n] int32: how
    far behind the context each token of a masked tree stands (None: its
    index).  Pages that no row sees may be gone."""
    _query(q)
    B, Hq, n, d = q.shape
    dev = q.device
    pages = _pages(k_pages, v_pages, None, d, dev)
    seen = _window(sink, window, depth, tree_mask)
    width, stride = _tree_args(q, page_table, seq_len, tree_len, tree_mask, depth, o, lse, ws)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_tree_window(q, k_pages, v_pages, page_table, seq_len, sink, window, tree_len, tree_mask, depth,
                                    o, lse, scale, ws)
    lib = load()
    sh = ctypes.byref(Shape(B, Hq, k_pages.shape[1], n, d, float(scale) if scale else 0.0))
    win = TreeWindowC(*seen, _at(depth))
    if o is None:
        o = torch.empty_like(q)
    if ws is None:
        ws = torch.empty(lib.msa_attn_tree_workspace(sh) or 1, dtype=torch.uint8, device=dev)
    st = lib.msa_attn_tree_window(sh, q.data_ptr(), ctypes.byref(pages), page_table.data_ptr(), width,
                                  seq_len.data_ptr(), _at(tree_len), _at(tree_mask), stride, ctypes.byref(win),
                                  o.data_ptr(), _at(lse), ws.data_ptr(), ws.numel(),
                                  torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, "msa_attn_tree_window")
    return o


def attn_tree_kv4(q, pages: KV4Pages, page_table, seq_len, sink: int = 0, window: int = 0, tree_len=None,
                  tree_mask=None, depth=None, o=None, lse=None, scale=None, ws=None, stream=None):
    """msa_attn_tree_kv4: attn_tree over a 4-bit cache; with window > 0 as
    attn_tree_window (0: every key, and then no sink and no depth)."""
    _query(q)
    B, Hq, n, d = q.shape
    dev = q.device
    held = _kv4(pages).view(None, d, dev)
    if not window and (sink or depth is not None):
        raise ValueError("sink, depth: need a window")
    seen = _window(sink, window, depth, tree_mask) if window else None
    width, stride = _tree_args(q, page_table, seq_len, tree_len, tree_mask, depth, o, lse, ws)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return attn_tree_kv4(q, pages, page_table, seq_len, sink, window, tree_len, tree_mask, depth, o, lse, scale,
                                 ws)
    lib = load()
    sh = ctypes.byref(Shape(B, Hq, pages.data.shape[1], n, d, float(scale) if scale else 0.0))
    win = ctypes.byref(TreeWindowC(*seen, _at(depth))) if seen else None
    if o is None:
        o = torch.empty_like(q)
    if ws is None:
        ws = torch.empty(lib.msa_attn_tree_kv4_workspace(sh) or 1, dtype=torch.uint8, device=dev)
    st = lib.msa_attn_tree_kv4(sh, q.data_ptr(), ctypes.byref(held), page_table.data_ptr(), width, seq_len.data_ptr(),
                               _at(tree_len), _at(tree_mask), stride, win, o.data_ptr(), _at(lse), ws.data_ptr(),
                               ws.numel(), torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        raise MsaError(st, "msa_attn_tree_kv4")
    return o


def attn_tree_workspace(B, Hq, Hkv, n, d) -> int:
    """Workspace bytes of attn_tree (0: unsupported shape)."""
    return int(load().msa_attn_tree_workspace(ctypes.byref(Shape(B, Hq, Hkv, n, d, 0.0))))


def attn_tree_kv4_workspace(B, Hq, Hkv, n, d) -> int:
    """Workspace bytes of attn_tree_kv4 (0: unsupported shape)."""
    return int(load().msa_attn_tree_kv4_workspace(ctypes.byref(Shape(B, Hq, Hkv, n, d, 0.0))))


def kernel_launches() -> int:
    """Kernels launched through the library by this process so far."""
    return int(load().msa_kernel_launches())


def check_wait_timeout(limit_ms: int, stream=None):
    """Launch the failure-detection check (a bounded wait that runs out)."""
    _check(load().msa_check_wait_timeout(int(limit_ms), _stream(stream)), "msa_check_wait_timeout")


def poll_device_status(stream=None) -> int:
    """Synchronise the stream and read/clear the device error word (status code)."""
    return int(load().msa_poll_device_status(_stream(stream)))
