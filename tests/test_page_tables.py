"""Page tables and slot maps built on the GPU (msa_build_page_tables).

CPU: the reference itself (growing and rolling back restores the pool) and the
host checks.  GPU: every table, stack, slot and position equal to the reference's,
over grow, shrink, mixed, refused and repeated calls."""
import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import long_context_prefill_gb300 as msa
from paged_ref import resize

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _pool(rng, S, width, N, lens, page):
    perm = rng.permutation(N).tolist()
    table, used = [], 0
    for x in lens:
        p = -(-x // page)
        table.append(perm[used:used + p] + [-7] * (width - p))
        used += p
    left = perm[used:]
    return table, list(lens), left + [-9] * (N - len(left)), [len(left), 0, 0, 0]


def test_reference_rolls_back():
    rng = np.random.default_rng(0)
    for page in (16, 64):
        lens = rng.integers(0, 300, 9).tolist()
        table, sl, stack, state = _pool(rng, 9, 40, 300, lens, page)
        before = (list(sl), list(stack), list(state))
        new = [x + int(rng.integers(0, 200)) for x in lens]
        cu, slots, pos = resize(table, sl, stack, state, new, page, tok_cap=5000)
        assert sl == new and cu[-1] == sum(new) - sum(lens)
        live = [x for x in slots if x >= 0]
        assert len(live) == len(set(live)) == cu[-1]
        owned = [p for s in range(9) for p in table[s][:-(-new[s] // page)]]
        assert len(owned) == len(set(owned)) and not set(owned) & set(stack[:state[0]])
        resize(table, sl, stack, state, lens, page)
        assert (sl, stack, state) == before


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_gb300 import build
    build.build()
    return msa.load()


def test_refusals(lib):
    P = ctypes.c_void_p(0x10000)

    def call(pool=None, new=ctypes.c_void_p(0x20000), depth=None, T=0, cap=0, cu=None, slots=None, pos=None, **kw):
        base = dict(n_seqs=4, num_pages=64, page_size=16, max_pages=8, page_table=0x10000, seq_len=0x30000,
                    free_pages=0x40000, state=0x50000)
        base.update(kw)
        c = msa.PagePoolC(*(base[k] for k, _ in msa.PagePoolC._fields_))
        return lib.msa_build_page_tables(ctypes.byref(c), new, depth, T, cap, cu, slots, pos, None)

    inv, uns = msa.MSA_ERR_INVALID_ARG, msa.MSA_ERR_UNSUPPORTED
    assert lib.msa_build_page_tables(None, P, None, 0, 0, None, None, None, None) == inv
    assert call(n_seqs=0) == inv
    assert call(max_pages=0) == inv
    assert call(num_pages=0) == inv
    assert call(page_size=0) == inv
    assert call(page_size=48) == uns
    assert call(page_size=256) == uns
    assert call(n_seqs=8193) == uns
    assert call(num_pages=1 << 27) == uns
    assert call(page_table=0) == inv
    assert call(state=0x50002) == inv
    assert call(new=None) == inv
    assert call(new=ctypes.c_void_p(0x30000)) == inv  # the pool's own lengths
    assert call(T=-1) == inv
    assert call(cap=-1) == inv
    assert call(slots=P, T=(1 << 29) - 1) == uns  # 2^31 - 4 token outputs
    assert call(slots=P, cap=(1 << 31) - 1) == uns
    assert call(pos=P) == inv    # positions without slots
    assert call(depth=P) == inv


def test_binding_refusals():
    i32 = dict(dtype=torch.int32)
    pool = msa.PagePool.empty(4, 8, 64, 16, "cpu")
    new = torch.zeros(4, **i32)
    for call, what in [
        (lambda: msa.build_page_tables(pool, new[:3]), "new_len: shape"),
        (lambda: msa.build_page_tables(pool, new.long()), "new_len: dtype"),
        (lambda: msa.build_page_tables(pool, new, slots=new), "need seq_tokens"),
        (lambda: msa.build_page_tables(pool, new, seq_tokens=2, depth=new), "depth: 4 elements"),
        (lambda: msa.build_page_tables(pool, new, seq_tokens=1, depth=[0] * 4), "depth: a torch.Tensor"),
        (lambda: msa.build_page_tables(pool, new, tok_cap=6, slots=new), "slots: shape"),
        (lambda: msa.build_page_tables(pool, new, tok_cap=-6), "tok_cap"),
        (lambda: msa.build_page_tables(pool, new), "page_table: must be on a CUDA device"),
        (lambda: msa.PagePool(new, new, new, new, 16), "page_table: a 2-d"),
        (lambda: msa.PagePool(torch.zeros(4, 8, **i32), new[:3], new, new, 16), "seq_len: shape"),
        (lambda: msa.PagePool(torch.zeros(4, 8, **i32), new, new, new[:2], 16), "state: shape"),
    ]:
        with pytest.raises(ValueError, match=what):
            call()


class Both:
    """A pool on the GPU and the reference's lists, kept in step."""

    def __init__(self, lists, page):
        self.table, self.lens, self.stack, self.state = lists
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.pool = msa.PagePool(t(self.table), t(self.lens), t(self.stack), t(self.state), page)
        self.page = page

    def step(self, new, T=0, cap=0, depth=None, what=""):
        t = torch.tensor(new, dtype=torch.int32, device="cuda")
        d = None if depth is None else torch.tensor(depth, dtype=torch.int32, device="cuda")
        got = msa.build_page_tables(self.pool, t, seq_tokens=T, tok_cap=cap, depth=d)
        want = resize(self.table, self.lens, self.stack, self.state, list(new), self.page, T, None if T else (cap or None), depth)
        for g, w, name in zip(got, want, ("cu", "slots", "positions")):
            assert (g is None) == (w is None), f"{what}: {name}"
            if g is not None:
                assert g.tolist() == w, f"{what}: {name}"
        p = self.pool
        assert p.page_table.tolist() == self.table, f"{what}: page_table"
        assert p.seq_len.tolist() == self.lens, f"{what}: seq_len"
        assert p.free_pages.tolist() == self.stack, f"{what}: free_pages"
        assert p.state.tolist() == self.state, f"{what}: state"
        return got


@pytest.mark.gpu
@pytest.mark.parametrize("S,page,top", [(1, 16, 5), (1, 64, 40000), (7, 16, 100), (64, 64, 3000), (513, 128, 500),
                                        (1021, 16, 300)])
def test_grow_mix_and_roll_back(cuda_lib, S, page, top):
    rng = np.random.default_rng(S + page)
    lens = rng.integers(0, top + 1, S).tolist()
    width = -(-(3 * top + 70) // page)
    need = sum(-(-x // page) for x in lens)
    b = Both(_pool(rng, S, width, need + S * width // 2 + 5, lens, page), page)
    grown = [x + int(rng.integers(0, top)) for x in lens]
    b.step(grown, cap=sum(grown) - sum(lens) + 3, what="packed prefill")
    T = 48
    step = [x + int(rng.integers(0, T + 1)) for x in grown]
    depth = rng.integers(0, T, S * T).tolist()
    b.step(step, T=T, depth=depth, what="padded trees")
    b.step([g + int(rng.integers(0, s - g + 1)) for g, s in zip(grown, step)], what="accepted")
    mixed = [0 if rng.random() < 0.4 else min(x + int(rng.integers(0, top + 1)), width * page) for x in b.lens]
    b.step(mixed, cap=S * (top + 1), what="finish some, grow others")
    b.step([0] * S, what="all finished")
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_refused_requests_keep_what_they_have(cuda_lib):
    rng = np.random.default_rng(5)
    page = 16
    b = Both(_pool(rng, 6, 20, 30, [100, 0, 40, 33, 7, 16], page), page)  # 7+3+3+1+1 pages held, 15 free
    b.step([100 + 64, 12 * 16, 41, 64, 16, 17], cap=1000, what="out of pages from request 1 on")
    assert b.state[1] == 3 and b.lens[2] == 41 and b.lens[4] == 16  # those that need no page are served
    b.step([0, 150, 41, 64, 16, 17], cap=1000, what="released pages serve the same call")
    b.step([3, 160, 50, 70, 20, 20], cap=9, what="packed tokens end at the capacity")
    assert b.state[1] > 0
    assert cuda_lib.poll_device_status() == 0
    b.step([3, 160, 50, 70, 20, 21 + 8], T=8, what="padded: more new tokens than fit")
    assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX
    b.step([-1, 160, 20 * 16 + 1, 70, 20, 20], cap=100, what="bad lengths")
    assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
def test_inconsistent_pool_is_left_alone(cuda_lib):
    rng = np.random.default_rng(6)
    lists = _pool(rng, 3, 4, 8, [16, 16, 16], 16)
    lists[3][0] = 8  # says every page is free while three are held
    b = Both(lists, 16)
    b.step([0, 32, 16], cap=16, what="more pages than the pool has")
    assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX
    assert b.lens == [16, 16, 16] and b.state[0] == 8


@pytest.mark.gpu
def test_stack_with_a_page_outside_the_pool(cuda_lib):
    pool = msa.PagePool.empty(2, 4, 8, 16, "cuda")
    pool.free_pages[7] = 99  # top of the stack
    _, slots, _ = msa.build_page_tables(pool, torch.tensor([16, 16], dtype=torch.int32, device="cuda"), seq_tokens=16)
    assert cuda_lib.poll_device_status() == msa.MSA_ERR_INDEX
    assert slots[:16].tolist() == [-1] * 16 and slots[16:].tolist() == list(range(16, 32))


@pytest.mark.gpu
def test_captured_steps_follow_the_lengths(cuda_lib):
    """A captured grow-by-one replayed: lengths, pages and slots move on."""
    pool = msa.PagePool.empty(5, 8, 40, 16, "cuda")
    new = torch.zeros(5, dtype=torch.int32, device="cuda")
    cu = torch.empty(6, dtype=torch.int32, device="cuda")
    slots, pos = (torch.empty(5, dtype=torch.int32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        torch.add(pool.seq_len, 1, out=new)
        msa.build_page_tables(pool, new, seq_tokens=1, cu_new=cu, slots=slots, positions=pos)
    table, lens, stack, state = [[-1] * 8 for _ in range(5)], [0] * 5, list(range(39, -1, -1)), [40, 0, 0, 0]
    for step in range(40):
        graph.replay()
        _, ws, wp = resize(table, lens, stack, state, [x + 1 for x in lens], 16, seq_tokens=1)
        torch.cuda.synchronize()
        assert slots.tolist() == ws and pos.tolist() == wp and pool.seq_len.tolist() == lens, step
    assert pool.page_table.tolist() == table and pool.state.tolist() == state
    assert cuda_lib.poll_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[2437, 2438, 2456, 2457, 8192], [8192, 2438]])
def test_many_requests_in_a_fresh_process(cuda_lib, sizes):
    """Tables of up to the 8192 requests a pool may have, around the size whose scans need more shared memory than a
    kernel has by default; each size as the first of its kind in a process, and after a larger one."""
    code = f"""
import sys
sys.path[:0] = {[ROOT, os.path.join(ROOT, "tests")]!r}
import torch
import long_context_prefill_gb300 as msa
from paged_ref import resize
for S in {sizes}:
    pool = msa.PagePool.empty(S, 3, 2 * S, 16, "cuda")
    table, lens, stack, state = [[-1] * 3 for _ in range(S)], [0] * S, list(range(2 * S - 1, -1, -1)), [2 * S, 0, 0, 0]
    for new in ([(7 * s) % 33 for s in range(S)], [(5 * s) % 49 for s in range(S)], [0] * S):
        got = msa.build_page_tables(pool, torch.tensor(new, dtype=torch.int32, device="cuda"), tok_cap=24 * S)
        want = resize(table, lens, stack, state, new, 16, tok_cap=24 * S)
        assert [t.tolist() for t in got] == list(want), S
        assert pool.seq_len.tolist() == lens and pool.free_pages.tolist() == stack and pool.state.tolist() == state, S
        assert pool.page_table.tolist() == table, S
assert msa.poll_device_status() == 0
"""
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


@pytest.mark.gpu
def test_pools_of_different_sizes_from_two_threads(cuda_lib):
    """Two host threads, each with its own pool and stream, of sizes that need different amounts of shared memory."""
    def work(S, failed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                pool = msa.PagePool.empty(S, 2, 2 * S, 16, "cuda")
                lens = [torch.full((S,), x, dtype=torch.int32, device="cuda") for x in (17, 0)]
                for x in range(400):
                    msa.build_page_tables(pool, lens[x & 1])
                msa.build_page_tables(pool, lens[0])
                assert bool((pool.seq_len == 17).all()) and pool.state.tolist() == [0, 0, 0, 0]
        except Exception as e:  # noqa: BLE001  (a thread's failure is the test's)
            failed.append((S, e))

    failed = []
    threads = [threading.Thread(target=work, args=(S, failed)) for S in (2600, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert cuda_lib.poll_device_status() == 0


def test_pool_follows_its_tensors():
    """A tensor put in another's place, or one whose storage was replaced, is the one that the next call uses; one that
    does not fit is refused by name."""
    pool = msa.PagePool.empty(4, 8, 64, 16, "cpu")
    i32 = dict(dtype=torch.int32)
    old = [pool.page_table, pool.seq_len, pool.free_pages, pool.state]
    pool.page_table, pool.seq_len = torch.zeros(4, 9, **i32), torch.ones(4, **i32)
    pool.free_pages, pool.state = torch.zeros(70, **i32), torch.zeros(4, **i32)
    c = pool.view()
    assert (c.n_seqs, c.num_pages, c.page_size, c.max_pages) == (4, 70, 16, 9)
    assert [c.page_table, c.seq_len, c.free_pages, c.state] == [
        t.data_ptr() for t in (pool.page_table, pool.seq_len, pool.free_pages, pool.state)]
    assert all(t.data_ptr() != getattr(c, k) for t, k in zip(old, ("page_table", "seq_len", "free_pages", "state")))
    pool.seq_len.data = torch.full((4,), 5, **i32)
    assert pool.view().seq_len == pool.seq_len.data_ptr()
    new = torch.zeros(4, **i32)
    for name, bad, what in [("seq_len", torch.zeros(3, **i32), "seq_len: shape"), ("state", torch.zeros(4), "state: dtype"),
                            ("free_pages", new[None], "free_pages: a 1-d"), ("page_table", new, "page_table: a 2-d"),
                            ("page_table", torch.zeros(4, 9, **i32).t(), "page_table: must be contiguous"),
                            ("page_size", 1 << 32, "page_size")]:
        keep = getattr(pool, name)
        setattr(pool, name, bad)
        with pytest.raises(ValueError, match=what):
            msa.build_page_tables(pool, new)
        setattr(pool, name, keep)
    pool.seq_len.data = torch.zeros(3, **i32)
    with pytest.raises(ValueError, match="seq_len: shape"):
        msa.build_page_tables(pool, new)


@pytest.mark.gpu
def test_pool_with_a_tensor_replaced(cuda_lib):
    pool = msa.PagePool.empty(2, 4, 8, 16, "cuda")
    first = pool.seq_len
    pool.seq_len = torch.zeros(2, dtype=torch.int32, device="cuda")
    msa.build_page_tables(pool, torch.tensor([20, 3], dtype=torch.int32, device="cuda"))
    assert pool.seq_len.tolist() == [20, 3] and first.tolist() == [0, 0]
    second = pool.seq_len.detach()  # keeps the storage
    pool.seq_len.data = torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    msa.build_page_tables(pool, torch.tensor([33, 0], dtype=torch.int32, device="cuda"))
    assert pool.seq_len.tolist() == [33, 0] and second.tolist() == [20, 3]
    assert pool.state.tolist() == [5, 0, 0, 0]
    assert cuda_lib.poll_device_status() == 0


def test_token_counts_beyond_32_bits_are_refused():
    """Counts that the library's 32-bit arguments would cut off (to 0: no tokens at all)."""
    pool = msa.PagePool.empty(1, 8, 64, 16, "cpu")
    new = torch.zeros(1, dtype=torch.int32)
    for kw in (dict(seq_tokens=1 << 32), dict(tok_cap=1 << 32), dict(seq_tokens=1 << 31), dict(tok_cap=(1 << 33) + 5)):
        with pytest.raises(ValueError, match="seq_tokens, tok_cap: more than"):
            msa.build_page_tables(pool, new, **kw)


@pytest.mark.gpu
def test_tables_on_a_given_stream(cuda_lib):
    """Calls ordered on a stream other than the current one."""
    rng = np.random.default_rng(19)
    lists = _pool(rng, 70, 40, 4000, rng.integers(0, 300, 70).tolist(), 16)
    b = Both(lists, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        new = [x + int(rng.integers(0, 100)) for x in b.lens]
        t = torch.tensor(new, dtype=torch.int32, device="cuda")
        side.wait_stream(torch.cuda.current_stream())
        got = msa.build_page_tables(b.pool, t, tok_cap=7000, stream=side)
        side.synchronize()
        want = resize(b.table, b.lens, b.stack, b.state, new, 16, tok_cap=7000)
        assert [x.tolist() for x in got] == list(want)
        assert b.pool.page_table.tolist() == b.table and b.pool.seq_len.tolist() == b.lens
    assert cuda_lib.poll_device_status() == 0
