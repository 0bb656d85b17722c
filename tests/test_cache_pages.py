"""Page management of the cache against a host model: tables, lengths, counts and page contents
after extends, forks, frees and compactions, refusals, and random runs of all of them."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.cache import Pages


def make(pages, ps, Hkv, D, rows, width, layout="NHD", device="cuda", pool=True):
    inner = (ps, Hkv, D) if layout == "NHD" else (Hkv, ps, D)
    both = torch.randn(pages, 2, *inner, device=device).to(torch.bfloat16)
    k, v = (both[:, 0], both[:, 1]) if pool else (both[:, 0].contiguous(), both[:, 1].contiguous())
    i32 = dict(dtype=torch.int32, device=device)
    return k, v, torch.full((rows, width), 99, **i32), torch.full((rows,), 5, **i32), torch.full((pages,), 3, **i32)


def cache_of(arrays, Hq, layout="NHD"):
    import long_context_grpo_gb300 as ls
    return ls.PagedCache(*arrays, Hq=Hq, layout=layout)


def host(c):
    return Pages(c.page_table, c.seq_len, c.refcount, c.page_size)


def same(c, m):
    assert np.array_equal(c.page_table.cpu().numpy(), m.table)
    assert np.array_equal(c.seq_len.cpu().numpy(), m.len)
    assert np.array_equal(c.refcount.cpu().numpy(), m.ref)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def moved(before, moves, layout):
    """The pages after the moves, which read what was there before them."""
    out = before.clone()
    for src, dst, tokens in moves:
        if layout == "NHD":
            out[dst, :tokens] = before[src, :tokens]
        else:
            out[dst, :, :tokens] = before[src, :, :tokens]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("ps,layout,pool", [(16, "NHD", True), (64, "HND", True), (128, "NHD", False), (256, "HND", False)])
@pytest.mark.parametrize("Hkv,D", [(1, 64), (8, 128), (3, 64)])
def test_a_life_of_a_cache(ps, layout, pool, Hkv, D):
    import long_context_grpo_gb300 as ls
    pages, rows, width = 37, 7, 9
    c = cache_of(make(pages, ps, Hkv, D, rows, width, layout, pool=pool), Hkv, layout)
    c.reset()
    m = host(c)
    assert (m.table == -1).all() and not m.len.any() and not m.ref.any()
    # grow: nothing, part of a page, a page exactly, several; again from the middle of a page
    for add in ((0, 1, ps, 3 * ps + 2), (ps, ps - 1, 1, 0)):
        c.extend(i32(4, 0, 2, 6), i32(*add))
        m.extend([4, 0, 2, 6], add)
        same(c, m)
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    c.fork(i32(6, 6, 2), i32(1, 3, 5))
    m.fork([6, 6, 2], [1, 3, 5])
    same(c, m)
    assert torch.equal(c.k_pages, moved(k0, m.moves, layout)) and torch.equal(c.v_pages, moved(v0, m.moves, layout))
    c.extend(i32(1, 3, 6), i32(ps, 1, ps - 2))
    m.extend([1, 3, 6], [ps, 1, ps - 2])
    same(c, m)
    c.free(i32(6, 0, 5))
    m.free([6, 0, 5])
    same(c, m)
    # gather into a larger and a smaller pool, then together in place
    k0, v0 = c.k_pages.clone(), c.v_pages.clone()
    n = i32(-1)
    live = int((m.ref > 0).sum())
    for size in (pages + 5, live, live - 2):
        d = cache_of(make(size, ps, Hkv, D, rows, width, layout), Hkv, layout)
        kd, vd = d.k_pages.clone(), d.v_pages.clone()
        c.compact(into=d, n_live=n)
        want = m.compact_into(size)
        same(d, want)
        same(c, m)
        assert n.item() == live
        for src, dst, _ in want.moves:
            kd[dst], vd[dst] = k0[src], v0[src]
        assert torch.equal(d.k_pages, kd) and torch.equal(d.v_pages, vd)
        assert ls.device_status() == ((0, 0) if size >= live else (7, 4))
        d.close()
    c.compact(n_live=n)
    m.compact()
    same(c, m)
    assert n.item() == live and (c.refcount[live:] == 0).all() and (c.refcount[:live] > 0).all()
    assert torch.equal(c.k_pages, moved(k0, m.moves, layout)) and torch.equal(c.v_pages, moved(v0, m.moves, layout))
    c.compact()
    same(c, m)
    c.free(torch.arange(rows, dtype=torch.int32, device="cuda"))
    assert not c.refcount.any() and not c.seq_len.any()
    c.compact(n_live=n)
    assert n.item() == 0
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_refused_entries_leave_their_rows_and_are_reported():
    import long_context_grpo_gb300 as ls
    c = cache_of(make(10, 16, 1, 64, 6, 4), 1)
    c.reset()
    m = host(c)

    def both(name, *lists, bits):
        k0 = c.k_pages.clone()
        getattr(c, name)(*(i32(*x) for x in lists))
        getattr(m, name)(*lists)
        same(c, m)
        assert ls.device_status() == ((7, bits) if bits else (0, 0)), (name, lists)
        if name == "fork":
            assert torch.equal(c.k_pages, moved(k0, m.moves, "NHD"))

    both("extend", (0, 6, -1, 1, 0, 2), (20, 5, 5, -1, 9, 65), bits=2)     # rows, counts, twice, too long
    both("extend", (1, 2, 3), (33, 64, 16), bits=0)                        # the eight pages left
    both("extend", (4, 5), (1, 17), bits=4)
    both("free", (2, 2, 9, -3), bits=2)
    both("fork", (0, 0, 0, 7, 0, 3), (3, 4, 4, 5, 0, 2), bits=2)           # full child, child twice, parent row, itself
    both("extend", (5,), (64,), bits=4)
    both("fork", (1, 1), (5, 2), bits=2)
    both("free", (0, 1, 2, 3, 4, 5), bits=0)
    assert not c.refcount.any()


@pytest.mark.gpu
def test_want_of_pages_for_forks():
    import long_context_grpo_gb300 as ls
    c = cache_of(make(5, 16, 1, 64, 8, 4), 1)
    c.reset()
    m = host(c)
    c.extend(i32(0, 1), i32(17, 16))
    m.extend([0, 1], [17, 16])
    # two free pages: the third part-filled fork goes without, the whole-page one needs none
    c.fork(i32(0, 0, 0, 1, 2), i32(3, 4, 5, 6, 7))
    m.fork([0, 0, 0, 1, 2], [3, 4, 5, 6, 7])
    same(c, m)
    assert m.refused == 1 and ls.device_status() == (7, 4)


@pytest.mark.gpu
def test_wild_tables_are_reported_and_not_followed():
    """A page or a length outside the pool in the arrays: nothing is read or written through it."""
    import long_context_grpo_gb300 as ls
    k, v, table, length, ref = make(6, 16, 2, 64, 4, 3)
    table.fill_(-1)
    table[0, 0], table[0, 1], table[1, 0] = 1 << 30, 2, -9
    length.copy_(i32(20, 3, 999999, -4))
    ref.zero_()
    ref[2] = 1
    c = cache_of((k, v, table, length, ref), 2)
    k0 = k.clone()
    c.fork(i32(2, 3), i32(1, 1))
    assert ls.device_status() == (7, 2)
    length[3] = 0
    c.fork(i32(0), i32(3))                 # its first page is not in the pool, its last is copied
    assert ls.device_status() == (7, 2)
    assert ref.tolist() == [1, 0, 1, 0, 0, 0] and table[3].tolist() == [1 << 30, 0, -1]
    assert torch.equal(k[1:], k0[1:]) and torch.equal(k[0, :4], k0[2, :4])
    c.free(i32(0, 1, 2))
    assert ls.device_status() == (7, 2)
    assert ref.tolist() == [1, 0, 0, 0, 0, 0]
    c.compact()
    assert ls.device_status()[1] in (0, 2)
    assert ref.tolist() == [1, 0, 0, 0, 0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(4))
def test_random_lives(seed):
    import long_context_grpo_gb300 as ls
    rng = np.random.default_rng(seed)
    ps, layout = int(rng.choice([16, 32, 64])), ["NHD", "HND"][seed % 2]
    pages, rows, width = 3000, 60, 120
    c = cache_of(make(pages, ps, 1, 64, rows, width, layout), 1, layout)
    c.reset()
    m = host(c)
    for _ in range(30):
        op = rng.choice(["extend", "extend", "fork", "free", "compact"])
        k0, moves = c.k_pages.clone(), []
        if op == "compact":
            c.compact()
            m.compact()
            moves = m.moves
        else:
            n = int(rng.integers(1, 20))
            a = rng.integers(0, rows, n)
            if op == "free":
                c.free(i32(*a))
                m.free(a)
            else:
                x = rng.integers(0, 40 * ps, n) if op == "extend" else rng.integers(0, rows, n)
                getattr(c, op)(i32(*a), i32(*x))
                getattr(m, op)(a, x)
                moves = m.moves if op == "fork" else []
        same(c, m)
        assert torch.equal(c.k_pages, moved(k0, moves, layout)), op
        ls.device_status()


@pytest.mark.gpu
def test_large_pools_and_long_lists():
    """More pages than one scan step, 1024 entries, counts above one."""
    pages, rows, width = 150001, 1100, 200
    c = cache_of(make(pages, 16, 1, 64, rows, width), 1)
    c.reset()
    m = host(c)
    r = np.arange(1024)
    add = (r * 37) % 1600
    c.extend(torch.from_numpy(r).int().cuda(), torch.from_numpy(add).int().cuda())
    m.extend(r, add)
    same(c, m)
    c.free(torch.arange(0, 1024, 3, dtype=torch.int32, device="cuda"))
    m.free(range(0, 1024, 3))
    par, chi = np.full(70, 1), np.arange(1030, 1100)
    c.fork(torch.from_numpy(par).int().cuda(), torch.from_numpy(chi).int().cuda())
    m.fork(par, chi)
    same(c, m)
    k0 = c.k_pages.clone()
    c.compact()
    m.compact()
    same(c, m)
    assert torch.equal(c.k_pages, moved(k0, m.moves, "NHD"))


@pytest.mark.gpu
def test_captured_and_replayed_with_other_lists():
    c = cache_of(make(64, 16, 2, 64, 8, 8), 2)
    c.reset()
    m = host(c)
    rows, add, ws = i32(0, 1), i32(5, 40), torch.empty(c.pages_workspace_bytes(), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.extend(rows, add, workspace=ws)
    for r, a in (((0, 1), (5, 40)), ((2, 0), (17, 12)), ((3, 1), (0, 1))):
        rows.copy_(i32(*r))
        add.copy_(i32(*a))
        g.replay()
        m.extend(r, a)
        same(c, m)


@pytest.mark.gpu
def test_empty_lists_and_another_stream():
    c = cache_of(make(8, 16, 1, 64, 3, 4), 1)
    c.reset()
    c.free(i32())
    c.extend(i32(), i32())
    c.fork(i32(), i32())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rows, add = i32(1), i32(30)
    with torch.cuda.stream(s):
        c.extend(rows, add)
    s.synchronize()
    assert c.seq_len.tolist() == [0, 30, 0]


def test_refusals_on_the_host():
    from long_context_grpo_gb300 import build
    build.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    base = dict(num_pages=8, page_size=16, Hq=4, Hkv=2, D=64, layout=0, softmax_scale=0.0, page_stride=16 * 128,
                k_pages=0x1000, v_pages=0x2000, num_rows=3, table_width=4, page_table=0x3000, seq_len=0x4000, refcount=0x5000)
    h = ctypes.c_void_p()
    make_ = lambda **kw: L.ls_cache_create(ctypes.byref(b.CacheDesc(**{**base, **kw})), ctypes.byref(h))  # noqa: E731
    assert L.ls_cache_create(None, ctypes.byref(h)) == 1
    for kw in (dict(k_pages=None), dict(refcount=None), dict(num_pages=0), dict(num_rows=0), dict(table_width=0), dict(Hkv=0),
               dict(layout=2), dict(softmax_scale=-1.0), dict(page_stride=2047)):
        assert make_(**kw) == 1, kw
    for kw in (dict(D=96), dict(Hq=3), dict(Hq=34), dict(page_size=8), dict(page_size=48), dict(page_size=512),
               dict(num_pages=1 << 31), dict(table_width=1 << 28)):
        assert make_(**kw) == 2, kw
    assert make_(page_stride=2052) == 4 and make_(k_pages=0x1008) == 4 and make_(page_table=0x3002) == 4
    assert h.value is None
    # calls without a handle
    assert L.ls_cache_reset(None, None) == 3 and L.ls_cache_extend(None, 1, 0x10, 0x10, 0x100, 1 << 20, None) == 3
    assert L.ls_cache_fork(None, 1, 0x10, 0x10, 0x100, 1 << 20, None) == 3 and L.ls_cache_free(None, 1, 0x10, None) == 3
    assert L.ls_cache_compact(None, None, None, 0x100, 1 << 20, None) == 3
    assert L.ls_cache_append(None, None, None) == 3 and L.ls_cache_attn(None, None, None, 0, None) == 3
    assert L.ls_cache_pages_workspace_bytes(None) == 0 and L.ls_cache_attn_workspace_bytes(None, 1, 1, 1, 1) == 0
    assert L.ls_cache_destroy(None) == 0


@pytest.mark.gpu
def test_refusals_of_a_live_handle():
    import long_context_grpo_gb300 as ls
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    c = cache_of(make(8, 16, 2, 64, 3, 4), 4)
    ws = c.pages_workspace_bytes()
    assert L.ls_cache_extend(c._h, 1025, 0x100, 0x100, 0x1000, ws, None) == 2
    assert L.ls_cache_extend(c._h, -1, 0x100, 0x100, 0x1000, ws, None) == 1
    assert L.ls_cache_extend(c._h, 1, None, 0x100, 0x1000, ws, None) == 1
    assert L.ls_cache_extend(c._h, 1, 0x102, 0x100, 0x1000, ws, None) == 4
    assert L.ls_cache_extend(c._h, 1, 0x100, 0x100, 0x1000, ws - 256, None) == 8
    assert L.ls_cache_fork(c._h, 1, 0x100, 0x100, 0x1008, ws, None) == 4
    assert L.ls_cache_free(c._h, 1025, 0x100, None) == 2
    for other in (make(8, 32, 2, 64, 3, 4), make(8, 16, 2, 64, 4, 4), make(8, 16, 2, 64, 3, 5), make(8, 16, 1, 64, 3, 4)):
        d = cache_of(other, 4)
        assert L.ls_cache_compact(c._h, d._h, None, 0x1000, ws, None) == 2
    twin = ls.PagedCache(c.k_pages, c.v_pages, c.page_table, c.seq_len, c.refcount, Hq=4)
    assert L.ls_cache_compact(c._h, twin._h, None, 0x1000, ws, None) == 1
    base = dict(S=1, T=2, cu_new=0x100, k_new=0x200, k_stride=128, v_new=0x300, v_stride=128)
    ap = lambda **kw: L.ls_cache_append(c._h, ctypes.byref(b.CacheAppendDesc(**{**base, **kw})), None)  # noqa: E731
    for kw in (dict(S=0), dict(T=0), dict(cu_new=None), dict(v_new=None), dict(k_stride=127), dict(q=0x400, q_out=0x500)):
        assert ap(**kw) == 1, kw
    assert ap(S=2049) == 2 and ap(k_new=0x201) == 4
    base2 = dict(S=2, T=2, cu_new=0x100, max_new=1, max_len=9, q=0x1000, q_stride=256, o=0x2000, lse=0x3000, group=1)
    at = lambda wsb=1 << 30, **kw: L.ls_cache_attn(c._h, ctypes.byref(b.CacheAttnDesc(**{**base2, **kw})), 0x10000, wsb, None)  # noqa: E731
    for kw in (dict(S=0), dict(T=0), dict(max_new=0), dict(max_len=0), dict(group=0), dict(group=2), dict(S=3, group=2, shared_len=0x100),
               dict(q=None), dict(lse=None), dict(q_stride=255)):
        assert at(**kw) == 1, kw
    assert at(S=2049) == 2 and at(q=0x1008) == 4 and at(q_stride=260) == 4 and at(wsb=0) == 8
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_a_list_that_asks_for_more_than_2_31_pages():
    """17 rows that each ask for all their 2^27 - 1 table columns: none fits, nothing changes; a row that fits
    before them is served."""
    import long_context_grpo_gb300 as ls
    width, rows, ps = (1 << 27) - 1, 18, 16
    k = torch.zeros(40, 2, ps, 1, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    c = ls.PagedCache(k[:, 0], k[:, 1], table, torch.zeros(rows, dtype=torch.int32, device="cuda"),
                      torch.zeros(40, dtype=torch.int32, device="cuda"), Hq=1)
    c.extend(torch.arange(rows, dtype=torch.int32, device="cuda"),
             torch.tensor([20] + [width * ps] * (rows - 1), dtype=torch.int32, device="cuda"))
    assert ls.device_status() == (7, 4)
    assert c.seq_len.tolist() == [20] + [0] * (rows - 1) and int(c.refcount.sum()) == 2
    assert table[0, :3].tolist() == [0, 1, -1] and int(table[1:, :64].max()) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("rows,spread", [(1024, 1), (3000, 1), (70000, 17), (1024 * 64, 64)])
def test_lists_of_1024_entries_with_rows_listed_again(rows, spread):
    """Every position of the longest list: later entries of a row are left out, wherever they stand."""
    import long_context_grpo_gb300 as ls
    rng = np.random.default_rng(rows)
    c = cache_of(make(4000, 16, 1, 64, rows, 3), 1)
    c.reset()
    m = host(c)
    some = rng.permutation(rows // spread)[:700] * spread        # (rows that fall into few slots of a table too)
    lst = np.concatenate([some[:500], rng.choice(some, 524)])
    rng.shuffle(lst)
    add = rng.integers(0, 49, 1024)
    c.extend(i32(*lst), i32(*add))
    m.extend(lst, add)
    assert ls.device_status() == (7, 2)
    same(c, m)
    empty = np.nonzero(m.len == 0)[0]
    kids = rng.choice(empty[:600], 1024)
    full = np.nonzero(m.len > 0)[0]
    parents = rng.choice(full, 1024)
    c.fork(i32(*parents), i32(*kids))
    m.fork(parents, kids)
    assert ls.device_status() == (7, 2)
    same(c, m)


@pytest.mark.gpu
def test_a_row_that_grows_within_its_page_needs_none():
    """Behind an entry that went without pages, an entry that needs none is done."""
    import long_context_grpo_gb300 as ls
    c = cache_of(make(4, 16, 1, 64, 4, 4), 1)
    c.reset()
    m = host(c)
    for rows, add, bits in (((0, 1), (20, 5), 0), ((2, 0, 1, 3), (40, 12, 11, 0), 4), ((1, 2, 0), (1, 16, 0), 4), ((3, 2), (1, 0), 4)):
        c.extend(i32(*rows), i32(*add))
        m.extend(rows, add)
        same(c, m)
        assert ls.device_status() == ((7, bits) if bits else (0, 0)), rows
    assert c.seq_len.tolist() == [32, 17, 0, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("into", [False, True])
def test_compaction_judges_the_listed_pages(into):
    """What a table holds behind a row's length is not listed (it becomes -1); a page outside the pool within
    the length, on either side, and a length outside the table are reported."""
    import long_context_grpo_gb300 as ls
    for page, column, length, bits in ((1 << 30, 2, 20, 0), (6, 2, 32, 0), (-5, 2, 20, 0), (-1, 1, 20, 2), (-9, 0, 1, 2), (6, 1, 17, 2),
                                       (1 << 30, 2, 33, 2), (-1, 2, 33, 2), (-1, 2, 49, 2), (-1, 2, -1, 2), (-1, 2, 1 << 30, 2)):
        k, v, table, length_, ref = make(6, 16, 2, 64, 3, 3)
        table.copy_(torch.tensor([[1, 4, -1], [5, 3, -1], [-1, -1, -1]], dtype=torch.int32))
        table[1, column] = page
        length_.copy_(i32(30, length, 0))
        ref.zero_()
        pages = [1, 4] + [p for p in table[1].tolist() if 0 <= p < 6]
        ref[pages] = 1
        c = cache_of((k, v, table, length_, ref), 2)
        d = cache_of(make(6, 16, 2, 64, 3, 3), 2) if into else c
        m = host(c)
        k0 = k.clone()
        c.compact(into=d if into else None)
        assert ls.device_status() == ((7, bits) if bits else (0, 0)), (page, column, length)
        live = [p for p in range(6) if m.ref[p]]
        assert d.refcount.tolist() == [1] * len(live) + [0] * (6 - len(live))
        want, got = m.table, d.page_table.cpu().numpy()
        for r in range(3):
            for j in range(3):
                p = int(want[r, j])
                assert (got[r, j] == -1) if not 0 <= p < 6 else torch.equal(d.k_pages[int(got[r, j])], k0[p])
        assert torch.equal(d.seq_len, c.seq_len)
