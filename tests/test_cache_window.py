"""Attention over the paged cache through a sliding window with the first tokens in sight, against float64.

Tolerance of o as in test_cache_attn.py: the probabilities are rounded to bf16 once (2^-8 of each, so 2^-8
of sum p |v|), o itself once (2^-8 of it); scores and sums are fp32 (2^-14 of sum p |v| covers exponents up to
2^8)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.cache import attend, sequence
from test_cache_attn import SHAPES, build, cu


def check(cache, table, lens, n_new, q, o, lse, layout, window, sinks, rows=None, cu0=0):
    at = cu0
    for b, n in enumerate(n_new):
        r = b if rows is None else rows[b]
        # pages out of sight may be listed as anything
        row = np.where(np.asarray(table[r]) < 0, 0, table[r])
        k, v = (sequence(x, row, lens[r], layout) for x in (cache.k_pages, cache.v_pages))
        qo = q[at:at + n].double().cpu().numpy()
        with np.errstate(invalid="ignore"):      # (keys that nobody sees may hold NaN)
            wo, wl, wa = attend(qo, k, v, cache.D ** -0.5, window, sinks)
        go, gl = o[at:at + n].double().cpu().numpy(), lse[at:at + n].double().cpu().numpy()
        none = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), none)
        assert (go[none] == 0).all()
        assert (np.abs(go - wo) <= 2 ** -8 * (np.abs(wo) + wa) + 2 ** -14 * wa + 1e-30).all(), (b, np.abs(go - wo).max())
        assert (np.abs(gl[~none] - wl[~none]) <= 2 ** -20 * np.abs(wl[~none]) + 2e-5).all()
        at += n


KINDS = {"token": ([1] * 9, [1, 2, 15, 16, 17, 127, 128, 129, 700]), "few": ([2, 3, 1, 4], [2, 130, 1, 1021]),
         "chunk": ([130, 65], [130, 800]), "mixed": ([0, 1, 37, 0, 200, 5], [40, 513, 37, 0, 333, 5])}


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,ps,layout", SHAPES)
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (128, 130), (300, 0), (5000, 7)])
def test_against_float64(Hq, Hkv, D, ps, layout, kind, window, sinks):
    import long_context_grpo_gb300 as ls
    n, lens = KINDS[kind]
    make, table = build(lens, ps, Hkv, D, layout, seed=Hq + D, junk=float("nan"))
    c = make(Hq)
    T = sum(n)
    q = torch.randn(T, Hq, D, device="cuda").to(torch.bfloat16)
    o, lse = c.attn(q, cu(n), max_new=max(n), max_len=max(lens), window=window, sinks=sinks)
    check(c, table, lens, n, q, o, lse, layout, window, sinks)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("S,n,L", [(1, 1, 20000), (1, 3, 9999), (3, 1, 6001), (1, 50, 5000), (2, 260, 5000), (40, 2, 4500)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (4, 2, 64), (32, 8, 128)])
@pytest.mark.parametrize("window,sinks", [(1000, 4), (4096, 1), (2500, 700)])
def test_long_windows_split_and_joined(S, n, L, Hq, Hkv, D, window, sinks):
    import long_context_grpo_gb300 as ls
    lens = [L - 13 * b for b in range(S)]
    make, table = build(lens, 16, Hkv, D, seed=L, junk=float("inf"))
    c = make(Hq)
    q = (torch.randn(S * n, Hq, D, device="cuda") * 2).to(torch.bfloat16)
    sight = dict(window=window, sinks=sinks)
    a = c.attn(q, cu([n] * S), max_new=n, max_len=L, **sight)
    few = min(S, 4)
    check(c, table, lens[:few], [n] * few, q, *a, "NHD", window, sinks)
    # the same bits again, and under larger bounds (another split) the same values
    again = c.attn(q, cu([n] * S), max_new=n, max_len=L, **sight)
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1])
    wide = c.attn(q, cu([n] * S), max_new=4 * n, max_len=8 * L, **sight)
    check(c, table, lens[:few], [n] * few, q, *wide, "NHD", window, sinks)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 70])
@pytest.mark.parametrize("group", [1, 4])
def test_a_window_past_every_sequence_is_plain_attention(n, group):
    import long_context_grpo_gb300 as ls
    lens = [600 + 9 * b for b in range(4)]
    make, table = build(lens, 32, 2, 128, seed=n, shared=512, group=group)
    c = make(8)
    q = torch.randn(4 * n, 8, 128, device="cuda").to(torch.bfloat16)
    kw = dict(max_new=n, max_len=max(lens), group=group)
    if group > 1:
        kw["shared_len"] = torch.tensor([512], dtype=torch.int32, device="cuda")
    o, lse = c.attn(q, cu([n] * 4), **kw)
    for window, sinks in ((max(lens), 0), (1 << 40, 3), (1, max(lens)), (1, 1 << 50)):
        a, b = c.attn(q, cu([n] * 4), window=window, sinks=sinks, **kw)
        # twice the rounding of the probabilities (2^-8 of a weighted mean of |v|, below 1 here) and of o
        assert bool(((a.double() - o.double()).abs() <= 2 ** -7 + 2 ** -7 * o.double().abs()).all())
        assert torch.allclose(b, lse, atol=4e-5, rtol=2 ** -20)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("ps,layout", [(16, "NHD"), (64, "HND"), (256, "NHD")])
@pytest.mark.parametrize("n", [1, 5, 90])
@pytest.mark.parametrize("sinks", [0, 4, 300])
def test_pages_out_of_sight_are_not_looked_at(ps, layout, n, sinks):
    """Table entries before the window may be anything, and so may the keys and values out of sight in the
    pages at the window's edge."""
    import long_context_grpo_gb300 as ls
    L, window = 2900, 333
    make, table = build([L] * 2, ps, 2, 64, layout, seed=n)
    c = make(8)
    q = torch.randn(2 * n, 8, 64, device="cuda").to(torch.bfloat16)
    kw = dict(max_new=n, max_len=L, window=window, sinks=sinks)
    o, lse = c.attn(q, cu([n] * 2), **kw)
    lo = L - n - window + 1
    for junk in (-1, 1 << 30):
        c.page_table[:, -(-sinks // ps):lo // ps] = junk
        for t in range(lo // ps * ps, lo):
            if t >= sinks:
                for x in (c.k_pages, c.v_pages):
                    p = table[:, t // ps]
                    for page in p:
                        (x[page, t % ps] if layout == "NHD" else x[page, :, t % ps]).fill_(float("nan"))
        a, b = c.attn(q, cu([n] * 2), **kw)
        assert torch.equal(a, o) and torch.equal(b, lse)
    assert ls.device_status() == (0, 0)
    # one in sight is reported
    c.page_table[0, lo // ps] = -1
    c.attn(q, cu([n] * 2), **kw)
    assert ls.device_status() == (7, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 33])
def test_rows_strides_and_tokens_that_see_nothing(n):
    import long_context_grpo_gb300 as ls
    lens = [700, 0, max(0, n - 5), 129]
    make, table = build(lens, 32, 2, 128, seed=1, width=30)
    c = make(6)
    rows = [3, 0, 2, 1, 3]
    new = [n, n, n, n, 0]
    T = sum(new) + 7
    q = torch.randn(T, 10, 128, device="cuda").to(torch.bfloat16)[:, 2:8]
    o = torch.full((T, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 6), 7.0, device="cuda")
    c.attn(q, cu(new, 3), max_new=n, max_len=700, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"), o=o, lse=lse,
           window=50, sinks=2)
    check(c, table, lens, new, q, o, lse, "NHD", 50, 2, rows=rows, cu0=3)
    for a in (o, lse):
        assert (a[:3] == 7).all() and (a[T - 4:] == 7).all()
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_wild_rows_lengths_and_bounds_are_reported(n):
    import long_context_grpo_gb300 as ls
    make, table = build([200] * 3, 16, 1, 64, seed=2)
    c = make(4)
    q = torch.randn(3 * n, 4, 64, device="cuda").to(torch.bfloat16)
    call = lambda m=n, **kw: c.attn(q, cu([n] * 3), max_new=m, max_len=200, window=90, sinks=3, **kw)  # noqa: E731
    want = call()
    for rows in ([0, 3, 2], [0, -1, 2]):
        o, lse = call(rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
        assert ls.device_status() == (7, 2)
        assert not o[n:2 * n].any() and torch.isneginf(lse[n:2 * n]).all()
        for b in (0, 2):
            assert torch.equal(o[b * n:(b + 1) * n], want[0][b * n:(b + 1) * n])
    for length in (-3, 201, 1 << 30, -(1 << 31), (1 << 31) - 1):
        c.seq_len[1] = length
        o, lse = call()
        assert ls.device_status() == (7, 2)
        assert not o[n:2 * n].any() and torch.isneginf(lse[n:2 * n]).all()
        assert torch.equal(o[2 * n:], want[0][2 * n:])
    c.seq_len[1] = 200
    if n > 1:
        for m in (1, 16, n - 1):
            o, lse = call(m)
            assert ls.device_status() == (7, 2) and not o.any() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("max_new", [1, 40, 2560])
@pytest.mark.parametrize("offsets", ["falls", "saw", "negative", "past"])
def test_offsets_that_are_not_a_partition_are_refused(offsets, max_new):
    import long_context_grpo_gb300 as ls
    S, n, L = 64, 40, 300
    make, table = build([L] * S, 64, 2, 64, seed=5)
    c = make(8)
    T = S * n
    q = torch.randn(T, 8, 64, device="cuda").to(torch.bfloat16)
    at = {"falls": [n * b - (200 if b == 30 else 0) for b in range(S + 1)], "saw": [T * (b % 2) for b in range(S + 1)],
          "negative": [-1] + [n * b for b in range(1, S + 1)], "past": [n * b for b in range(S)] + [T + 1]}[offsets]
    o, lse = c.attn(q, torch.tensor(at, dtype=torch.int32, device="cuda"), max_new=max_new, max_len=L, window=64, sinks=4)
    assert ls.device_status() == (7, 2)
    own = torch.zeros(T, dtype=torch.bool, device="cuda")
    own[:n] = offsets in ("falls", "past")
    assert not o[own].any() and torch.isneginf(lse[own]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,L", [(1, 90), (3, 20000), (70, 300), (70, 9000)])
@pytest.mark.parametrize("where", ["query", "key", "out of sight"])
def test_a_poisoned_query_or_key_reaches_the_rows_that_see_it(where, n, L):
    import long_context_grpo_gb300 as ls
    window, sinks = 60, 2
    make, table = build([L] * 2, 64, 2, 128, seed=L)
    c = make(8)
    q = torch.randn(2 * n, 8, 128, device="cuda").to(torch.bfloat16)
    call = lambda: c.attn(q, cu([n] * 2), max_new=n, max_len=L, window=window, sinks=sinks)  # noqa: E731
    want = call()
    sees = torch.zeros(2 * n, 8, dtype=torch.bool, device="cuda")
    if where == "query":
        q[n // 2, 5, 17] = float("nan")
        sees[n // 2, 5] = True
    else:
        pos = L - n + n // 2 - 3 if where == "key" else L - n - window
        c.k_pages[int(table[0, pos // 64]), pos % 64, 1, 3] = float("nan")
        p = torch.arange(L - n, L)
        sees[:n, 4:] = ((p >= pos) & (p < pos + window))[:, None].cuda()
    o, lse = call()
    assert torch.isnan(o[sees]).all() and torch.isnan(lse[sees]).all()
    assert torch.equal(o[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees])


@pytest.mark.gpu
def test_captured_decode_through_a_window():
    """One graph of extend, append and attention replayed for every new token; a workspace that held other
    things, shared with a second stream's eager call in between."""
    import long_context_grpo_gb300 as ls
    S, Hq, Hkv, D, ps = 3, 8, 2, 64, 16
    lens = [5, 0, 130]
    make, _ = build(lens, ps, Hkv, D, seed=6, width=20, spare=30)
    c = make(Hq)
    rows = torch.arange(S, dtype=torch.int32, device="cuda")
    one, cu1 = torch.ones(S, dtype=torch.int32, device="cuda"), cu([1] * S)
    q, k, v = (torch.zeros(S, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    pw = torch.empty(c.pages_workspace_bytes(), dtype=torch.uint8, device="cuda")
    aw = torch.empty(c.attn_workspace_bytes(S, S, 1, 320, window=40, sinks=3), dtype=torch.uint8, device="cuda")
    keep = [t.clone() for t in (c.seq_len, c.page_table, c.refcount)]

    def step():
        c.extend(rows, one, workspace=pw)
        c.append(k, v, cu1)
        return c.attn(q, cu1, max_new=1, max_len=320, workspace=aw, window=40, sinks=3)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = step()
    for a, b in zip((c.seq_len, c.page_table, c.refcount), keep):
        a.copy_(b)
    for i in range(60):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda").to(torch.bfloat16))
        aw.fill_(0xFF)
        g.replay()
        now = [n + i + 1 for n in lens]
        if i % 13 == 0 or i == 59:
            check(c, c.page_table.cpu().numpy(), now, [1] * S, q, o, lse, "NHD", 40, 3)
    assert ls.device_status() == (0, 0)


def test_refusals():
    from long_context_grpo_gb300 import build as lsbuild
    lsbuild.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    assert L.ls_cache_attn_window(None, ctypes.byref(b.CacheAttnDesc()), 4, 0, 0x1000, 1 << 20, None) == 3
    assert L.ls_cache_attn_window_workspace_bytes(None, 1, 1, 1, 1, 1, 0) == 0


@pytest.mark.gpu
def test_refusals_with_a_handle():
    import long_context_grpo_gb300 as ls
    make, _ = build([100], 16, 2, 64)
    c = make(4)
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    kw = dict(max_new=1, max_len=100)
    for window, sinks, status in ((0, 0, 1), (-1, 0, 1), (4, -1, 1)):
        assert c.attn_workspace_bytes(1, 1, 1, 100, window=window, sinks=sinks) == 0
        with pytest.raises(ls.LongStrawError) as e:
            c.attn(q, cu([1]), window=window, sinks=sinks, **kw)
        assert e.value.status == status
    with pytest.raises(ValueError):
        c.attn(q, cu([1]), sinks=4, **kw)
    need = c.attn_workspace_bytes(1, 1, 1, 100, window=9)
    with pytest.raises(ls.LongStrawError) as e:
        c.attn(q, cu([1]), window=9, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"), **kw)
    assert e.value.status == 8
