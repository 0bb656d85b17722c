"""Append to and attention over the paged cache against float64, sequence by sequence.

Tolerance of o: the probabilities are rounded to bf16 once (2^-8 of each, so 2^-8 of sum p |v|), o
itself once (2^-8 of it); scores and sums are fp32 (2^-14 of sum p |v| covers exponents up to 2^8)."""
import numpy as np
import pytest
import torch

from oracle.cache import attend, sequence
from oracle.rope import rope as ref_rope


def build(lens, ps, Hkv, D, layout="NHD", seed=0, shared=None, group=1, spare=3, junk=None, width=None):
    """A cache whose rows have these lengths over shuffled pages; `group` rows share `shared` tokens."""
    import long_context_grpo_gb300 as ls
    rng = np.random.default_rng(seed)
    need = [-(-max(n, 0) // ps) for n in lens]
    keep = 0 if shared is None else shared // ps
    total = sum(need) + spare
    order = list(rng.permutation(total))
    table = np.full((len(lens), width or max(need + [1])), -1, dtype=np.int32)
    for b, n in enumerate(need):
        lead = keep if group > 1 and b % group else 0
        table[b, :lead] = table[b - b % group, :lead]
        for j in range(lead, n):
            table[b, j] = order.pop()
    ref = np.bincount(table[table >= 0].ravel(), minlength=total).astype(np.int32)
    g = torch.Generator(device="cuda").manual_seed(seed)
    inner = (ps, Hkv, D) if layout == "NHD" else (Hkv, ps, D)
    both = torch.randn(total, 2, *inner, generator=g, device="cuda").to(torch.bfloat16)
    k, v = both[:, 0], both[:, 1]
    if junk is not None:            # what lies behind a sequence's end, and in pages that no row lists
        used = torch.zeros(total, ps, dtype=torch.bool)
        for b, n in enumerate(lens):
            for j in range(need[b]):
                used[table[b, j], :max(0, min(ps, n - j * ps))] = True
        mask = ~used.cuda()[:, :, None, None] if layout == "NHD" else ~used.cuda()[:, None, :, None]
        both.masked_fill_(mask[:, None], junk)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return (lambda Hq, **kw: ls.PagedCache(k, v, dev(table), dev(np.array(lens, dtype=np.int32)), dev(ref), Hq=Hq,
                                           layout=layout, **kw)), table


def check(cache, table, lens, n_new, q, o, lse, layout, rows=None, scale=None, cu0=0):
    at = cu0
    scale = cache.D ** -0.5 if scale is None else scale
    K, V = cache.k_pages, cache.v_pages
    for b, n in enumerate(n_new):
        r = b if rows is None else rows[b]
        k = sequence(K, table[r], lens[r], layout)
        v = sequence(V, table[r], lens[r], layout)
        qo = q[at:at + n].double().cpu().numpy()
        wo, wl, wa = attend(qo, k, v, scale)
        go, gl = o[at:at + n].double().cpu().numpy(), lse[at:at + n].double().cpu().numpy()
        none = np.isneginf(wl)
        assert np.array_equal(np.isneginf(gl), none)
        assert (go[none] == 0).all()
        assert (np.abs(go - wo) <= 2 ** -8 * (np.abs(wo) + wa) + 2 ** -14 * wa + 1e-30).all(), (b, np.abs(go - wo).max())
        assert (np.abs(gl[~none] - wl[~none]) <= 2 ** -20 * np.abs(wl[~none]) + 2e-5).all()
        at += n


def cu(n, start=0):
    return torch.tensor([start] + list(start + np.cumsum(n)), dtype=torch.int32, device="cuda")


SHAPES = [  # Hq, Hkv, D, page, layout
    (2, 2, 64, 16, "NHD"), (8, 2, 128, 64, "HND"), (5, 1, 128, 32, "NHD"), (16, 1, 64, 128, "HND"), (24, 3, 128, 256, "NHD"),
    (40, 8, 128, 128, "NHD"), (13, 1, 128, 16, "HND"), (7, 7, 64, 64, "NHD")]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,ps,layout", SHAPES)
@pytest.mark.parametrize("kind", ["token", "few", "chunk", "mixed"])
def test_against_float64(Hq, Hkv, D, ps, layout, kind):
    import long_context_grpo_gb300 as ls
    n, lens = {"token": ([1] * 9, [1, 2, 15, 16, 17, 127, 128, 129, 700]),
               "few": ([2, 3, 1, 4], [2, 130, 1, 1021]),
               "chunk": ([130, 65], [130, 800]),
               "mixed": ([0, 1, 37, 0, 200, 5], [40, 513, 37, 0, 333, 5])}[kind]
    make, table = build(lens, ps, Hkv, D, layout, seed=Hq + D, junk=float("nan"))
    c = make(Hq)
    T = sum(n)
    q = torch.randn(T, Hq, D, device="cuda").to(torch.bfloat16)
    o, lse = c.attn(q, cu(n), max_new=max(n), max_len=max(lens))
    check(c, table, lens, n, q, o, lse, layout)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("S,n,L", [(1, 1, 20000), (1, 3, 9999), (3, 1, 6001), (1, 50, 5000), (2, 260, 3000)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (4, 2, 64), (32, 8, 128)])
def test_long_sequences_split_and_joined(S, n, L, Hq, Hkv, D):
    import long_context_grpo_gb300 as ls
    lens = [L - 13 * b for b in range(S)]
    make, table = build(lens, 64, Hkv, D, seed=L, junk=float("inf"))
    c = make(Hq)
    q = (torch.randn(S * n, Hq, D, device="cuda") * 2).to(torch.bfloat16)
    a = c.attn(q, cu([n] * S), max_new=n, max_len=L)
    check(c, table, lens, [n] * S, q, *a, "NHD")
    # the same bits again, and under larger bounds (another split) the same values
    again = c.attn(q, cu([n] * S), max_new=n, max_len=L)
    assert torch.equal(a[0], again[0]) and torch.equal(a[1], again[1])
    wide = c.attn(q, cu([n] * S), max_new=4 * n, max_len=8 * L)
    check(c, table, lens, [n] * S, q, *wide, "NHD")
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,ps", [(8, 2, 128, 64), (4, 4, 64, 16), (32, 8, 128, 128), (16, 1, 128, 32)])
@pytest.mark.parametrize("group,n,shared", [(2, 1, 512), (4, 1, 1000), (8, 1, 2048), (4, 3, 640), (2, 40, 1280), (3, 1, 0), (4, 2, 100)])
def test_groups_that_share_their_first_pages(Hq, Hkv, D, ps, group, n, shared):
    """Any shared length (whole pages are shared below it), ragged tails, a second group with another length."""
    import long_context_grpo_gb300 as ls
    S = 2 * group
    lens = [shared + n + 1 + (37 * b) % 200 for b in range(S)]
    make, table = build(lens, ps, Hkv, D, seed=group + n, shared=shared // ps * ps, group=group, junk=float("nan"))
    c = make(Hq)
    new = [n if b != 1 else max(1, n - 1) for b in range(S)]
    q = torch.randn(sum(new), Hq, D, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([shared // ps * ps, shared // ps * ps // 2], dtype=torch.int32, device="cuda")
    o, lse = c.attn(q, cu(new), max_new=n, max_len=max(lens), group=group, shared_len=sl)
    check(c, table, lens, new, q, o, lse, "NHD")
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_a_group_with_tokens_inside_the_shared_part():
    """New tokens whose positions lie before the end of the shared pages see only their own past."""
    import long_context_grpo_gb300 as ls
    lens, n = [300, 300, 290, 64], [20, 1, 5, 3]
    make, table = build(lens, 16, 2, 64, seed=3, shared=64, group=4)
    c = make(4)
    q = torch.randn(sum(n), 4, 64, device="cuda").to(torch.bfloat16)
    o, lse = c.attn(q, cu(n), max_new=20, max_len=300, group=4, shared_len=torch.tensor([64], dtype=torch.int32, device="cuda"))
    check(c, table, lens, n, q, o, lse, "NHD")
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,L", [(1, 90), (120, 700), (2, 9000)])
@pytest.mark.parametrize("skip", [8, 16, 24])
def test_output_on_any_16_byte_boundary(D, n, L, skip):
    """`o` inside a larger tensor: the same bits, and nothing beside it is written."""
    make, table = build([L] * 3, 64, 2, D, seed=L)
    c = make(8)
    q = torch.randn(3 * n, 8, D, device="cuda").to(torch.bfloat16)
    want, lse = c.attn(q, cu([n] * 3), max_new=n, max_len=L)
    check(c, table, [L] * 3, [n] * 3, q, want, lse, "NHD")
    room = torch.full((want.numel() + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    o = room[skip:skip + want.numel()].view(want.shape)
    c.attn(q, cu([n] * 3), max_new=n, max_len=L, o=o)
    assert torch.equal(o, want)
    assert bool((room[:skip] == 7).all()) and bool((room[skip + want.numel():] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 33])
def test_rows_scale_strides_and_tokens_that_see_nothing(n):
    """Rows in any order and twice, q rows of a wider tensor, packed rows that no entry owns, a length below
    the number of new tokens (the first ones see nothing), a length of zero."""
    import long_context_grpo_gb300 as ls
    lens = [700, 0, max(0, n - 5), 129]
    make, table = build(lens, 32, 2, 128, seed=1, width=30)
    c = make(6, softmax_scale=0.3)
    rows = [3, 0, 2, 1, 3]
    new = [n, n, n, n, 0]
    T = sum(new) + 7
    wide = torch.randn(T, 10, 128, device="cuda").to(torch.bfloat16)
    q = wide[:, 2:8]
    o = torch.full((T, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 6), 7.0, device="cuda")
    c.attn(q, cu(new, 3), max_new=n, max_len=700, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"), o=o, lse=lse)
    check(c, table, lens, new, q, o, lse, "NHD", rows=rows, scale=0.3, cu0=3)
    for a in (o, lse):
        assert (a[:3] == 7).all() and (a[T - 4:] == 7).all()
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40])
def test_wild_rows_lengths_and_pages_are_reported(n):
    import long_context_grpo_gb300 as ls
    lens = [200, 200, 200]
    make, table = build(lens, 16, 1, 64, seed=2)
    c = make(4)
    q = torch.randn(3 * n, 4, 64, device="cuda").to(torch.bfloat16)
    want = c.attn(q, cu([n] * 3), max_new=n, max_len=200)
    for rows in ([0, 3, 2], [0, -1, 2]):
        o, lse = c.attn(q, cu([n] * 3), max_new=n, max_len=200, rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
        assert ls.device_status() == (7, 2)
        assert not o[n:2 * n].any() and torch.isneginf(lse[n:2 * n]).all()
        for b in (0, 2):
            assert torch.equal(o[b * n:(b + 1) * n], want[0][b * n:(b + 1) * n])
    for length in (-3, 201, 1 << 30):
        c.seq_len[1] = length
        o, lse = c.attn(q, cu([n] * 3), max_new=n, max_len=200)
        assert ls.device_status() == (7, 2)
        assert not o[n:2 * n].any() and torch.isneginf(lse[n:2 * n]).all()
        assert torch.equal(o[2 * n:], want[0][2 * n:])
    c.seq_len[1] = 200
    # a page outside the pool counts as zeros
    page = int(c.page_table[1, 4])
    zk, zv = c.k_pages[page].clone(), c.v_pages[page].clone()
    c.k_pages[page], c.v_pages[page] = 0, 0
    zero = c.attn(q, cu([n] * 3), max_new=n, max_len=200)
    c.k_pages[page], c.v_pages[page] = zk, zv
    assert ls.device_status() == (0, 0)
    for wild in (-1, 1 << 30, c.num_pages):
        c.page_table[1, 4] = wild
        o, lse = c.attn(q, cu([n] * 3), max_new=n, max_len=200)
        assert ls.device_status() == (7, 2)
        assert torch.equal(o, zero[0]) and torch.equal(lse, zero[1])
    # more new tokens than the bound: that entry is left out
    c.page_table[1, 4] = page
    if n > 1:
        o, lse = c.attn(q, cu([n, n, n]), max_new=n - 1, max_len=200)
        assert ls.device_status() == (7, 2) and not o.any() and torch.isneginf(lse).all()


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 4])
@pytest.mark.parametrize("offsets", ["falls", "saw", "negative", "past"])
def test_offsets_that_are_not_a_partition_are_refused(offsets, group):
    """Runs that overlap would make more jobs than the workspace's lists hold: no entry is done."""
    import long_context_grpo_gb300 as ls
    S, n, L = 64, 40, 300
    make, table = build([L] * S, 64, 2, 64, seed=5)
    c = make(8)
    T = S * n
    q = torch.randn(T, 8, 64, device="cuda").to(torch.bfloat16)
    at = {"falls": [n * b - (200 if b == 30 else 0) for b in range(S + 1)], "saw": [T * (b % 2) for b in range(S + 1)],
          "negative": [-1] + [n * b for b in range(1, S + 1)], "past": [n * b for b in range(S)] + [T + 1]}[offsets]
    at = torch.tensor(at, dtype=torch.int32, device="cuda")
    sl = torch.full((S // group,), 64, dtype=torch.int32, device="cuda") if group > 1 else None
    o, lse = c.attn(q, at, max_new=T, max_len=L, group=group, shared_len=sl)
    assert ls.device_status() == (7, 2)
    own = torch.zeros(T, dtype=torch.bool, device="cuda")
    own[:n] = offsets in ("falls", "past")
    assert not o[own].any() and torch.isneginf(lse[own]).all()
    want = c.attn(q, cu([n] * S), max_new=n, max_len=L)
    check(c, table, [L] * S, [n] * S, q, *want, "NHD")
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_far_pages_of_a_large_pool():
    """Element offsets past 2^32: the last pages of a 9 GB pool."""
    import long_context_grpo_gb300 as ls
    N, ps, Hkv, D = 18000, 256, 4, 128
    both = torch.zeros(N, 2, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pages = [N - 1, N - 2, 3]
    both[pages] = torch.randn(3, 2, ps, Hkv, D, device="cuda").to(torch.bfloat16)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i(pages, [N - 3, -1, -1])
    c = ls.PagedCache(both[:, 0], both[:, 1], table, i(700, 0), torch.zeros(N, dtype=torch.int32, device="cuda"), Hq=8)
    for n in (1, 70):
        q = torch.randn(n, 8, D, device="cuda").to(torch.bfloat16)
        o, lse = c.attn(q, cu([n]), max_new=n, max_len=700)
        check(c, table.cpu().numpy(), [700], [n], q, o, lse, "NHD")
    c.seq_len[1] = 256
    k, v = (torch.randn(256, Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    c.append(k, v, cu([256]), rows=i(1))
    assert torch.equal(both[N - 3, 0], k) and torch.equal(both[N - 3, 1], v)
    c.refcount[N - 3] = 1
    c.fork(i(), i())
    c.compact()
    assert torch.equal(both[0, 0], k) and c.page_table[1, 0] == 0
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("layout,ps", [("NHD", 16), ("HND", 32), ("NHD", 256), ("HND", 128)])
@pytest.mark.parametrize("n", [1, 90])
def test_pages_apart_from_one_another(layout, ps, n):
    """A page stride that is no multiple of the page or its rows: the gaps are left as they were."""
    import long_context_grpo_gb300 as ls
    Hkv, D, N = 3, 64, 40
    size = ps * Hkv * D
    inner = (ps, Hkv, D) if layout == "NHD" else (Hkv, ps, D)
    raw = [torch.full((N, size + 8), 9.0, device="cuda").to(torch.bfloat16) for _ in range(2)]
    k, v = (x[:, :size].unflatten(1, inner) for x in raw)
    k.copy_(torch.randn(k.shape, device="cuda"))
    v.copy_(torch.randn(v.shape, device="cuda"))
    L = 2 * ps + 130
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    width = -(-L // ps)
    table = torch.from_numpy(np.random.default_rng(ps).permutation(N)[:2 * width].reshape(2, width).astype(np.int32)).cuda()
    ref = torch.bincount(table.flatten().long(), minlength=N).int()
    c = ls.PagedCache(k, v, table, i32(L, L - 7), ref, Hq=6, layout=layout)
    kn, vn = (torch.randn(2 * n, Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    c.append(kn, vn, cu([n, n]))
    q = torch.randn(2 * n, 6, D, device="cuda").to(torch.bfloat16)
    o, lse = c.attn(q, cu([n, n]), max_new=n, max_len=L)
    check(c, table.cpu().numpy(), [L, L - 7], [n, n], q, o, lse, layout)
    before = [sequence(x, table[0].cpu().numpy(), L, layout) for x in (k, v)]
    c.compact()
    for x, y in zip((k, v), before):
        assert np.array_equal(sequence(x, c.page_table[0].cpu().numpy(), L, layout), y)
    assert all((x[:, size:] == 9).all() for x in raw)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("layout,ps", [("NHD", 16), ("HND", 64), ("NHD", 256)])
@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (20, False), (None, False)])
def test_append_with_and_without_rotation(layout, ps, rot, inter):
    import long_context_grpo_gb300 as ls
    lens, new = [5, 400, 0, 77, 260], [5, 130, 0, 3, 1]
    make, table = build(lens, ps, 2, 128, layout, seed=4, width=30)
    c = make(6)
    T = sum(new) + 2
    k, v = (torch.randn(T, 2, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, 6, 128, device="cuda").to(torch.bfloat16)
    before = c.k_pages.clone(), c.v_pages.clone()
    f, a = ls.rope_freqs(rot, 1e4) if rot else (None, 1.0)
    q_out = torch.full_like(q, 7.0)
    if rot:
        c.append(k, v, cu(new, 1), q=q, q_out=q_out, inv_freq=f, interleaved=inter, attn_factor=a)
    else:
        assert c.append(k, v, cu(new, 1)) == (None, None)
    assert ls.device_status() == (0, 0)
    want_k, want_v = before
    at = 1
    for b, n in enumerate(new):
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")
        kb = k[at:at + n]
        if rot and n:
            qb, kb = ls.rope(q[at:at + n], kb, f, positions=pos, interleaved=inter)
            assert torch.equal(q_out[at:at + n], qb)
            want = ref_rope(k[at:at + n].double().cpu().numpy(), pos.cpu().numpy(), f.numpy(), inter)
            assert (np.abs(kb.double().cpu().numpy() - want) <= 2 ** -8 * np.abs(want) + 2 ** -18).all()
        for i in range(n):
            p, s = int(table[b, int(pos[i]) // ps]), int(pos[i]) % ps
            sl = (p, s) if layout == "NHD" else (p, slice(None), s)
            want_k[sl], want_v[sl] = kb[i], v[at + i]
        at += n
    assert torch.equal(c.k_pages, want_k) and torch.equal(c.v_pages, want_v)
    assert (q_out[0] == 7).all() and (q_out[T - 1] == 7).all()


@pytest.mark.gpu
def test_append_leaves_out_what_has_no_place():
    import long_context_grpo_gb300 as ls
    make, table = build([3, 40, 20], 16, 1, 64, seed=5, width=4)
    c = make(1)
    before = c.k_pages.clone()
    k, v = (torch.randn(9, 1, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    # five new tokens of a length of three: two are left out
    c.append(k[:5], v[:5], cu([5]))
    before[table[0, 0], :3] = k[2:5]
    assert torch.equal(c.k_pages, before) and ls.device_status() == (0, 0)
    for wild in (1 << 30, -1):
        c.page_table[1, 2] = wild
        c.append(k, v, cu([9]), rows=torch.tensor([1], dtype=torch.int32, device="cuda"))
        before[table[1, 1], 15:] = k[:1]
        assert torch.equal(c.k_pages, before) and ls.device_status() == (7, 2)
    c.append(k, v, cu([9]), rows=torch.tensor([3], dtype=torch.int32, device="cuda"))
    assert torch.equal(c.k_pages, before) and ls.device_status() == (7, 2)


@pytest.mark.gpu
def test_captured_decode_replayed_as_the_sequences_grow():
    """One graph of extend, append and attention, replayed for every new token; two graphs share the
    workspaces; a second stream runs the eager calls."""
    import long_context_grpo_gb300 as ls
    S, Hq, Hkv, D, ps = 3, 8, 2, 64, 16
    lens = [5, 0, 130]
    make, table = build(lens, ps, Hkv, D, seed=6, width=20, spare=30)
    c = make(Hq)
    rows = torch.arange(S, dtype=torch.int32, device="cuda")
    one, cu1 = torch.ones(S, dtype=torch.int32, device="cuda"), cu([1] * S)
    f, _ = ls.rope_freqs(D, 1e4)
    q, k, v = (torch.zeros(S, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    qr = torch.empty_like(q)
    pw = torch.empty(c.pages_workspace_bytes(), dtype=torch.uint8, device="cuda")
    aw = torch.empty(c.attn_workspace_bytes(S, S, 1, 320), dtype=torch.uint8, device="cuda")
    keep = [t.clone() for t in (c.seq_len, c.page_table, c.refcount, c.k_pages, c.v_pages)]

    def step():
        c.extend(rows, one, workspace=pw)
        c.append(k, v, cu1, q=q, q_out=qr, inv_freq=f)
        return c.attn(qr, cu1, max_new=1, max_len=320, workspace=aw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for a, b in zip((c.seq_len, c.page_table, c.refcount, c.k_pages, c.v_pages), keep):
        a.copy_(b)
    for i in range(40):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda").to(torch.bfloat16))
        g, (o, lse) = graphs[i % 2]
        g.replay()
        now = [n + i + 1 for n in lens]
        assert c.seq_len.tolist() == now
        if i % 13 == 0 or i == 39:
            check(c, c.page_table.cpu().numpy(), now, [1] * S, qr, o, lse, "NHD")
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,max_new,over", [(8, 1, 10), (4, 1, 20), (4, 1, 5), (4, 3, 40), (2, 1, 300)])
def test_an_entry_over_the_bound_spoils_none_of_its_group(D, group, max_new, over):
    """Its tokens count among the group's, which may pass what the call's bounds allow a segment of shared
    keys: the others' outputs are theirs all the same, and the next group's."""
    import long_context_grpo_gb300 as ls
    shared, S = 1280, 2 * group
    lens = [shared + 400 + 3 * b for b in range(S)]
    make, table = build(lens, 64, 2, D, seed=over, shared=shared, group=group, junk=float("nan"))
    c = make(8)
    new = [over if b == group - 1 else max_new for b in range(S)]
    T = sum(new)
    q = torch.randn(T, 8, D, device="cuda").to(torch.bfloat16)
    sl = torch.full((2,), shared, dtype=torch.int32, device="cuda")
    ws = torch.full((c.attn_workspace_bytes(S, T, max_new, max(lens)),), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = c.attn(q, cu(new), max_new=max_new, max_len=max(lens), group=group, shared_len=sl, workspace=ws)
    assert ls.device_status() == (7, 2)
    at = sum(new[:group - 1])
    bad = slice(at, at + over)
    assert not o[bad].any() and torch.isneginf(lse[bad]).all()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[bad] = False
    rows = [b for b in range(S) if b != group - 1]
    check(c, table, lens, [max_new] * (S - 1), q[keep], o[keep], lse[keep], "NHD", rows=rows)


@pytest.mark.gpu
@pytest.mark.parametrize("n,L", [(1, 90), (3, 40000), (70, 300), (70, 40000)])
@pytest.mark.parametrize("group", [1, 2])
@pytest.mark.parametrize("where", ["query", "last key", "first key"])
def test_a_poisoned_query_or_key_reaches_the_rows_that_see_it(where, group, n, L):
    """NaN outputs for these, in short and in split sequences, of their own and shared; the same bits as
    without it for all others."""
    import long_context_grpo_gb300 as ls
    Hq, Hkv = 8, 2
    shared = 64 if group > 1 and L < 256 else (L // 2 // 128 * 128 if group > 1 else 0)
    make, table = build([L] * 2, 64, Hkv, 128, seed=L, shared=shared, group=group)
    c = make(Hq)
    q = torch.randn(2 * n, Hq, 128, device="cuda").to(torch.bfloat16)
    sl = torch.tensor([shared], dtype=torch.int32, device="cuda") if group > 1 else None
    call = lambda: c.attn(q, cu([n] * 2), max_new=n, max_len=L, group=group, shared_len=sl)  # noqa: E731
    want = call()
    sees = torch.zeros(2 * n, Hq, dtype=torch.bool, device="cuda")
    if where == "query":
        q[n // 2, 5, 17] = float("nan")
        sees[n // 2, 5] = True
    else:
        # a key of key head 1: of the middle new token, or the prompt's first one (in shared pages both entries')
        pos = L - n + n // 2 if where == "last key" else 0
        c.k_pages[int(table[0, pos // 64]), pos % 64, 1, 3] = float("nan")
        sees[n // 2 if pos else 0:n, 4:] = True
        if pos < shared:
            sees[n:, 4:] = True
    o, lse = call()
    assert torch.isnan(o[sees]).all() and torch.isnan(lse[sees]).all()
    assert torch.equal(o[~sees], want[0][~sees]) and torch.equal(lse[~sees], want[1][~sees])
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("rotated", [False, True])
def test_append_refuses_offsets_that_are_not_a_partition_and_wild_lengths(rotated):
    """Rows whose tables list pages behind their ends: nothing is written there (nor anywhere by offsets that
    fall or leave the packed rows), and the device status says so."""
    import long_context_grpo_gb300 as ls
    S, T, ps = 4, 60, 16
    make, table = build([160] * S, ps, 2, 64, seed=8)
    c = make(4)
    k, v = (torch.randn(T, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, 4, 64, device="cuda").to(torch.bfloat16)
    f = ls.rope_freqs(64)[0]
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens = i32(*[100] * S)

    def call(offsets):
        before, q_out = c.k_pages.clone(), torch.full_like(q, 7.0)
        if rotated:
            c.append(k, v, offsets, q=q, q_out=q_out, inv_freq=f)
        else:
            c.append(k, v, offsets)
        return before, q_out

    for offsets in ((0, 50, 10, 30, 60), (0, 60, 0, 60, 60), (-1, 10, 20, 30, 60), (0, 10, 20, 30, 61), (5, 4, 4, 4, 60)):
        c.seq_len.copy_(lens)
        before, q_out = call(i32(*offsets))
        assert ls.device_status() == (7, 2), offsets
        assert torch.equal(c.k_pages, before) and bool((q_out == 7).all()), offsets
    for wild in (-1, -(1 << 31), 161, 1 << 30, (1 << 31) - 1):
        c.seq_len.copy_(lens)
        c.seq_len[1] = wild
        before, q_out = call(i32(0, 5, 25, 25, 60))
        assert ls.device_status() == (7, 2), wild
        want = before.clone()
        for b, t0, n in ((0, 0, 5), (3, 25, 35)):
            pos = torch.arange(100 - n, 100, device="cuda")
            kb, qb = k[t0:t0 + n], q[t0:t0 + n]
            if rotated:
                qb, kb = ls.rope(qb, kb, f, positions=pos)
                assert torch.equal(q_out[t0:t0 + n], qb)
            for j, p in enumerate(pos.tolist()):
                want[int(table[b, p // ps]), p % ps] = kb[j]
        assert torch.equal(c.k_pages, want) and bool((q_out[5:25] == 7).all()), wild
    # an entry that has nothing new is not looked at
    c.seq_len.copy_(lens)
    c.seq_len[1] = -5
    call(i32(0, 5, 5, 25, 60))
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("n,L", [(1, 30000), (3, 9999), (60, 20000), (300, 5000)])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (32, 8, 64)])
def test_another_split_of_the_same_sequence(n, L, Hq, Hkv, D):
    """Alone and beside others a sequence is cut into other chunks: the same values either way."""
    import long_context_grpo_gb300 as ls
    lens = [L] + [L - 171 * b for b in range(1, 24)]
    make, table = build(lens, 64, Hkv, D, seed=n)
    c = make(Hq)
    q = torch.randn(24 * n, Hq, D, device="cuda").to(torch.bfloat16)
    for S in (1, 2, 5, 24):
        o, lse = c.attn(q[:S * n], cu([n] * S), max_new=n, max_len=L)
        check(c, table, lens[:1], [n], q[:n], o[:n], lse[:n], "NHD")
        if S == 1:
            alone = o.clone(), lse.clone()
            again = c.attn(q[:n], cu([n]), max_new=4 * n, max_len=8 * L)
            assert torch.equal(o, again[0]) and torch.equal(lse, again[1])      # bounds move no split
        # twice the rounding of the probabilities (2^-8 of a weighted mean of |v|, below 1 here) and of o
        assert bool(((o[:n].double() - alone[0].double()).abs() <= 2 ** -7 + 2 ** -7 * alone[0].double().abs()).all())
        assert torch.allclose(lse[:n], alone[1], atol=4e-5, rtol=2 ** -20)
    assert ls.device_status() == (0, 0)
