"""Calls at once on two streams, and graphs that share a workspace: the bits of one call alone."""
import pytest
import torch


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def caches(S, L, Hq, Hkv, D, ps=32):
    """Two handles over the same pages, tables and lengths."""
    import long_context_grpo_gb300 as ls
    per = -(-L // ps)
    both = torch.randn(S * per, 2, ps, Hkv, D, device="cuda").to(torch.bfloat16)
    table = torch.randperm(S * per, device="cuda").to(torch.int32).view(S, per)
    length, ref = torch.full((S,), L, dtype=torch.int32, device="cuda"), torch.ones(S * per, dtype=torch.int32, device="cuda")
    return [ls.PagedCache(both[:, 0], both[:, 1], table, length, ref, Hq=Hq) for _ in range(2)]


def jobs():
    """(name, call(which) -> outputs): `which` 0 and 1 have workspaces and handles of their own."""
    import long_context_grpo_gb300 as ls
    out = []
    for n, L in ((1, 9000), (70, 2500)):
        c = caches(3, L, 8, 2, 128)
        q = torch.randn(3 * n, 8, 128, device="cuda").to(torch.bfloat16)
        at = i32(0, n, 2 * n, 3 * n)
        out.append(("attn %d" % n, lambda w, c=c, q=q, at=at, n=n, L=L: c[w].attn(q, at, max_new=n, max_len=L)))
    for T, V in ((200, 1000), (90, 33000), (40, 151936), (3, 310000)):
        x = torch.randn(T, V, device="cuda").to(torch.bfloat16)
        ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
        old, A, w = torch.full((T,), -8.0, device="cuda"), torch.randn(T, device="cuda"), torch.rand(T, device="cuda")
        out.append(("loss %d" % V, lambda _, x=x, ids=ids, old=old, A=A, w=w: tuple(
            ls.policy_loss(x, ids, old, A, w, logp_ref=old + 0.1, beta=0.1, kl="k3"))))
    x = torch.randn(700, 24, 128, device="cuda").to(torch.bfloat16)
    f, _ = ls.rope_freqs(128)
    out.append(("rope", lambda _, x=x, f=f: ls.rope(x[:, :16], x[:, 16:], f, pos0=7)))
    return out


def same(got, want, name):
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.gpu
def test_two_streams_at_once():
    import long_context_grpo_gb300 as ls
    todo = jobs()
    want = [fn(0) for _, fn in todo]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for w, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[w].append([fn(w) for _, fn in (todo if w == 0 else todo[::-1])])
    torch.cuda.synchronize()
    for w in range(2):
        for run in got[w]:
            for (name, _), g, x in zip(todo, run if w == 0 else run[::-1], want):
                same(g, x, name)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_graphs_that_share_a_workspace():
    """Two captured calls of other sizes in one workspace, replayed in turns and in a row."""
    import long_context_grpo_gb300 as ls
    c = caches(4, 6000, 8, 2, 64)[0]
    shapes = [(1, 6000), (50, 6000)]
    ws = torch.empty(max(c.attn_workspace_bytes(4, 4 * n, n, L) for n, L in shapes), dtype=torch.uint8, device="cuda")
    lw = torch.empty(ls.policy_loss_workspace_bytes(300), dtype=torch.uint8, device="cuda")
    graphs = []
    for n, L in shapes:
        q = torch.randn(4 * n, 8, 64, device="cuda").to(torch.bfloat16)
        at = i32(*range(0, 4 * n + 1, n))
        x = torch.randn(6 * n, 5000 if n == 1 else 800, device="cuda").to(torch.bfloat16)
        ids = torch.zeros(6 * n, dtype=torch.int32, device="cuda")
        z, one = torch.full((6 * n,), -7.0, device="cuda"), torch.ones(6 * n, device="cuda")

        def call(q=q, at=at, x=x, ids=ids, z=z, one=one, n=n, L=L):
            o = c.attn(q, at, max_new=n, max_len=L, workspace=ws)
            r = ls.policy_loss(x, ids, z, one, one, workspace=lw, loss=torch.empty(1, device="cuda"))
            return list(o) + list(r)

        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out, want, call))        # (the call keeps its inputs alive)
    ws.fill_(255)
    lw.fill_(255)
    for order in ((0, 1, 0, 1), (0, 0, 1, 1), (1, 0, 0, 1)):
        for i in order:
            for t in graphs[i][1]:
                t.view(torch.uint8).fill_(7)
            graphs[i][0].replay()
        torch.cuda.synchronize()
        for _, out, want, _ in graphs:
            same(out, want, "graph")
    assert ls.device_status() == (0, 0)
