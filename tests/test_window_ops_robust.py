"""The operators of windowed layers, head norms and token scores where calls meet: injected launch failures, two
streams at once, graphs that share a workspace, waits that give up, tensors past 2^31 elements, and the descriptors
against the header."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from test_cache_attn import build
from test_ops_streams import caches, i32, same

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def replay(seed=0, P=300, R=140, Hq=8, Hkv=2, D=128, **sight):
    import long_context_grpo_gb300 as ls
    g = torch.Generator(device="cuda").manual_seed(seed)
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    kp, vp, ks, vs = bf(P, Hkv, D), bf(P, Hkv, D), bf(R, Hkv, D), bf(R, Hkv, D)
    q, d = bf(R, Hq, D), bf(R, Hq, D)
    acc = torch.empty(2, P, Hkv, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=Hq, **sight)

    def call():
        o, lse = p.fwd(q, ks, vs)
        return (o, lse, *p.bwd(q, ks, vs, o, lse, d))

    return call


@pytest.mark.gpu
def test_injected_launch_failures():
    import long_context_grpo_gb300 as ls
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    make, _ = build([100], 16, 1, 64, seed=1)
    c = make(2)
    x = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    kv = x[:, :1].contiguous()
    lg, ids = torch.randn(4, 64, device="cuda").to(torch.bfloat16), i32(0, 1, 2, 3)
    z = torch.zeros(4, device="cuda")
    w = torch.ones(64, device="cuda")
    f, _ = ls.rope_freqs(64)
    calls = [("attn", lambda: c.attn(x, i32(0, 4), 4, 100, window=9, sinks=1)),
             ("append", lambda: c.append(kv, kv, i32(0, 4), inv_freq=f, norm_eps=1e-6)),
             ("norm", lambda: ls.norm_rope(x, None, w, None, f)),
             ("norm bwd", lambda: ls.norm_rope_bwd(x, None, x, None, w, None, f)),
             ("scores", lambda: ls.token_scores(lg, ids, top=3)),
             ("scores bwd", lambda: ls.token_scores_bwd(lg, ids, z, z, d_logp=z)), ("replay", replay(window=7, sinks=1))]
    for name, fn in calls:
        assert L.ls_debug_fail_launch(0) == 0
        with pytest.raises(ls.LongStrawError) as ex:
            fn()
        assert ex.value.status == 5 and "injected" in str(ex.value), name
        assert L.ls_debug_fail_launch_pending() == -1
        fn()
        torch.cuda.synchronize()
        assert ls.device_status() == (0, 0), name


def jobs():
    """(name, call(which) -> outputs): `which` 0 and 1 have workspaces and handles of their own."""
    import long_context_grpo_gb300 as ls
    out = []
    for n, L, sight in ((1, 9000, dict(window=4096, sinks=4)), (70, 2500, dict(window=600, sinks=0)), (2, 700, dict(window=64, sinks=3))):
        c = caches(3, L, 8, 2, 128)
        q = torch.randn(3 * n, 8, 128, device="cuda").to(torch.bfloat16)
        at = i32(0, n, 2 * n, 3 * n)
        out.append(("attn %d" % n, lambda w, c=c, q=q, at=at, n=n, L=L, s=sight: c[w].attn(q, at, max_new=n, max_len=L, **s)))
    for T, V, top in ((200, 1000, 5), (90, 33000, 20), (4, 151936, 1)):
        x = torch.randn(T, V, device="cuda").to(torch.bfloat16)
        ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
        dl = torch.randn(T, device="cuda")

        def score(_, x=x, ids=ids, top=top, dl=dl):
            r = ls.token_scores(x, ids, top=top, temperature=0.8)
            return (*r, ls.token_scores_bwd(x, ids, r.logp, r.lse, r.entropy, dl, dl, temperature=0.8))

        out.append(("scores %d" % V, score))
    x = torch.randn(700, 24, 128, device="cuda").to(torch.bfloat16)
    dx, w = torch.randn_like(x), torch.randn(128, device="cuda")
    f, _ = ls.rope_freqs(128)
    out.append(("norm", lambda _: ls.norm_rope(x[:, :16], x[:, 16:], w, w, f, pos0=7)))
    out.append(("norm bwd", lambda _: tuple(ls.norm_rope_bwd(dx[:, :16], dx[:, 16:], x[:, :16], x[:, 16:], w, w, f, pos0=7))))
    both = [replay(window=200, sinks=5) for _ in range(2)]
    out.append(("replay", lambda which: both[which]()))
    return out


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
    """Captured calls of other sizes in one workspace, replayed in turns and in a row, over what the last one left."""
    import long_context_grpo_gb300 as ls
    c = caches(4, 6000, 8, 2, 64)[0]
    shapes = [(1, dict(window=3000, sinks=4)), (50, dict(window=500, sinks=0)), (3, dict(window=5000, sinks=200))]
    ws = torch.empty(max(c.attn_workspace_bytes(4, 4 * n, n, 6000, **s) for n, s in shapes), dtype=torch.uint8, device="cuda")
    nw = torch.empty(ls.norm_rope_bwd_workspace_bytes(900, 64), dtype=torch.uint8, device="cuda")
    w, (f, _) = torch.ones(64, device="cuda"), ls.rope_freqs(64)
    graphs = []
    for n, sight in shapes:
        q = torch.randn(4 * n, 8, 64, device="cuda").to(torch.bfloat16)
        at = i32(*range(0, 4 * n + 1, n))
        x = torch.randn(17 * n, 4, 64, device="cuda").to(torch.bfloat16)

        def call(q=q, at=at, x=x, n=n, sight=sight):
            o = c.attn(q, at, max_new=n, max_len=6000, workspace=ws, **sight)
            r = ls.norm_rope_bwd(x, None, x, None, w, None, f, workspace=nw)
            return [*o, r.dq, r.dq_weight]

        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out, want, call))
    ws.fill_(255)
    nw.fill_(255)
    for order in ((0, 1, 2, 0), (0, 0, 1, 1), (2, 1, 0, 2)):
        for i in order:
            for t in graphs[i][1]:
                t.view(torch.uint8).fill_(7)
            graphs[i][0].replay()
            torch.cuda.synchronize()
            same(graphs[i][1], graphs[i][2], "graph")
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_a_captured_windowed_replay():
    """Forward, backward and finalization of the touched rows in one graph, replayed over other inputs."""
    import long_context_grpo_gb300 as ls
    P, R, H, D = 500, 90, 4, 64
    bf = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    kp, vp, ks, vs, q, d = bf(P, 1, D), bf(P, 1, D), bf(R, 1, D), bf(R, 1, D), bf(R, H, D), bf(R, H, D)
    acc = torch.empty(2, P, 1, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=H, window=100, sinks=2)
    ws = torch.empty(p.bwd_workspace_bytes(R), dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 99, 1, D, dtype=torch.bfloat16, device="cuda")

    def call():
        o, lse = p.fwd(q, ks, vs)
        r = p.bwd(q, ks, vs, o, lse, d, workspace=ws)
        p.finalize_rows(P - 99, 99, dk_out=out[0], dv_out=out[1], reset=True)
        return (o, lse, *r, out)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = call()
    for _ in range(3):
        q.copy_(bf(R, H, D))
        d.copy_(bf(R, H, D))
        want = [t.clone() for t in call()]
        acc[:, :2] = 0
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        same(got, want, "replay")


@pytest.mark.gpu
@pytest.mark.parametrize("polls", [1, 64])
def test_waits_that_give_up(tmp_path, polls):
    """A library whose attention waits give up after a few polls, unless they are over by then: every call through a
    window returns, in the cache and in the replay, the status says so, and the context stays usable."""
    script = """
import sys
from long_context_grpo_gb300 import build as lb
lb.BUILD_DIR, lb.LIB = sys.argv[1] + "/obj", sys.argv[1] + "/lib.so"
lb.FLAGS = lb.FLAGS + ["-DLS_WAIT_LIMIT_NS=0ull", "-DLS_WAIT_POLLS=%su" % sys.argv[2], '-DLS_WAIT_POLL="test_wait"']
lb.build(force=True)
import torch
import long_context_grpo_gb300 as ls
assert ls.library_path == lb.LIB
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
ps, Hq, Hkv, total = 64, 16, 4, 0
for S, n, lens, window, sinks in ((20, 1, 6000, 4000, 4), (3, 200, 6000, 1000, 300), (1, 300, 30000, 9000, 0), (6, 3, 500, 64, 8)):
    for D in (64, 128):
        pages = -(-lens // ps)
        table = torch.arange(S * pages, dtype=torch.int32, device="cuda").view(S, pages)
        both = torch.randn(S * pages, 2, ps, Hkv, D, device="cuda").to(torch.bfloat16)
        c = ls.PagedCache(both[:, 0], both[:, 1], table, i32(*[lens] * S), i32(*[1] * (S * pages)), Hq=Hq)
        q = torch.randn(S * n, Hq, D, device="cuda").to(torch.bfloat16)
        R = 40 * n if n < 100 else n
        kp, ks, qr = (torch.randn(m, h, D, device="cuda").to(torch.bfloat16) for m, h in ((lens, Hkv), (R, Hkv), (R, Hq)))
        acc = torch.empty(2, lens, Hkv, D, device="cuda")
        p = ls.Prefix(kp, kp, acc[0], acc[1], Hq=Hq, window=window, sinks=sinks)
        gave_up = 0
        for _ in range(10):
            c.attn(q, i32(*[n * x for x in range(S + 1)]), max_new=n, max_len=lens, window=window, sinks=sinks)
            o, lse = p.fwd(qr, ks, ks)
            p.bwd(qr, ks, ks, o, lse, qr)
            torch.cuda.synchronize()
            status = ls.device_status()
            assert status in ((0, 0), (6, 1)), status
            gave_up += status == (6, 1)
        print(S, n, D, gave_up, "of 10")
        total += gave_up
x = torch.ones(1 << 20, device="cuda")
assert x.sum().item() == 1 << 20
assert total > 0 or sys.argv[2] != "1"
print("all returned")
"""
    r = subprocess.run([sys.executable, "-c", script, str(tmp_path), str(polls)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0 and "all returned" in r.stdout, r.stdout + r.stderr


@pytest.mark.gpu
def test_norms_past_2_31_elements():
    import long_context_grpo_gb300 as ls
    T, H, D = 600001, 28, 128
    x = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn(D, device="cuda")
    f, _ = ls.rope_freqs(D)
    y, _ = ls.norm_rope(x, None, w, None, f)
    rows = torch.tensor([0, 599186, 599187, T - 1], device="cuda")
    assert 599187 * H * D > 1 << 31
    want, _ = ls.norm_rope(x[rows], None, w, None, f, positions=rows)
    assert torch.equal(y[rows], want)
    r = ls.norm_rope_bwd(y, None, x, None, w, None, f, dq_out=y)
    part = ls.norm_rope_bwd(want, None, x[rows], None, w, None, f, positions=rows)
    assert torch.equal(r.dq[rows], part.dq)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 70])
def test_far_pages_of_a_large_pool(n):
    """Element offsets past 2^32 through a window."""
    import long_context_grpo_gb300 as ls
    N, ps, Hkv, D = 18000, 256, 4, 128
    both = torch.zeros(N, 2, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    near, far = [0, 1, 2], [N - 1, N - 2, N - 3]
    both[near] = torch.randn(3, 2, ps, Hkv, D, device="cuda").to(torch.bfloat16)
    both[far] = both[near]
    table = i32(*near, *far).view(2, 3)
    c = ls.PagedCache(both[:, 0], both[:, 1], table, i32(700, 700), torch.ones(N, dtype=torch.int32, device="cuda"), Hq=8)
    q = torch.randn(n, 8, D, device="cuda").to(torch.bfloat16).repeat(2, 1, 1)
    o, lse = c.attn(q, i32(0, n, 2 * n), max_new=n, max_len=700, window=300, sinks=9)
    assert torch.equal(o[:n], o[n:]) and torch.equal(lse[:n], lse[n:]) and bool(o.any())
    k, v = (torch.randn(2 * n, Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    k[n:], v[n:] = k[:n], v[:n]
    c.append(k, v, i32(0, n, 2 * n), norm_eps=1e-6)
    assert torch.equal(both[far], both[near]) and torch.equal(both[N - 3, 1, 700 - 512 - n:700 - 512], v[n:])


def test_structures_match_the_header(tmp_path):
    """sizeof and the last field's offset of every new descriptor, from the header itself."""
    from long_context_grpo_gb300 import _lib as b
    last = {"ls_token_scores_desc": ("top_logp", "TokenScoresDesc"), "ls_token_scores_bwd_desc": ("dlogits", "TokenScoresBwdDesc"),
            "ls_head_norm": ("eps", "HeadNorm"), "ls_head_norm_grad": ("dk_weight", "HeadNormGrad")}
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "%s/include/longstraw.h"\nint main(void){\n' % ROOT
    for c, (f, _) in last.items():
        src += 'printf("%%zu %%zu\\n", sizeof(%s), offsetof(%s, %s));\n' % (c, c, f)
    (tmp_path / "t.c").write_text(src + "return 0;}\n")
    subprocess.run(["gcc", "-std=c99", str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    out = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout.split()
    for i, (f, py) in enumerate(last.values()):
        D = getattr(b, py)
        assert (ctypes.sizeof(D), getattr(D, f).offset) == (int(out[2 * i]), int(out[2 * i + 1])), py


def test_binding_refuses_before_the_library():
    import long_context_grpo_gb300 as ls
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        ls.norm_rope(x, None, None, None)
    with pytest.raises(TypeError):
        ls.norm_rope(None, None, None, None)
    with pytest.raises(TypeError):
        ls.token_scores(None, None)
    with pytest.raises(TypeError):
        ls.token_scores_bwd(x[0], None, None, None)


@pytest.mark.gpu
def test_a_window_past_64_bits_is_one_past_the_sequence():
    import long_context_grpo_gb300 as ls
    mk, _ = build([200], 16, 1, 64, seed=5, width=20)
    c = mk(2)
    q = torch.randn(3, 2, 64, device="cuda").to(torch.bfloat16)
    offsets = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    want = c.attn(q, offsets, 3, 200, window=200)
    for window, sinks in ((1 << 64) + 1, 0), (5, (1 << 64) + 1), (1 << 200, 1 << 70):      # all keys are in sight
        got = c.attn(q, offsets, 3, 200, window=window, sinks=sinks)
        # lse is near log 200; sums of at most 200 terms in another order: 8 x 2^-24 of their value
        assert torch.allclose(got[1], want[1], rtol=2.0 ** -20, atol=0)
    with pytest.raises(ls.LongStrawError):
        c.attn(q, offsets, 3, 200, window=-(1 << 70))
