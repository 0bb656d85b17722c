"""Launch failures injected into the new entry points: reported, recovered from, no device status."""
import pytest
import torch


@pytest.mark.gpu
def test_injected_launch_failures_of_the_group_operators():
    import long_context_grpo_gb300 as ls
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    both = torch.randn(8, 2, 16, 1, 64, device="cuda").to(torch.bfloat16)
    c = ls.PagedCache(both[:, 0], both[:, 1], i32([0, 0], [0, 0]), i32(0, 0), i32(*[0] * 8), Hq=2)
    c.reset()
    x = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    kv = x[:, :1].contiguous()
    lg = torch.randn(4, 64, device="cuda").to(torch.bfloat16)
    z = torch.zeros(4, device="cuda")
    f, _ = ls.rope_freqs(64)
    calls = [("reset", c.reset), ("extend", lambda: c.extend(i32(0), i32(4))), ("append", lambda: c.append(kv, kv, i32(0, 4))),
             ("attn", lambda: c.attn(x, i32(0, 4), 4, 4)), ("fork", lambda: c.fork(i32(0), i32(1))), ("compact", c.compact),
             ("free", lambda: c.free(i32(0, 1))), ("rope", lambda: ls.rope(x, None, f)),
             ("policy", lambda: ls.policy_loss(lg, i32(0, 1, 2, 3), z, z, z))]
    for name, fn in calls:
        before = c.seq_len.clone(), c.refcount.clone()
        assert L.ls_debug_fail_launch(0) == 0
        with pytest.raises(ls.LongStrawError) as ex:
            fn()
        assert ex.value.status == 5 and "injected" in str(ex.value), name
        assert torch.equal(before[0], c.seq_len) and torch.equal(before[1], c.refcount)
        fn()
        torch.cuda.synchronize()
        assert ls.device_status() == (0, 0), name


@pytest.mark.gpu
def test_kernel_times_of_the_group_operators():
    import long_context_grpo_gb300 as ls
    ls.timing_enable(True)
    try:
        ls.timing_read()
        x = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
        ls.rope(x, None, ls.rope_freqs(64)[0])
        got = ls.timing_read()
    finally:
        ls.timing_enable(False)
    assert got["rope"][1] == 1 and got["rope"][0] > 0 and got["cache_attn"][1] == 0


@pytest.mark.gpu
def test_lists_and_flat_tensors_are_refused_by_name():
    import long_context_grpo_gb300 as ls
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    both = torch.randn(8, 2, 16, 1, 64, device="cuda").to(torch.bfloat16)
    c = ls.PagedCache(both[:, 0], both[:, 1], i32([0, 0], [0, 0]), i32(0, 0), i32(*[0] * 8), Hq=2)
    x = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    kv = x[:, :1].contiguous()
    f, _ = ls.rope_freqs(64)
    for name, fn in [("rows", lambda: c.extend([0], [4])), ("parents", lambda: c.fork([0], [1])), ("rows", lambda: c.free([0])),
                     ("cu_new", lambda: c.append(kv, kv, [0, 4])), ("cu_new", lambda: c.attn(x, [0, 4], 4, 4)),
                     ("q and k", lambda: ls.rope(x, kv.view(-1), f)), ("q or k", lambda: ls.rope(None, None, f)),
                     ("rows", lambda: c.free(i32([0, 1]).view(1, 2)))]:
        with pytest.raises(TypeError, match=name):
            fn()


def test_wait_limit_of_the_operators_is_validated_on_the_host():
    from long_context_grpo_gb300 import build as lsbuild
    lsbuild.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    assert L.ls_debug_wait_limit(10_000_000_001) == 1
    assert L.ls_debug_wait_limit(10_000_000_000) == 0 and L.ls_debug_wait_limit(0) == 0
    assert L.ls_debug_wait_limit(-1) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,pad,shift", [(3000, 5000, 0, 0), (1500, 32000, 0, 0), (1500, 32003, 1, 3), (700, 50257, 7, 0),
                                           (500, 151936, 0, 0), (300, 151937, 1, 5), (200, 300001, 0, 1)])
@pytest.mark.parametrize("limit", [0, 1, 1000, 5000, 20000])
def test_policy_loss_waits_that_give_up(T, V, pad, shift, limit):
    """A short limit runs out while copies and exchanges are under way: the call reports it, the tokens that
    are not NaN are right, the loss is NaN, and the next call is as ever.  Cluster sizes 1, 2, 4 and 8; gradient
    rows on the logits' alignment and `shift` elements beside it; a third of the tokens left out."""
    import long_context_grpo_gb300 as ls
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(T, V + pad, generator=g, device="cuda", dtype=torch.bfloat16) * 2)[:, :V]
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    old = -torch.rand(T, generator=g, device="cuda") * 20
    adv = torch.randn(T, generator=g, device="cuda")
    w = (torch.rand(T, generator=g, device="cuda") >= 1 / 3).float() / T
    w[0] = 1 / T
    room = torch.empty(T * (V + 8) + 16, dtype=torch.bfloat16, device="cuda")
    d = room[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    call = lambda: ls.policy_loss(x, ids, old, adv, w, dlogits=d)  # noqa: E731
    want = call()
    grad = want.dlogits.clone()
    assert ls.device_status() == (0, 0)
    for _ in range(3):
        try:
            assert L.ls_debug_wait_limit(limit) == 0
            r = call()
            torch.cuda.synchronize()
        finally:
            L.ls_debug_wait_limit(-1)
        status = ls.device_status()
        lost = torch.isnan(r.logp)
        assert status == ((6, 1) if lost.any() else status) and status in ((0, 0), (6, 1))
        assert limit > 0 or lost.any()
        assert not lost[w == 0].any() and torch.isnan(r.loss).item() == lost.any().item()
        assert torch.equal(r.logp[~lost], want.logp[~lost]) and torch.equal(r.clip_mask[~lost], want.clip_mask[~lost])
        assert torch.equal(r.dlogits[~lost], grad[~lost])
        r = call()
        assert torch.equal(r.loss, want.loss) and torch.equal(r.dlogits, grad) and torch.equal(r.logp, want.logp)
        assert ls.device_status() == (0, 0)



@pytest.mark.gpu
@pytest.mark.parametrize("polls", [1, 64])
def test_cache_attention_waits_that_give_up(tmp_path, polls):
    """A library whose attention waits give up after a few polls, unless they are over by then: every call
    returns, the copies in flight have landed (the calls follow one another on the same shared memory), the
    status says so, and the context stays usable."""
    import subprocess
    import sys
    from pathlib import Path
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
for S, n, lens, group in ((20, 1, 6000, 1), (8, 1, 9000, 8), (3, 200, 6000, 1), (1, 300, 30000, 1), (4, 40, 5000, 2)):
    for D in (64, 128):
        pages, shared = -(-lens // ps), lens // 2 // 128 * 128
        table = torch.arange(S * pages, dtype=torch.int32, device="cuda").view(S, pages)
        for x in range(S):
            table[x, :shared // ps] = table[x - x % group, :shared // ps]
        both = torch.randn(S * pages, 2, ps, Hkv, D, device="cuda").to(torch.bfloat16)
        c = ls.PagedCache(both[:, 0], both[:, 1], table, i32(*[lens] * S), i32(*[1] * (S * pages)), Hq=Hq)
        q = torch.randn(S * n, Hq, D, device="cuda").to(torch.bfloat16)
        sl = i32(*[shared] * (S // group)) if group > 1 else None
        gave_up = 0
        for _ in range(20):
            o, lse = c.attn(q, i32(*[n * x for x in range(S + 1)]), max_new=n, max_len=lens, group=group, shared_len=sl)
            torch.cuda.synchronize()
            status = ls.device_status()
            assert status in ((0, 0), (6, 1)), status
            gave_up += status == (6, 1)
        print(S, n, D, gave_up, "of 20")
        total += gave_up
x = torch.ones(1 << 20, device="cuda")
assert x.sum().item() == 1 << 20
assert total > 0 or sys.argv[2] != "1"
print("all returned")
"""
    root = Path(__file__).resolve().parent.parent
    r = subprocess.run([sys.executable, "-c", script, str(tmp_path), str(polls)], cwd=root, capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0 and "all returned" in r.stdout, r.stdout + r.stderr
