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
