"""No window, said as None or 0 to a prefix and as None to the cache."""
import pytest
import torch


@pytest.mark.gpu
def test_no_window_is_none_or_zero_for_a_prefix():
    import long_context_grpo_gb300 as ls
    bf = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    kp, vp, ks, vs, q = bf(200, 1, 64), bf(200, 1, 64), bf(30, 1, 64), bf(30, 1, 64), bf(30, 2, 64)
    acc = torch.empty(2, 200, 1, 64, device="cuda")
    want = ls.Prefix(kp, vp, acc[0], acc[1], Hq=2).fwd(q, ks, vs)
    for window in (None, 0):
        p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=2, window=window)
        assert all(torch.equal(x, y) for x, y in zip(p.fwd(q, ks, vs), want))
        p.set_window(9, 1)
        assert not torch.equal(p.fwd(q, ks, vs)[0], want[0])
        p.set_window(window)
        assert all(torch.equal(x, y) for x, y in zip(p.fwd(q, ks, vs), want))
        with pytest.raises(ls.LongStrawError):
            ls.Prefix(kp, vp, acc[0], acc[1], Hq=2, window=window, sinks=1)
