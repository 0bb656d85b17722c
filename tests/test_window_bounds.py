"""Bounds of the windowed attention at the ends of their ranges, and refused offsets."""
import ctypes

import pytest
import torch

from test_cache_attn import build, cu


@pytest.mark.gpu
def test_no_workspace_for_bounds_that_are_refused():
    import long_context_grpo_gb300 as ls
    from long_context_grpo_gb300 import _lib as b
    make, _ = build([16], 16, 256, 64)
    c = make(256)
    T = (1 << 31) - 1
    bounds = dict(max_new=T, max_len=1000)
    # its jobs cannot be counted in 31 bits
    assert c.attn_workspace_bytes(1, T, window=9, **bounds) == 0
    assert c.attn_workspace_bytes(1, T >> 8, window=9, **bounds) > 0
    p = torch.zeros(256, dtype=torch.uint8, device="cuda").data_ptr()
    d = b.CacheAttnDesc(S=1, T=T, cu_new=p, q=p, q_stride=256 * 64, o=p, lse=p, group=1, **bounds)
    assert b._lib().ls_cache_attn_window(c._h, ctypes.byref(d), 9, 0, p, 256, None) == 2
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_first_tokens_up_to_the_longest_sequence_there_is():
    """All keys in sight, by first tokens that fill 31 bits or nearly so: the same split of the work."""
    import long_context_grpo_gb300 as ls
    make, _ = build([500], 16, 1, 64, seed=2, width=40)
    c = make(2)
    most = (1 << 31) - 1
    want = c.attn_workspace_bytes(1, 1, 1, most, window=1, sinks=most - 128)
    assert want > 1 << 10
    for sinks in (most - 126, most - 1, most, 1 << 50):
        assert c.attn_workspace_bytes(1, 1, 1, most, window=1, sinks=sinks) == want
    q = torch.randn(1, 2, 64, device="cuda").to(torch.bfloat16)
    o = [c.attn(q, cu([1]), max_new=1, max_len=most, window=1, sinks=s) for s in (most - 128, most, 1 << 50)]
    assert all(torch.equal(x, y) for a in o[1:] for x, y in zip(a, o[0]))
    assert ls.device_status() == (0, 0)
