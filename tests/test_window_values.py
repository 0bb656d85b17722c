"""How far a value that is not finite reaches in the attention over the cache: the entry's tokens that see it, and those that
share its products, up to 2 (128 // g) - 1 tokens before or behind one that does (g query heads a key head); without a
window, where keys behind a product's tokens are not cleared, up to 127 more before it."""
import pytest
import torch

from test_cache_attn import build, cu


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 64), (2, 2, 128), (4, 2, 64), (10, 2, 128), (16, 1, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n,window,sinks", [(700, 60, 0), (700, 200, 3), (300, 1, 0), (130, 129, 1), (600, None, 0)])
def test_how_far_a_value_reaches(n, window, sinks, bad, Hq, Hkv, D):
    import long_context_grpo_gb300 as ls
    L, g = n + 900, Hq // Hkv
    make, table = build([L] * 2, 64, Hkv, D, seed=n + sinks)
    c = make(Hq)
    q = torch.randn(2 * n, Hq, D, device="cuda").to(torch.bfloat16)
    sight = dict() if window is None else dict(window=window, sinks=sinks)
    call = lambda: c.attn(q, cu([n] * 2), max_new=n, max_len=L, **sight)  # noqa: E731
    want = call()
    window = window or L
    # seen first by the entry's first token (and not by its second), by one in its middle, by one whose window ends the entry
    for pos in {max(L - n - window + 1, 0), L - n + n // 3, L - window} - {0}:
        page, row = int(table[0, pos // 64]), pos % 64
        keep = c.v_pages[page, row].clone()
        c.v_pages[page, row, 0] = bad
        o, lse = call()
        p = torch.arange(L - n, L)
        sees = torch.zeros(2 * n, Hq, dtype=torch.bool)
        sees[:n, :g] = ((p >= pos) & (p < pos + window))[:, None]
        reach = 2 * (128 // g) - 1
        near = torch.zeros_like(sees)
        before = reach if sight else reach + 127
        near[:n, :g] = ((p >= max(pos, L - n) - before) & (p < pos + window + reach))[:, None]
        o, lse = o.cpu(), lse.cpu()
        assert (~torch.isfinite(o[sees])).all()
        assert torch.equal(o[~near], want[0].cpu()[~near]) and torch.equal(lse, want[1].cpu())
        c.v_pages[page, row] = keep
    assert ls.device_status() == (0, 0)
