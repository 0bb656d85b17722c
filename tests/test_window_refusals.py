"""Offsets that are no partition: the windowed attention does no entry, and every token's output says so."""
import pytest
import torch

from test_cache_attn import build


@pytest.mark.gpu
@pytest.mark.parametrize("max_new", [1, 40, 2560])
@pytest.mark.parametrize("offsets", ["falls", "saw", "negative", "past", "late", "wild"])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (16, 1, 128)])
def test_every_token_of_refused_offsets_is_zero(Hq, Hkv, D, offsets, max_new):
    import long_context_grpo_gb300 as ls
    S, n, L = 64, 40, 300
    make, _ = build([L] * S, 64, Hkv, D, seed=5)
    c = make(Hq)
    T = S * n
    q = torch.randn(T, Hq, D, device="cuda").to(torch.bfloat16)
    plain = [n * b for b in range(S + 1)]
    at = {"falls": [x - (200 if b == 30 else 0) for b, x in enumerate(plain)], "saw": [T * (b % 2) for b in range(S + 1)],
          "negative": [-1] + plain[1:], "past": plain[:-1] + [T + 1], "late": [500 + x for x in plain],
          "wild": [(-1) ** b * (b * 2654435761 % (1 << 31)) for b in range(S + 1)]}[offsets]
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    c.attn(q, torch.tensor(at, dtype=torch.int32, device="cuda"), max_new=max_new, max_len=L, window=64, sinks=4, o=o, lse=lse)
    assert ls.device_status() == (7, 2)
    free = 500 if offsets == "late" else 0        # (tokens before the first entry are nobody's)
    assert (o[:free] == 7.0).all() and (lse[:free] == 7.0).all()
    assert not o[free:].any() and torch.isneginf(lse[free:]).all()
