"""Scores of given tokens and their gradient at every temperature and size of logits that the calls accept, against
float64.  Tolerances of the scores as in test_token_scores.py."""
import numpy as np
import pytest
import torch

from test_token_scores import check

COLD = [10.0 ** -k for k in range(1, 37)]


def rows(V, std, around, seed, scale=1.0):
    """40 rows: the given token is the largest, tied with it, the next one or any."""
    g = torch.Generator().manual_seed(seed)
    T = 40
    x = ((torch.randn(T, V, generator=g) * std + around) * scale).to(torch.bfloat16)
    x[5:10, 3] = x[5:10].amax(1)             # a tie
    x[10:15, ::2] = x[10:15].amax(1, keepdim=True)
    order = x.float().argsort(dim=1, descending=True, stable=True)
    at = torch.randint(0, V, (T,), generator=g)
    at[:20] = order[:20, 0]
    at[20:30] = order[20:30, min(1, V - 1)]
    return x.cuda(), at.to(torch.int32).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", COLD + [1e3, 1e9, 1e20, 1e36])
@pytest.mark.parametrize("V", [9, 700, 20000])
def test_scores_at_every_temperature(V, temperature):
    import long_context_grpo_gb300 as ls
    for std, around in ((2.0, 10.0), (3.0, -24.0), (0.01, 200.0)):
        x, ids = rows(V, std, around, V)
        check(ls.token_scores(x, ids, top=4, temperature=temperature), x, ids, 4, temperature)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [10.0 ** k for k in range(1, 37)])
def test_scores_of_large_logits(scale):
    import long_context_grpo_gb300 as ls
    for V, around in ((700, 10.0), (20000, -9.0)):
        x, ids = rows(V, 1.0, around, V, scale)
        check(ls.token_scores(x, ids, top=4), x, ids, 4, 1.0)
    assert ls.device_status() == (0, 0)
