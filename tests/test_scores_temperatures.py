"""Scores of given tokens and their gradient at every temperature and size of logits that the calls accept, against
float64.  Tolerances of the scores as in test_token_scores.py."""
import numpy as np
import pytest
import torch

from oracle.scores import scores_grad
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


def grad_check(got, x, ids, dl, de, t, lse):
    """Every value of the gradient.  log p is right to 4 x 2^-24 |lse| (lse as it is given, its product with
    log2 e, the temperature's factor, the fused difference) or, past 4,096, to what its parts relative to the row's
    maximum are, and to 2^-23 of itself; an exponential to 2^-22, products to 2^-22; both hold 1 / t's exponent (2^-23 of it); probabilities below 2^-126 may be 0."""
    x, dl, de, lse = (a.double().cpu().numpy() for a in (x, dl, de, lse))
    i = ids.cpu().numpy()
    want = scores_grad(x, i, dl, de, t)
    z = x / t
    m = z.max(1, keepdims=True)
    logp = np.maximum(z - m - np.log(np.exp(z - m).sum(1, keepdims=True)), -1000.0)
    p = np.exp(logp)
    ent = -(p * logp).sum(1)
    dl, de, ent = np.abs(dl)[:, None], np.abs(de)[:, None], ent[:, None]
    off = 4 * 2.0 ** -24 * np.minimum(np.abs(lse), 4096.0)[:, None] + 2.0 ** -23 * np.abs(logp) + 2.0 ** -21
    off += 2.0 ** -23 * max(0.0, -np.log2(t))
    size = (dl + de * (np.abs(logp) + ent + 1.0)) / t
    room = 2.0 ** -8 * np.abs(want) + (p * off + 2.0 ** -126) * size + 2.0 ** -133
    at = (np.arange(len(x)), i)
    # the given token's 1 - p: expm1 of a log-probability rounded to fp32 (at most 2^-24 x p |log p|, below 2^-25)
    room[at] += 2.0 ** -22 * dl[:, 0] / t
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    err = np.abs(g - want)
    assert (err <= room).all(), (err / room).max()


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [2.0 ** -120, 1e-36, 2.0 ** 120])
def test_gradient_at_the_ends(temperature):
    """Gradients of ordinary size whose quotient by the temperature is past fp32 only where a probability is not 0."""
    import long_context_grpo_gb300 as ls
    x = torch.zeros(4, 3000, dtype=torch.bfloat16)
    x[:, 7] = 2.0
    x[1, 9:] = float("-inf")
    x = x.cuda()
    ids = torch.tensor([7, 7, 7, 7], dtype=torch.int32, device="cuda")
    dl, de = torch.tensor([1000.0, -3.0, 0.0, 1.0], device="cuda"), torch.tensor([0.0, 1.0, -50.0, 1.0], device="cuda")
    r = ls.token_scores(x, ids, temperature=temperature)
    got = ls.token_scores_bwd(x, ids, r.logp, r.lse, r.entropy, dl, de, temperature=temperature).double().cpu()
    if temperature < 1:             # the largest logit has all of the probability: nothing moves it
        assert not got.any()
    else:
        assert torch.isfinite(got).all()


def both(x, ids, temperature, seed):
    """The gradient of scores and entropies, into a tensor of its own and in place."""
    import long_context_grpo_gb300 as ls
    g = torch.Generator().manual_seed(seed)
    dl, de = (torch.randn(len(ids), generator=g).cuda() for _ in range(2))
    r = ls.token_scores(x, ids, temperature=temperature)
    got = ls.token_scores_bwd(x, ids, r.logp, r.lse, r.entropy, dl, de, temperature=temperature)
    grad_check(got, x, ids, dl, de, temperature, r.lse)
    y = torch.empty(len(ids), x.shape[1] + 8, dtype=x.dtype, device="cuda").fill_(7.0)
    y[:, :x.shape[1]] = x
    z = y[:, :x.shape[1]]
    assert torch.equal(ls.token_scores_bwd(z, ids, r.logp, r.lse, r.entropy, dl, de, temperature=temperature, dlogits=z), got)
    assert (y[:, x.shape[1]:] == 7.0).all() and ls.device_status() == (0, 0)
    only = ls.token_scores_bwd(x, ids, r.logp, r.lse, d_logp=dl, temperature=temperature)
    grad_check(only, x, ids, dl, 0 * de, temperature, r.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [0.03, 0.005] + COLD + [1e3, 1e20])
@pytest.mark.parametrize("V", [9, 700, 20000])
def test_gradient_at_every_temperature(V, temperature):
    for std, around in ((2.0, 10.0), (3.0, -24.0), (40.0, -3000.0)):
        both(*rows(V, std, around, V), temperature, V)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [10.0 ** k for k in range(1, 37, 5)])
def test_gradient_of_large_logits(scale):
    for V, around in ((700, 10.0), (20000, -9.0)):
        both(*rows(V, 1.0, around, V, scale), 1.0, V)


@pytest.mark.gpu
def test_masked_tokens_of_cold_rows():
    """Masked logits, the given token among them, where lse is past what exponents from it could hold."""
    import long_context_grpo_gb300 as ls
    x, ids = rows(3000, 2.0, 30.0, 1)
    x[:, 100::3] = float("-inf")
    ids[::4] = 103
    r = ls.token_scores(x, ids, temperature=1e-3)
    dl = torch.ones(len(ids), device="cuda")
    grad_check(ls.token_scores_bwd(x, ids, r.logp, r.lse, d_logp=dl, temperature=1e-3), x, ids, dl, 0 * dl, 1e-3, r.lse)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(3, 13000), (400, 13000), (400, 13001), (300, 13387)])
@pytest.mark.parametrize("temperature", [0.01, 0.03, 0.2])
def test_maxima_that_grow_within_a_warp(T, V, temperature):
    """Two likely tokens of which the larger one comes a step behind the other, in the same warp: the sums change
    their reference by a whole number of its roundings."""
    import long_context_grpo_gb300 as ls
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, V, generator=g)
    at = torch.randint(0, 4096, (T,), generator=g)
    row = torch.arange(T)
    small = (4.0 + 11.9 * torch.rand(T, generator=g)).to(torch.bfloat16)
    x[row, at] = small.float()
    x[row, at + 4096] = (small.float() * (1.0 + 2.0 ** -7)).to(torch.bfloat16).float()      # the next value or the one after it
    x, ids = x.to(torch.bfloat16).cuda(), at.to(torch.int32).cuda()
    check(ls.token_scores(x, ids, top=3, temperature=temperature), x, ids, 3, temperature)
