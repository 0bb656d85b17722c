"""Scores of given tokens and their gradient against float64.

Tolerances.  An exponential is off by 2^-22 and its argument z by two fp32 roundings and that of log2 e /
temperature (3 x 2^-24 |z|, with weights p below 2^-22 (entropy + 1)); the sums are compensated; so
log S is off by 2^-21 (entropy + 1) and a value v, rounded once, by 2^-24 |v| besides.  The entropy adds sum e z
with fp32 additions of up to 2^7 terms a thread (2^-17 of it, and of it only the sum's rounding: at
most 2^-20 with pairwise parts of 32).  The gradient is bf16 of p's own relative error 2^-18 (lse is rounded to fp32:
|lse| 2^-24, below 2^-18 for |lse| < 60) and of what cancels in log p + entropy."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.scores import scores, scores_grad


def make(T, V, seed, std=2.0, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, V + pad + offset, generator=g) * std
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    x[torch.arange(T), ids.long() + offset] += 15.0 * torch.rand(T, generator=g)
    return x.to(torch.bfloat16).cuda()[:, offset:offset + V], ids.cuda()


def host(t):
    return t.double().cpu().numpy()


def check(r, x, ids, top, temperature):
    lp, lse, ent, order, tl = scores(host(x), ids.cpu().numpy(), top, temperature)
    room = 2.0 ** -20 * (np.nan_to_num(ent) + 1.0)
    for got, want in ((r.logp, lp), (r.lse, lse), (r.entropy, ent)):
        got = host(got)
        # (values past fp32's largest, 3.4e38, are infinite in it: -3.3e38 - 3.3e38)
        with np.errstate(over="ignore"):
            f = np.isfinite(want.astype(np.float32))
        want = np.where(f | np.isnan(want), want, np.copysign(np.inf, want))
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
        assert (got[~f & ~np.isnan(want)] == want[~f & ~np.isnan(want)]).all()
        err = np.abs(got[f] - want[f])
        assert (err <= (room + 2.0 ** -22 * np.abs(want))[f]).all(), err.max()
    assert r.top_ids.shape == r.top_logp.shape == (len(lp), top)
    assert np.array_equal(r.top_ids.cpu().numpy(), order)
    got = host(r.top_logp)
    with np.errstate(over="ignore"):
        f = np.isfinite(tl.astype(np.float32))
    assert np.array_equal(np.isnan(got), np.isnan(tl)) and np.array_equal(np.isneginf(got), ~f & ~np.isnan(tl))
    assert (np.abs(got[f] - tl[f]) <= (room[:, None] + 2.0 ** -22 * np.abs(tl))[f]).all()


SIZES = [(1, 1), (3, 2), (5, 31), (4, 33), (33, 1024), (7, 1000), (2, 8193), (3, 32000), (1, 151936), (300, 4097), (700, 640),
         (2, 70001)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("top", [0, 1, 5, 64])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_against_float64(T, V, top, pad, offset):
    import long_context_grpo_gb300 as ls
    top = min(top, V)
    x, ids = make(T, V, T + V, pad=pad, offset=offset)
    t = 0.7 if top == 5 else 1.0
    check(ls.token_scores(x, ids, top=top, temperature=t), x, ids, top, t)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 400])
@pytest.mark.parametrize("V", [40, 2000, 33000])
@pytest.mark.parametrize("kind", ["equal", "few", "rising", "falling", "steps", "last", "zeros", "tiny", "huge", "lowest"])
def test_ties_masks_and_orders(kind, V, T):
    """Ties go to the lowest index, wherever the best logits lie."""
    import long_context_grpo_gb300 as ls
    inf = float("inf")
    x = torch.zeros(T, V)
    if kind == "few":               # what a grammar leaves
        x.fill_(-inf)
        x[:, 5::V // 3] = torch.randn(T, len(range(5, V, V // 3)))
    elif kind == "rising":
        x += torch.linspace(-20, 20, V)
    elif kind == "falling":
        x += torch.linspace(20, -20, V)
    elif kind == "steps":
        x += torch.arange(V) // 37 % 11
    elif kind == "last":
        x.fill_(-inf)
        x[:, -2:] = 3.0
    elif kind == "zeros":
        x[:, ::2] = -0.0
    elif kind == "tiny":
        x = torch.randn(T, V) * 1e-38
    elif kind == "huge":
        x = torch.randn(T, V).sign() * 3.3e38
    elif kind == "lowest":          # masks of the type's lowest value
        x = torch.randn(T, V)
        x[:, V // 4:] = torch.finfo(torch.bfloat16).min
        x[0] = torch.finfo(torch.bfloat16).min
    x = x.to(torch.bfloat16).cuda()
    ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    for top in (1, 20, 40):
        check(ls.token_scores(x, ids, top=top), x, ids, top, 1.0)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [24, 3000, 40000])
def test_rows_without_a_distribution_and_wild_ids(V):
    import long_context_grpo_gb300 as ls
    x, ids = make(9, V, V)
    x[1] = -float("inf")
    x[2, V // 2] = float("nan")
    x[3, V - 1] = float("inf")
    x[4, 0] = -float("nan")
    x[5, 7] = -float("inf")
    ids[5] = 7
    r = ls.token_scores(x, ids, top=8)
    check(r, x, ids, 8, 1.0)
    assert ls.device_status() == (0, 0)
    assert torch.isnan(r.logp[1:5]).all() and bool((r.top_ids[1:5] == -1).all()) and float(r.logp[5]) == -float("inf")
    ids[6], ids[8] = V, -1
    check(ls.token_scores(x, ids, top=8), x, ids, 8, 1.0)
    assert ls.device_status() == (7, 2)


@pytest.mark.gpu
def test_likely_tokens_keep_their_small_log_probabilities():
    """Rows whose given token has nearly all of the probability: relative accuracy of what is left."""
    import long_context_grpo_gb300 as ls
    T, V = 64, 5000
    x = torch.randn(T, V)
    ids = torch.arange(T, dtype=torch.int32)
    x[torch.arange(T), ids.long()] = torch.linspace(8, 40, T)
    x, ids = x.to(torch.bfloat16).cuda(), ids.cuda()
    r = ls.token_scores(x, ids)
    lp, _, ent, _, _ = scores(host(x), ids.cpu().numpy())
    # compensated sums: 2^-22 an exponential, 2^-46 of the whole
    assert (np.abs(host(r.logp) - lp) <= 2.0 ** -17 * np.abs(lp) + 2.0 ** -42).all()
    assert (np.abs(host(r.entropy) - ent) <= 2.0 ** -16 * ent + 2.0 ** -42).all()


def grad_check(got, x, ids, dl, de, t):
    x, dl, de = host(x), host(dl), host(de)
    want = scores_grad(x, ids.cpu().numpy(), dl, de, t)
    lp, lse, ent, _, _ = scores(x, ids.cpu().numpy(), 0, t)
    logp = np.maximum(x / t - lse[:, None], -1000.0)
    p = np.exp(logp)
    # p to 2^-18, log p + entropy to 2^-19 of its parts
    size = p * (np.abs(dl)[:, None] + np.abs(de)[:, None] * (np.abs(logp) + ent[:, None])) / t
    room = 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * size + 2.0 ** -133
    row = np.arange(len(x))
    room[row, ids.cpu().numpy()] += 2.0 ** -17 * np.abs(dl) / t
    err = np.abs(host(got) - want)
    assert (err <= room).all(), (err / room).max()


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,pad,offset", [(1, 1, 0, 0), (5, 33, 0, 0), (40, 1000, 3, 1), (3, 8200, 8, 0), (2, 151936, 0, 0),
                                            (130, 8192, 0, 0)])
@pytest.mark.parametrize("which", ["both", "logp", "entropy"])
def test_gradient_against_float64(T, V, pad, offset, which):
    import long_context_grpo_gb300 as ls
    x, ids = make(T, V, T, pad=pad, offset=offset)
    g = torch.Generator().manual_seed(T)
    dl, de = torch.randn(T, generator=g).cuda(), torch.randn(T, generator=g).cuda()
    t = 0.6
    r = ls.token_scores(x, ids, temperature=t)
    kw = {"both": dict(d_logp=dl, d_entropy=de), "logp": dict(d_logp=dl), "entropy": dict(d_entropy=de)}[which]
    if which != "logp":
        kw["entropy"] = r.entropy
    got = ls.token_scores_bwd(x, ids, r.logp, r.lse, temperature=t, **kw)
    zero = torch.zeros(T, device="cuda")
    grad_check(got, x, ids, kw.get("d_logp", zero), kw.get("d_entropy", zero), t)
    # in place, within a wider tensor
    keep = x.clone()
    out = ls.token_scores_bwd(x, ids, r.logp, r.lse, temperature=t, dlogits=x, **kw)
    assert out is x and torch.equal(x, got) and not torch.equal(keep, x)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_gradient_is_a_difference():
    import long_context_grpo_gb300 as ls
    T, V, t = 3, 50, 1.3
    x, ids = make(T, V, 3)
    dl, de = torch.tensor([1.0, -2.0, 0.5], device="cuda"), torch.tensor([0.3, 0.0, -1.0], device="cuda")
    r = ls.token_scores(x, ids, temperature=t)
    got = host(ls.token_scores_bwd(x, ids, r.logp, r.lse, r.entropy, dl, de, temperature=t))
    X, I = host(x), ids.cpu().numpy()
    for at in ((0, 7), (1, int(I[1])), (2, 49)):
        ends = []
        for s in (1e-5, -1e-5):
            y = X.copy()
            y[at] += s
            lp, _, ent, _, _ = scores(y, I, 0, t)
            ends.append((host(dl) * lp + host(de) * ent).sum())
        assert abs(got[at] - (ends[0] - ends[1]) / 2e-5) <= 2.0 ** -7 * abs(got[at]) + 1e-7


@pytest.mark.gpu
def test_gradient_of_rows_that_are_left_out_masked_or_wild():
    import long_context_grpo_gb300 as ls
    T, V = 7, 9000
    x, ids = make(T, V, 5)
    x[2, ::3] = -float("inf")
    ids[2] = 1
    x[3, ::3] = -float("inf")
    ids[3] = 3                      # the given token is masked itself
    r = ls.token_scores(x, ids)
    dl = torch.ones(T, device="cuda")
    de = torch.full((T,), 0.5, device="cuda")
    dl[1], de[1] = 0.0, 0.0
    x[1] = float("nan")
    for a in (r.logp, r.lse, r.entropy):
        a[1] = float("nan")
    got = ls.token_scores_bwd(x, ids, r.logp, r.lse, r.entropy, dl, de)
    assert not got[1].any() and torch.isfinite(got).all() and ls.device_status() == (0, 0)
    rows = [0, 2, 4, 5, 6]
    grad_check(got[rows], x[rows], ids[rows], dl[rows], de[rows], 1.0)
    # its one is the formula's: d_logp, at a probability of 0
    assert float(got[3, 3]) == 1.0 and not got[3, 6::3].any()
    r.lse[4] = float("nan")
    ids[5] = V
    bad = ls.token_scores_bwd(x, ids, r.logp, r.lse, d_logp=dl)
    assert not bad[5].any() and torch.isnan(bad[4, torch.arange(V, device="cuda") != int(ids[4])]).all()
    assert ls.device_status() == (7, 2)


@pytest.mark.gpu
def test_captured_on_another_stream():
    """A graph of scores and gradient replayed with other logits."""
    import long_context_grpo_gb300 as ls
    x, ids = make(6, 20000, 1)
    de = torch.randn(6, device="cuda")

    def step():
        r = ls.token_scores(x, ids, top=4)
        return r, ls.token_scores_bwd(x, ids, r.logp, r.lse, r.entropy, d_entropy=de)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r, d = step()
    for seed in (2, 3):
        y, i = make(6, 20000, seed)
        x.copy_(y)
        ids.copy_(i)
        g.replay()
        torch.cuda.synchronize()
        check(r, x, ids, 4, 1.0)
        grad_check(d, x, ids, torch.zeros_like(de), de, 1.0)


@pytest.mark.gpu
def test_rows_past_2_31_elements():
    import long_context_grpo_gb300 as ls
    T, V = 15000, 151936
    x = torch.empty(T, V, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    r = ls.token_scores(x, ids, top=3)
    rows = torch.tensor([0, 14133, 14134, 14135, T - 1], device="cuda")
    part = ls.TokenScores(*(a[rows] for a in r))
    check(part, x[rows], ids[rows], 3, 1.0)
    dl = torch.ones(T, device="cuda")
    d = ls.token_scores_bwd(x, ids, r.logp, r.lse, d_logp=dl, dlogits=x.clone())
    grad_check(d[rows], x[rows], ids[rows], dl[rows], 0 * dl[rows], 1.0)


def test_refusals():
    from long_context_grpo_gb300 import build as lsbuild
    lsbuild.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    base = dict(T=4, V=64, logits_stride=64, logits=0x1000, ids=0x2000, temperature=1.0, top=2, logp=0x3000, lse=0x4000,
                entropy=0x5000, top_ids=0x6000, top_logp=0x7000)
    call = lambda **kw: L.ls_token_scores(ctypes.byref(b.TokenScoresDesc(**{**base, **kw})), None)  # noqa: E731
    nan, inf = float("nan"), float("inf")
    assert L.ls_token_scores(None, None) == 1 and L.ls_token_scores_bwd(None, None) == 1
    for kw in (dict(logits=None), dict(ids=None), dict(logp=None), dict(T=0), dict(V=0), dict(logits_stride=63), dict(top=-1),
               dict(top=65), dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=nan), dict(temperature=inf),
               dict(temperature=1e-320), dict(top_ids=None), dict(top_logp=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(V=100, logits_stride=100, top=65), dict(V=(1 << 23) + 1, logits_stride=1 << 24), dict(T=1 << 28),
               dict(V=1 << 31, logits_stride=1 << 31, top=0)):
        assert call(**kw) == 2, kw
    for kw in (dict(logits=0x1001), dict(ids=0x2002), dict(logp=0x3002), dict(entropy=0x5001), dict(top_ids=0x6002)):
        assert call(**kw) == 4, kw
    base = dict(T=4, V=64, logits_stride=64, dlogits_stride=64, logits=0x1000, ids=0x2000, temperature=1.0, logp=0x3000,
                lse=0x4000, entropy=0x5000, d_logp=0x6000, d_entropy=0x7000, dlogits=0x8000)
    call = lambda **kw: L.ls_token_scores_bwd(ctypes.byref(b.TokenScoresBwdDesc(**{**base, **kw})), None)  # noqa: E731
    for kw in (dict(logits=None), dict(ids=None), dict(logp=None), dict(lse=None), dict(dlogits=None), dict(entropy=None),
               dict(d_logp=None, d_entropy=None), dict(T=0), dict(V=0), dict(logits_stride=63), dict(dlogits_stride=63),
               dict(temperature=0.0), dict(dlogits=0x1000, dlogits_stride=72)):
        assert call(**kw) == 1, kw
    assert call(T=1 << 28) == 2 and call(dlogits_stride=1 << 31) == 2
    assert call(dlogits=0x8001) == 4 and call(d_logp=0x6002) == 4


@pytest.mark.parametrize("temperature", [2.0 ** -121, 1e-40, 2.0 ** 121, 1e60])
def test_a_temperature_past_fp32_is_refused(temperature):
    from long_context_grpo_gb300 import build as lsbuild
    lsbuild.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    d = b.TokenScoresDesc(T=4, V=64, logits_stride=64, logits=0x1000, ids=0x2000, temperature=temperature, top=0, logp=0x3000)
    assert L.ls_token_scores(ctypes.byref(d), None) == 1
    d = b.TokenScoresBwdDesc(T=4, V=64, logits_stride=64, dlogits_stride=64, logits=0x1000, ids=0x2000,
                             temperature=temperature, logp=0x3000, lse=0x4000, d_logp=0x6000, dlogits=0x8000)
    assert L.ls_token_scores_bwd(ctypes.byref(d), None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("temperature", [2.0 ** -120, 2.0 ** 120])
def test_temperatures_at_the_ends(temperature):
    """The coldest row is its largest logit alone; at the hottest all ids are alike, to fp32's rounding of log V."""
    import long_context_grpo_gb300 as ls
    x = torch.zeros(3, 500, dtype=torch.bfloat16, device="cuda")
    x[:, 7] = 2.0
    x[2, 9:] = float("-inf")
    ids = torch.tensor([7, 7, 7], dtype=torch.int32, device="cuda")
    r = ls.token_scores(x, ids, top=2, temperature=temperature)
    n = torch.tensor([500.0, 500.0, 9.0], dtype=torch.float64)
    want = torch.zeros(3, dtype=torch.float64) if temperature < 1 else -n.log()
    assert torch.allclose(r.logp.double().cpu(), want, rtol=2.0 ** -23, atol=0)
    assert torch.allclose(r.entropy.double().cpu(), -want, rtol=2.0 ** -20, atol=0)
    assert r.top_ids.cpu().tolist() == [[7, 0]] * 3
    assert not torch.isnan(r.top_logp).any()


def test_packed_descriptors_have_the_structures_layout():
    from long_context_grpo_gb300 import _lib as b
    from long_context_grpo_gb300 import _ops
    for s, D in ((_ops._SCORES, b.TokenScoresDesc), (_ops._SCORES_BWD, b.TokenScoresBwdDesc)):
        values = [float(i + 1) if k is ctypes.c_double else i + 1 for i, (_, k) in enumerate(D._fields_)]
        got = D.from_buffer_copy(s.pack(*values).ljust(ctypes.sizeof(D), b"\0"))
        assert [getattr(got, n) for n, _ in D._fields_] == values
