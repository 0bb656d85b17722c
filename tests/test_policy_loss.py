"""The policy loss with a KL term against its float64 definition: kinds of KL, odd and padded
vocabularies, left-out tokens, in-place gradients, far values, graphs.

Tolerances: dlogits are rounded to bf16 once (half a step, 2^-8 of the value) from fp32 products of
a probability that carries the fp32 exponential of an argument below 2^5 (2^-24 x 2^5 x log2 e, doubled:
2^-17 of the probability)."""
import numpy as np
import pytest
import torch

from oracle.policy import policy_loss as ref_loss


def _inputs(T, V, seed, masked=0.2, std=2.0, pad=0, noise=0.25):
    g = torch.Generator().manual_seed(seed)
    wide = (torch.randn(T, V + pad, generator=g) * std).to(torch.bfloat16)
    x = wide[:, :V]
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    logp = torch.log_softmax(x.double(), 1).gather(1, ids.long()[:, None])[:, 0]
    old = (logp + noise * torch.randn(T, generator=g)).float()
    ref = (logp + noise * torch.randn(T, generator=g)).float()
    adv = torch.randn(T, generator=g)
    w = (torch.rand(T, generator=g) >= masked).float() / T
    return wide, ids, old, ref, adv, w


def _near_border(o, eps_low, eps_high):
    # |d - log border| below the fp32 error of the log-sum-exp: either side is right
    return (np.abs(o["d"] - np.log1p(eps_high)) < 1e-6) | (np.abs(o["d"] - np.log1p(-eps_low)) < 1e-6)


def _check(r, o, w, eps_low, eps_high):
    ok = ~_near_border(o, eps_low, eps_high)
    assert np.array_equal(r.clip_mask.cpu().numpy().astype(bool)[ok], o["clip"][ok])
    np.testing.assert_allclose(r.logp.double().cpu().numpy(), o["logp"], rtol=2 ** -23, atol=2e-6)
    np.testing.assert_allclose(r.kl.double().cpu().numpy(), o["kl"], rtol=1e-5, atol=4e-6)
    assert abs(r.loss.item() - o["loss"]) <= 2 ** -23 * abs(o["loss"]) + 1e-5 * np.abs(o["terms"]).sum() + 1e-12
    got = r.dlogits.double().cpu().numpy()[ok]
    tol = np.abs(o["dlogits"]) * 2 ** -8 + (np.abs(o["g"])[:, None] * o["p"] + np.abs(o["dlogits"])) * 2 ** -16 + 1e-36
    assert (np.abs(got - o["dlogits"][ok]) <= tol[ok]).all()
    gone = np.asarray(w) == 0
    assert not r.dlogits.cpu()[torch.from_numpy(gone)].any()


SHAPES = [(1, 1, 0), (3, 7, 0), (5, 31, 1), (17, 1024, 0), (33, 1001, 3), (9, 4096, 8), (300, 264, 0), (4, 32000, 0),
          (3, 50257, 7), (2, 151936, 64), (2, 151937, 0), (1, 200000, 0), (700, 1000, 1), (300, 4093, 2), (5, 38001, 1), (1, 310001, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,pad", SHAPES)
@pytest.mark.parametrize("kl", ["none", "k1", "k2", "k3"])
def test_against_float64(T, V, pad, kl):
    import long_context_grpo_gb300 as ls
    wide, ids, old, ref, adv, w = _inputs(T, V, seed=T * 7 + V, pad=pad)
    w[0] = 1.0 / T
    x = wide.cuda()[:, :V]
    r = ls.policy_loss(x, ids.cuda(), old.cuda(), adv.cuda(), w.cuda(), eps_low=0.2, eps_high=0.28,
                       logp_ref=None if kl == "none" else ref.cuda(), beta=0.05, kl=kl)
    o = ref_loss(wide[:, :V], ids, old, adv, w, 0.2, 0.28, ref, 0.05 if kl != "none" else 0.0, kl)
    _check(r, o, w, 0.2, 0.28)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,pad", [(20000, 600, 1), (9000, 3000, 0), (12000, 5000, 1), (9000, 8000, 0), (5000, 17001, 0),
                                     (4000, 32000, 8), (3000, 45000, 1), (1500, 75000, 0), (1200, 100000, 64),
                                     (1000, 151936, 1), (700, 300000, 0)])
@pytest.mark.parametrize("masked", [0.0, 0.5, 0.97])
def test_many_rows_a_block_with_tokens_left_out(T, V, pad, masked):
    """Every row of long runs against float64 on the GPU, twice: rows that are left out let some of a
    block's warps run ahead of others."""
    import long_context_grpo_gb300 as ls
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = (torch.randn(T, V + pad, generator=g, device="cuda", dtype=torch.bfloat16) * 2)[:, :V]
    ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    lp = ls.token_logp(x.contiguous(), ids)
    old, ref = (lp + 0.25 * torch.randn(T, generator=g, device="cuda") for _ in range(2))
    adv = torch.randn(T, generator=g, device="cuda")
    w = (torch.rand(T, generator=g, device="cuda") >= masked).float() / T
    call = lambda: ls.policy_loss(x, ids, old, adv, w, eps_low=0.2, eps_high=0.28, logp_ref=ref, beta=0.05, kl="k2")  # noqa: E731
    r, again = call(), call()
    assert all(torch.equal(a, b) for a, b in zip(r, again)) and ls.device_status() == (0, 0)
    loss = 0.0
    for a in range(0, T, 500):
        i = slice(a, a + 500)
        soft = torch.log_softmax(x[i].double(), 1)
        y = ids[i].long()[:, None]
        logp = soft.gather(1, y)[:, 0]
        d, A, used = logp - old[i].double(), adv[i].double(), w[i] != 0
        rho, kd = d.exp(), logp - ref[i].double()
        clip = ((A > 0) & (d > np.log(1.28))) | ((A < 0) & (d < np.log(0.8)))
        gt = torch.where(used, w[i].double() * (0.05 * kd - torch.where(clip, 0.0, rho * A)), 0.0)
        surr = torch.where(clip, rho.clamp(0.8, 1.28) * A, rho * A)
        loss += float((w[i].double() * (0.05 * kd * kd / 2 - surr)).sum())
        near = ((d - np.log(1.28)).abs() < 1e-6) | ((d - np.log(0.8)).abs() < 1e-6)
        p = soft.exp_()
        want = -gt[:, None] * p
        want.scatter_add_(1, y, gt[:, None])
        # g is the difference of two fp32 terms, each within 2^-21 of itself (an exponential, two
        # products); where they cancel that is all of g's error, and it scales the whole row
        off = w[i].double() * (0.05 * kd.abs() + (rho * A).abs()) * 2 ** -20
        hot = torch.zeros_like(p).scatter_(1, y, 1.0)
        tol = want.abs() * (2 ** -8 + 2 ** -16) + gt.abs()[:, None] * p * 2 ** -16 + off[:, None] * (p + hot) * 1.01 + 1e-36
        assert bool((((r.dlogits[i].double() - want).abs() <= tol).all(1) | near).all())
        assert torch.equal(r.clip_mask[i].bool() | near, (clip & used) | near)
        assert bool(((r.logp[i].double() - logp * used).abs() <= 2e-6).all())
    assert abs(r.loss.item() - loss) <= 1e-5 * float((w.double() * rho.max()).sum()) + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("V,pad", [(1024, 0), (1000, 16), (333, 2)])
def test_gradient_in_place_of_the_logits_and_untouched_padding(V, pad):
    import long_context_grpo_gb300 as ls
    wide, ids, old, ref, adv, w = _inputs(40, V, seed=3, pad=pad)
    args = (ids.cuda(), old.cuda(), adv.cuda(), w.cuda())
    a = ls.policy_loss(wide.cuda()[:, :V], *args, logp_ref=ref.cuda(), beta=0.1, kl="k3")
    buf = wide.cuda()
    b = ls.policy_loss(buf[:, :V], *args, logp_ref=ref.cuda(), beta=0.1, kl="k3", dlogits=buf[:, :V])
    assert torch.equal(a.dlogits, buf[:, :V]) and torch.equal(a.loss, b.loss)
    assert torch.equal(buf[:, V:].cpu(), wide[:, V:])


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1024, 1001, 151936])
def test_left_out_tokens_and_bad_ids(V):
    """Weight 0: the row may hold anything; an id outside the vocabulary is reported."""
    import long_context_grpo_gb300 as ls
    wide, ids, old, ref, adv, w = _inputs(6, V, seed=5, masked=0.0)
    w[1], w[4] = 0.0, 0.0
    wide[1], old[1], ref[4], ids[4] = float("nan"), float("inf"), float("nan"), -7
    r = ls.policy_loss(wide.cuda(), ids.cuda(), old.cuda(), adv.cuda(), w.cuda(), logp_ref=ref.cuda(), beta=0.1, kl="k3")
    o = ref_loss(wide, ids, old, adv, w, 0.2, 0.2, ref, 0.1, "k3")
    _check(r, o, w, 0.2, 0.2)
    assert ls.device_status() == (0, 0)
    ids[2] = V
    r = ls.policy_loss(wide.cuda(), ids.cuda(), old.cuda(), adv.cuda(), w.cuda(), logp_ref=ref.cuda(), beta=0.1, kl="k3")
    o = ref_loss(wide, ids, old, adv, w, 0.2, 0.2, ref, 0.1, "k3")
    assert abs(r.loss.item() - o["loss"]) < 1e-5
    assert not r.dlogits[2].any() and r.logp[2] == 0 and r.clip_mask[2] == 0
    assert ls.device_status() == (7, 2)
    all_out = ls.policy_loss(wide.cuda(), ids.cuda(), old.cuda(), adv.cuda(), 0 * w.cuda())
    assert all_out.loss.item() == 0 and not all_out.dlogits.any()
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [512, 509])
def test_masked_logits_and_far_values(V):
    """-inf logits have probability 0; logits hundreds apart; the type's lowest value."""
    import long_context_grpo_gb300 as ls
    wide, ids, old, ref, adv, w = _inputs(8, V, seed=9, masked=0.0)
    wide[0, 5:] = float("-inf")
    ids[0] = 3
    wide[1] = torch.finfo(torch.bfloat16).min
    wide[1, 2] = 0.0
    ids[1] = 2
    wide[2, 7] = 300.0
    ids[2] = 7
    wide[3] = -300.0
    wide[4, : V - 1] = float("-inf")
    ids[4] = V - 1
    for t in range(5):
        logp = torch.log_softmax(wide[t].double(), 0)[ids[t].long()]
        old[t], ref[t] = logp + 0.1, logp - 0.1
    r = ls.policy_loss(wide.cuda(), ids.cuda(), old.cuda(), adv.cuda(), w.cuda(), logp_ref=ref.cuda(), beta=0.1, kl="k3")
    o = ref_loss(wide, ids, old, adv, w, 0.2, 0.2, ref, 0.1, "k3")
    _check(r, o, w, 0.2, 0.2)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_poisoned_row_spoils_only_itself_and_the_loss(bad):
    import long_context_grpo_gb300 as ls
    wide, ids, old, ref, adv, w = _inputs(5, 4096, seed=2, masked=0.0)
    wide[3, 1234] = bad
    r = ls.policy_loss(wide.cuda(), ids.cuda(), old.cuda(), adv.cuda(), w.cuda())
    assert torch.isnan(r.loss).all() and torch.isnan(r.dlogits[3].float()).any() and torch.isnan(r.logp[3])
    keep = torch.tensor([0, 1, 2, 4])
    o = ref_loss(wide[keep], ids[keep], old[keep], adv[keep], w[keep], 0.2, 0.2)
    got = r.dlogits.cpu()[keep].double().numpy()
    assert np.linalg.norm(got - o["dlogits"]) <= 2 ** -8 * np.linalg.norm(o["dlogits"])


@pytest.mark.gpu
def test_same_as_the_loss_without_a_kl_term():
    """Weights 1/(G R), one advantage, no KL: the existing loss call's values."""
    import long_context_grpo_gb300 as ls
    wide, ids, old, _, _, _ = _inputs(200, 4096, seed=4)
    x, i, o = wide.cuda(), ids.cuda(), old.cuda()
    acc = torch.zeros(1, dtype=torch.float64, device="cuda")
    dl, mask, logp = ls.grpo_loss(x, i, o, -0.7, 0.2, 4, acc)
    r = ls.policy_loss(x, i, o, torch.full((200,), -0.7, device="cuda"), torch.full((200,), 1 / 800, device="cuda"))
    assert torch.equal(mask, r.clip_mask) and torch.allclose(logp, r.logp, atol=2e-6, rtol=0)
    assert abs(acc.item() - r.loss.item()) <= 1e-6 * abs(acc.item())
    # two values a rounding step apart at most
    assert ((dl.double() - r.dlogits.double()).abs() <= 2 ** -7 * dl.double().abs() + 1e-36).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
def test_gradient_against_differences(kl):
    """Central differences of the loss by one logit, a whole bf16 step each way."""
    import long_context_grpo_gb300 as ls
    T, V = 6, 24
    wide, ids, old, ref, adv, w = _inputs(T, V, seed=8, masked=0.0, std=1.0, noise=0.1)
    run = lambda x: ls.policy_loss(x.cuda(), ids.cuda(), old.cuda(), adv.cuda(), w.cuda(), logp_ref=ref.cuda(),  # noqa: E731
                                   beta=0.5, kl=kl)
    base = run(wide)
    for t in range(T):
        if base.clip_mask[t]:
            continue
        v = int(ids[t]) if t % 2 else (int(ids[t]) + 1) % V
        h = 2.0 ** -4
        x0 = wide.clone()
        x0[t, v] = (wide[t, v].float() / h).round() * h        # h-spaced points are exact in bf16
        up, down = x0.clone(), x0.clone()
        up[t, v], down[t, v] = x0[t, v] + h, x0[t, v] - h
        num = ref_loss(up, ids, old, adv, w, 0.2, 0.2, ref, 0.5, kl)
        den = ref_loss(down, ids, old, adv, w, 0.2, 0.2, ref, 0.5, kl)
        if num["clip"][t] or den["clip"][t]:
            continue
        ours = (run(up).loss.item() - run(down).loss.item()) / (2 * h)
        g = run(x0).dlogits[t, v].double().item()
        # the third derivative's h^2 / 6 (all factors below 4 |w|), bf16's half step, fp32 losses
        assert abs(ours - g) <= 4 / T * h * h + 2 ** -8 * abs(g) + 2 ** -22 / h


@pytest.mark.gpu
def test_two_graphs_of_one_shape_and_repeatability():
    import long_context_grpo_gb300 as ls
    wide, ids, old, ref, adv, w = (t.cuda() for t in _inputs(64, 32000, seed=1))
    ws = torch.empty(ls.policy_loss_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    call = lambda x: ls.policy_loss(x, ids, old, adv, w, logp_ref=ref, beta=0.1, kl="k3", workspace=ws)  # noqa: E731
    x2 = wide.flip(0).contiguous()
    want = [call(wide), call(x2)]
    graphs, outs = [], []
    for x in (wide, x2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:            # they share the workspace, in stream order
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


INF = float("inf")


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,pad", [(6, 500, 0), (6, 1001, 3), (6, 5000, 0), (6, 38001, 1), (6, 310001, 0)])
@pytest.mark.parametrize("kl", ["none", "k1", "k2", "k3"])
@pytest.mark.parametrize("what", ["sampled", "old -inf", "old +inf", "ref -inf", "ref +inf"])
def test_infinite_log_probabilities(T, V, pad, kl, what):
    """A sampled token whose logit is -inf, and infinite log-probabilities given, with both signs of A:
    infinities and NaN are where the float64 definition has them, finite outputs have its values."""
    import long_context_grpo_gb300 as ls
    if "ref" in what and kl == "none":
        pytest.skip("no reference without a KL term")
    wide, ids, old, ref, adv, w = _inputs(T, V, seed=V, masked=0.0, pad=pad)
    adv = adv.abs() + 0.1
    adv[1::2] *= -1                                    # rows 0, 2, .. A > 0; 1, 3, .. A < 0
    for t in (2, 3):
        if what == "sampled":
            wide[t, int(ids[t])] = -INF
        else:
            (old if "old" in what else ref)[t] = -INF if "-" in what else INF
    beta = 0.0 if kl == "none" else 0.05
    with np.errstate(all="ignore"):
        o = ref_loss(wide[:, :V], ids, old, adv, w, 0.2, 0.28, ref, beta, kl)
    r = ls.policy_loss(wide.cuda()[:, :V], ids.cuda(), old.cuda(), adv.cuda(), w.cuda(), eps_low=0.2, eps_high=0.28,
                       logp_ref=None if kl == "none" else ref.cuda(), beta=beta, kl=kl)
    assert np.array_equal(r.clip_mask.cpu().numpy().astype(bool), o["clip"])

    def same(got, want, tol):
        got, want = (np.asarray(x, dtype=np.float64) for x in (got.double().cpu().numpy(), want))
        fin = np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)])
        assert (np.abs(got[fin] - want[fin]) <= tol[fin]).all()

    with np.errstate(all="ignore"):
        same(r.logp, o["logp"], 2 ** -23 * np.abs(o["logp"]) + 2e-6)
        same(r.kl, o["kl"], 1e-5 * np.abs(o["kl"]) + 4e-6)
        same(r.loss, [o["loss"]], np.array([1e-5 * np.abs(o["terms"]).sum() + 1e-12]))
        # (as in test_many_rows_a_block_with_tokens_left_out: the fp32 terms that g is the difference of)
        A, rw = adv.double().numpy(), w.double().numpy()
        rk = o["logp"] - ref.double().numpy()
        slope = {"none": np.zeros(T), "k1": np.ones(T), "k2": rk, "k3": -np.expm1(-rk)}[kl]
        off = rw * (beta * np.abs(slope) + np.where(o["clip"], 0.0, np.exp(o["d"]) * np.abs(A))) * 2 ** -20
        hot = np.zeros_like(o["p"])
        hot[np.arange(T), ids.numpy()] = 1.0
        want = o["g"][:, None] * (hot - o["p"])       # as one product: -g p + g is inf - inf at a sampled -inf logit
        same(r.dlogits, want, np.abs(want) * (2 ** -8 + 2 ** -16) + np.abs(o["g"])[:, None] * o["p"] * 2 ** -16 +
             off[:, None] * (o["p"] + hot) * 1.01 + 1e-36)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,pad", [(8, 500, 0), (8, 1001, 3), (8, 5001, 0), (8, 38001, 1), (4, 310001, 0)])
@pytest.mark.parametrize("size", [1e4, 1e5, 3e7, 2e38])
def test_logits_far_from_zero(T, V, pad, size):
    """Equal logits far from zero share the probability; the rest, whole steps of bf16 below, have none."""
    import long_context_grpo_gb300 as ls
    g = torch.Generator().manual_seed(V)
    wide = (torch.randn(T, V + pad, generator=g) * 0.01 - 1).clamp(max=-0.9).mul(size).to(torch.bfloat16)
    wide[T // 2:] = (wide[T // 2:].float() + size).to(torch.bfloat16)       # these rows around zero
    top = torch.rand(T, V + pad, generator=g) < 0.02
    top[:, V // 3] = True
    level = torch.tensor([size, -size / 4] * (T // 2)).to(torch.bfloat16)[:, None]
    level[T // 2:] = torch.tensor(size).to(torch.bfloat16)
    wide = torch.where(top, level, wide)
    ids = torch.stack([top[t, :V].nonzero()[0, 0] for t in range(T)]).int()
    x = wide[:, :V]
    logp = torch.log_softmax(x.double(), 1).gather(1, ids.long()[:, None])[:, 0]
    old, adv, w = (logp + 0.05).float(), torch.randn(T, generator=g), torch.full((T,), 1.0 / T)
    o = ref_loss(x, ids, old, adv, w, 0.2, 0.2)
    assert np.isfinite(o["dlogits"]).all() and (np.abs(o["dlogits"]) > 0).sum() > T
    r = ls.policy_loss(wide.cuda()[:, :V], ids.cuda(), old.cuda(), adv.cuda(), w.cuda())
    _check(r, o, w, 0.2, 0.2)
