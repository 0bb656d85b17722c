"""Tensors of more than 2^31 elements: the last rows come out as those of a call on them alone."""
import numpy as np
import pytest
import torch

from oracle.cache import attend


@pytest.mark.gpu
@pytest.mark.parametrize("T,V", [(14500, 151936), (2200000, 1000), (7000, 310000)])
def test_policy_loss(T, V):
    import long_context_grpo_gb300 as ls
    assert T * V > 2 ** 31
    x = torch.empty(T, V, dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.randint(0, V, (T,), dtype=torch.int32, device="cuda")
    old, A, w = torch.full((T,), -8.0, device="cuda"), torch.randn(T, device="cuda"), torch.rand(T, device="cuda") / T
    r = ls.policy_loss(x, ids, old, A, w, logp_ref=old, beta=0.1, kl="k2")
    n = 40
    tail = ls.policy_loss(x[-n:], ids[-n:], old[-n:], A[-n:], w[-n:], logp_ref=old[-n:], beta=0.1, kl="k2")
    for a, b in ((r.dlogits, tail.dlogits), (r.logp, tail.logp), (r.kl, tail.kl), (r.clip_mask, tail.clip_mask)):
        assert torch.equal(a[-n:], b)
    # the sum of the tokens' terms, from the outputs in fp64: each of those is rounded once to fp32
    d = r.logp.double() - old.double()
    rho, Ad = d.exp(), A.double()
    surr = torch.minimum(rho * Ad, rho.clamp(0.8, 1.2) * Ad)
    terms = w.double() * (0.1 * r.kl.double() - surr)
    size = w.double() * (0.1 * r.kl.double() + surr.abs() * (1 + r.logp.double().abs()))
    assert abs(float(r.loss) - float(terms.sum())) <= 2 ** -23 * float(size.sum())
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_rope(inter):
    import long_context_grpo_gb300 as ls
    T, H, D = 140000, 120, 128
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda").normal_()
    assert q.numel() > 2 ** 31
    f, _ = ls.rope_freqs(D)
    k = q[:, :8]
    n = 50
    tail = ls.rope(q[-n:], k[-n:], f, pos0=T - n, interleaved=inter)
    out, ko = ls.rope(q, k, f, interleaved=inter)
    assert torch.equal(out[-n:], tail[0]) and torch.equal(ko[-n:], tail[1])
    ls.rope(q, None, f, interleaved=inter, q_out=q)
    assert torch.equal(q, out)


@pytest.mark.gpu
def test_cache_attention_and_append():
    import long_context_grpo_gb300 as ls
    Hq, Hkv, D, ps, S, n = 256, 16, 128, 64, 67, 1000
    lens = [n] * S + [90]
    T = sum(lens)
    assert T * Hq * D > 2 ** 31
    per = -(-n // ps)
    k = torch.zeros((S + 1) * per, 2, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange((S + 1) * per, dtype=torch.int32, device="cuda").view(S + 1, per)
    c = ls.PagedCache(k[:, 0], k[:, 1], table, i32(lens), torch.ones((S + 1) * per, dtype=torch.int32, device="cuda"), Hq=Hq)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda").normal_()
    kn, vn = (torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    cu = i32([0] + list(np.cumsum(lens)))
    f, _ = ls.rope_freqs(D)
    qr, _ = c.append(kn, vn, cu, q=q, inv_freq=f)
    tail = ls.rope(q[-90:], kn[-90:], f)
    assert torch.equal(qr[-90:], tail[0])
    assert torch.equal(k[S * per:, 0].reshape(-1, Hkv, D)[:90], tail[1])
    o, lse = c.attn(qr, cu, max_new=n, max_len=n)
    dbl = lambda t: t.double().cpu().numpy()  # noqa: E731
    wo, wl, wa = attend(dbl(qr[-90:]), dbl(tail[1]), dbl(vn[-90:]), D ** -0.5)
    assert (np.abs(dbl(o[-90:]) - wo) <= 2 ** -8 * (np.abs(wo) + wa) + 2 ** -14 * wa + 1e-30).all()
    assert (np.abs(dbl(lse[-90:]) - wl) <= 2 ** -20 * np.abs(wl) + 2e-5).all()
    assert ls.device_status() == (0, 0)
