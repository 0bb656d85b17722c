"""A group step as a user runs it: the prompt captured into pages chunk by chunk, forked to the
responses, tokens decoded, responses scored, the policy loss with the reference's KL term and
its gradient, rows retired and the pool compacted -- against float64."""
import numpy as np
import pytest
import torch

from oracle.cache import attend
from oracle.policy import policy_loss as ref_loss
from oracle.rope import rope as ref_rope


@pytest.mark.gpu
@pytest.mark.parametrize("ps,layout", [(16, "NHD"), (64, "HND")])
def test_capture_fork_decode_score_loss_retire(ps, layout):
    import long_context_grpo_gb300 as ls
    G, Hq, Hkv, D, V, P, R = 4, 8, 2, 64, 1000, 150, 5
    pages, rows, width = 80, 12, 16
    inner = (ps, Hkv, D) if layout == "NHD" else (Hkv, ps, D)
    both = torch.randn(pages, 2, *inner, device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    c = ls.PagedCache(both[:, 0], both[:, 1], new(rows, width), new(rows), new(pages), Hq=Hq, layout=layout)
    c.reset()
    f, factor = ls.rope_freqs(D, 1e6, "ramp", 4.0, 64)
    bf = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    Qp, Kp, Vp = bf(P, Hq, D), bf(P, Hkv, D), bf(P, Hkv, D)
    # row 0 was someone else's: the prompt's pages start behind it
    c.extend(i32(0), i32(3 * ps))
    outs = []
    for a in range(0, P, 64):
        n = min(64, P - a)
        c.extend(i32(1), i32(n))
        cu = i32(0, n)
        q, _ = c.append(Kp[a:a + n], Vp[a:a + n], cu, rows=i32(1), q=Qp[a:a + n], inv_freq=f, attn_factor=factor)
        outs.append(c.attn(q, cu, max_new=64, max_len=P, rows=i32(1)))
    c.free(i32(0))
    c.compact()
    children = i32(*range(2, 2 + G))
    c.fork(i32(*([1] * G)), children)
    shared = i32(P // ps * ps)
    Q, K, Vv = bf(R, G, Hq, D), bf(R, G, Hkv, D), bf(R, G, Hkv, D)
    cu = i32(*range(G + 1))
    for t in range(R):
        c.extend(children, i32(*([1] * G)))
        q, _ = c.append(K[t], Vv[t], cu, rows=children, q=Q[t], inv_freq=f, attn_factor=factor)
        outs.append(c.attn(q, cu, max_new=1, max_len=P + R, rows=children, group=G, shared_len=shared))
    # the float64 story of the same tokens; rotated values as the cache holds them, in bf16
    turn = lambda x, pos: torch.from_numpy(ref_rope(x.double().cpu().numpy(), pos, f.numpy(), False, factor)).to(torch.bfloat16)  # noqa: E731
    dbl = lambda x: x.double().cpu().numpy()  # noqa: E731
    s = D ** -0.5

    def close(got, want):
        o, lse, a = want
        # a rotated value that lies on a rounding border may be one step off: 2^-7 of a score's parts
        assert (np.abs(dbl(got[0]) - o) <= 2 ** -8 * (np.abs(o) + a) + 2 ** -6 * a).all()
        assert np.abs(dbl(got[1]) - lse).max() <= 2 ** -6

    kp, qp, vp = dbl(turn(Kp, np.arange(P))), dbl(turn(Qp, np.arange(P))), dbl(Vp)
    for i, a in enumerate(range(0, P, 64)):
        n = min(64, P - a)
        close(outs[i], attend(qp[a:a + n], kp[:a + n], vp[:a + n], s))
    for b in range(G):
        kr, qr = (dbl(turn(x[:, b], P + np.arange(R))) for x in (K, Q))
        k, v = np.concatenate([kp, kr]), np.concatenate([vp, dbl(Vv[:, b])])
        for t in range(R):
            o, lse = outs[-R + t]
            close((o[b:b + 1], lse[b:b + 1]), attend(qr[t:t + 1], k[:P + t + 1], v[:P + t + 1], s))
    # scoring and the loss: current, old and reference logits of the G R tokens
    T = G * R
    cur, old, ref = ((torch.randn(T, V, device="cuda") * 0.3).to(torch.bfloat16) for _ in range(3))
    old, ref = (cur.float() + 0.1 * old.float()).to(torch.bfloat16), (cur.float() + 0.1 * ref.float()).to(torch.bfloat16)
    ids = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    lo, lr = ls.token_logp(old, ids), ls.token_logp(ref, ids)
    adv = torch.tensor([1.0, -1.0, 0.5, -0.5], device="cuda").repeat_interleave(R)
    w = torch.full((T,), 1.0 / T, device="cuda")
    r = ls.policy_loss(cur, ids, lo, adv, w, eps_low=0.2, eps_high=0.28, logp_ref=lr, beta=0.04, kl="k3")
    o = ref_loss(cur, ids, lo, adv, w, 0.2, 0.28, lr, 0.04, "k3")
    assert abs(r.loss.item() - o["loss"]) <= 1e-5 * np.abs(o["terms"]).sum()
    assert np.linalg.norm(dbl(r.dlogits) - o["dlogits"]) <= 2 ** -8 * np.linalg.norm(o["dlogits"])
    # the gradient through the rotation of the last token's keys
    dk = bf(G, Hkv, D)
    _, dx = ls.rope(None, dk, f, pos0=P + R - 1, attn_factor=factor, inverse=True)
    want = ref_rope(dbl(dk), P + R - 1 + np.arange(G), f.numpy(), False, factor, True)
    assert (np.abs(dbl(dx) - want) <= 2 ** -8 * np.abs(want) + 2 ** -17).all()
    c.free(children)
    c.free(i32(1))
    assert not c.refcount.any() and not c.seq_len.any()
    assert ls.device_status() == (0, 0)
