"""A group's step of a model with head norms and windowed layers, as a user runs it: the prompt captured into pages
through the window, responses decoded and scored with alternatives, replayed for the gradient, which goes back
through the attention, the rotation and the norms -- against float64."""
import numpy as np
import pytest
import torch

from oracle.cache import attend
from oracle.norm_rope import norm_rope, norm_rope_grad
from oracle.scores import scores, scores_grad
from test_replay_window import mask, near, reference

EPS = 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("ps,layout,window,sinks", [(16, "NHD", 40, 4), (64, "HND", 130, 0), (32, "NHD", 1000, 0)])
def test_capture_decode_score_replay_gradient(ps, layout, window, sinks):
    import long_context_grpo_gb300 as ls
    G, Hq, Hkv, D, V, P, R = 3, 8, 2, 64, 1000, 150, 20
    pages, rows, width = 60, 6, 16
    inner = (ps, Hkv, D) if layout == "NHD" else (Hkv, ps, D)
    both = torch.full((pages, 2, *inner), float("nan"), device="cuda").to(torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    new = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    c = ls.PagedCache(both[:, 0], both[:, 1], new(rows, width), new(rows), new(pages), Hq=Hq, layout=layout)
    c.reset()
    f, factor = ls.rope_freqs(D, 1e6, "ramp", 4.0, 64)
    bf = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    wq, wk = 1.0 + 0.3 * torch.randn(D, device="cuda"), 1.0 + 0.3 * torch.randn(D, device="cuda")
    on_the_way = dict(inv_freq=f, attn_factor=factor, q_weight=wq, k_weight=wk, norm_eps=EPS)
    sight = dict(window=window, sinks=sinks)
    # projections before their norms: the prompt's, and every response's
    Qp, Kp, Vp = 3.0 * bf(P, Hq, D), 3.0 * bf(P, Hkv, D), bf(P, Hkv, D)
    Q, K, Vr = 3.0 * bf(G, R, Hq, D), 3.0 * bf(G, R, Hkv, D), bf(G, R, Hkv, D)
    captured = []
    for a in range(0, P, 64):
        n = min(64, P - a)
        c.extend(i32(0), i32(n))
        cu = i32(0, n)
        q, _ = c.append(Kp[a:a + n], Vp[a:a + n], cu, rows=i32(0), q=Qp[a:a + n], **on_the_way)
        captured.append(c.attn(q, cu, max_new=64, max_len=P, rows=i32(0), **sight))
    children = i32(*range(1, 1 + G))
    c.fork(i32(*([0] * G)), children)
    cu = i32(*range(G + 1))
    decoded = []
    for t in range(R):
        c.extend(children, i32(*([1] * G)))
        q, _ = c.append(K[:, t].contiguous(), Vr[:, t].contiguous(), cu, rows=children, q=Q[:, t].contiguous(), **on_the_way)
        decoded.append(c.attn(q, cu, max_new=1, max_len=P + R, rows=children, **sight))

    # normed and turned in float64 and rounded once: a value on a rounding border may be one step off
    dbl = lambda x: x.double().cpu().numpy()  # noqa: E731
    turn = lambda x, w, pos: torch.from_numpy(  # noqa: E731
        norm_rope(dbl(x), dbl(w), EPS, pos, f.numpy(), False, factor)).to(torch.bfloat16).cuda()

    def close(got, q, k, v):
        o, lse, a = attend(dbl(q), dbl(k), dbl(v), D ** -0.5, window, sinks)
        assert (np.abs(dbl(got[0]) - o) <= 2 ** -8 * (np.abs(o) + a) + 2 ** -5 * a).all()
        assert np.abs(dbl(got[1]) - lse).max() <= 2 ** -5

    kp, qp = turn(Kp, wk, np.arange(P)), turn(Qp, wq, np.arange(P))
    for i, a in enumerate(range(0, P, 64)):
        n = min(64, P - a)
        close(captured[i], qp[a:a + n], kp[:a + n], Vp[:a + n])
    for b in range(G):
        kr, qr = turn(K[b], wk, P + np.arange(R)), turn(Q[b], wq, P + np.arange(R))
        for t in (0, 7, R - 1):
            o, lse = decoded[t]
            close((o[b:b + 1], lse[b:b + 1]), qr[t:t + 1], torch.cat((kp, kr[:t + 1])), torch.cat((Vp, Vr[b, :t + 1])))

    # scores of the responses with alternatives, and the gradient that a policy's loss sends back
    T = G * R
    logits = (torch.randn(T, V, device="cuda") * 2).to(torch.bfloat16)
    ids = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    s = ls.token_scores(logits, ids, top=4, temperature=0.9)
    lp, lse, ent, order, _ = scores(dbl(logits), ids.cpu().numpy(), 4, 0.9)
    assert np.array_equal(s.top_ids.cpu().numpy(), order) and np.abs(dbl(s.entropy) - ent).max() <= 2.0 ** -17
    dl, de = torch.randn(T, device="cuda") / T, torch.full((T,), -0.01 / T, device="cuda")
    d = ls.token_scores_bwd(logits, ids, s.logp, s.lse, s.entropy, dl, de, temperature=0.9)
    want = scores_grad(dbl(logits), ids.cpu().numpy(), dbl(dl), dbl(de), 0.9)
    assert np.linalg.norm(dbl(d) - want) <= 2 ** -8 * np.linalg.norm(want)

    # the replay of each response against the resident prompt, and back through rotation and norm
    kpk, _ = ls.norm_rope(None, Kp, None, wk, f, attn_factor=factor, eps=EPS)[::-1]
    acc = torch.empty(2, P, Hkv, D, device="cuda")
    p = ls.Prefix(kpk, Vp, acc[0], acc[1], Hq=Hq, **sight)
    total, room = np.zeros((2, P, Hkv, D)), torch.zeros(2, P, Hkv, D, dtype=torch.float64, device="cuda")
    for b in range(G):
        q, k = ls.norm_rope(Q[b], K[b], wq, wk, f, pos0=P, attn_factor=factor, eps=EPS)
        o, l = p.fwd(q, k, Vr[b])
        for t in (0, R - 1):        # the replay's forward is the decoding's
            err = (o[t].double() - decoded[t][0][b].double()).abs()
            assert bool((err <= 2 ** -7 * o[t].double().abs() + 2 ** -6 * o.double().abs().amax()).all())
        do = bf(R, Hq, D)
        dq, dk, dv = p.bwd(q, k, Vr[b], o, l, do)
        w, tol = reference(q, torch.cat((kpk, k)), torch.cat((Vp, Vr[b])), do, mask(P, R, window, sinks), D ** -0.5)
        near(dq, w["dq"], tol["dq"], rounded=False)
        near(dk, w["dk"][P:], tol["dk"][P:])
        near(dv, w["dv"][P:], tol["dv"][P:])
        total += np.stack((dbl(w["dk"][:P]), dbl(w["dv"][:P])))
        room += torch.stack((tol["dk"][:P], tol["dv"][:P]))
        r = ls.norm_rope_bwd(dq, dk, Q[b], K[b], wq, wk, f, pos0=P, attn_factor=factor, eps=EPS)
        for got, gw, dy, x, weight in ((r.dq, r.dq_weight, dq, Q[b], wq), (r.dk, r.dk_weight, dk, K[b], wk)):
            dx, dw, size, terms = norm_rope_grad(dbl(dy), dbl(x), dbl(weight), EPS, P + np.arange(R), f.numpy(), False, factor)
            assert (np.abs(dbl(got) - dx) <= 2 ** -8 * np.abs(dx) + 2 ** -16 * size.max(-1, keepdims=True)).all()
            assert (np.abs(dbl(gw) - dw) <= 2 ** -16 * terms).all()
    near(acc, torch.from_numpy(total).cuda(), room, rounded=False)
    c.free(i32(*range(1 + G)))
    assert not c.refcount.any() and ls.device_status() == (0, 0)
