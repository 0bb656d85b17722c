"""Replay through a sliding window with the first tokens in sight, forward and backward, against float64.

Tolerances, element by element, from the roundings on the way: probabilities and dS are bf16 where they meet
the values, keys and queries (2^-8 of each), the output is bf16 (2^-8 of it, and Delta = sum dO O takes it
rounded), each gradient is rounded once more (2^-8; none for the fp32 accumulators); scores and sums in fp32
count as 2^-12 of every term."""
import pytest
import torch


def mask(P, R, window, sinks, device="cuda"):
    at = torch.arange(P + R, device=device)
    pos = P + torch.arange(R, device=device)[:, None]
    return (at <= pos) & ((at > pos - window) | (at < sinks))


def reference(q, k, v, d, seen, scale):
    """Values of o, lse, dq, dk, dv and their tolerances; k, v over prompt and response, float64."""
    R, Hq, D = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    q, k, v, d = (x.double() for x in (q, k, v, d))
    out = {n: torch.zeros_like(x) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    tol = {n: torch.zeros_like(x) for n, x in out.items()}
    out["lse"] = torch.zeros(R, Hq, dtype=torch.float64, device=q.device)
    e, f = 2.0 ** -8, 2.0 ** -12
    for h in range(Hq):
        kh, vh, qh, dh = k[:, h // g], v[:, h // g], q[:, h], d[:, h]
        s = (qh @ kh.T * scale).masked_fill(~seen, -float("inf"))
        out["lse"][:, h] = torch.logsumexp(s, 1)
        p = torch.softmax(s, 1)
        o, a = p @ vh, p @ vh.abs()
        out["o"][:, h] = o
        tol["o"][:, h] = e * (o.abs() + a) + f * a
        dp = dh @ vh.T
        ds = p * (dp - (dh * o).sum(1, keepdim=True))
        tds = e * ds.abs() + p * (dh.abs() * tol["o"][:, h]).sum(1, keepdim=True) + \
            f * p * (dh.abs() @ vh.abs().T + (dh.abs() * o.abs()).sum(1, keepdim=True))
        out["dq"][:, h] = scale * ds @ kh
        tol["dq"][:, h] = scale * tds @ kh.abs()
        out["dk"][:, h // g] += scale * ds.T @ qh
        tol["dk"][:, h // g] += scale * tds.T @ qh.abs()
        out["dv"][:, h // g] += p.T @ dh
        tol["dv"][:, h // g] += (e + f) * p.T @ dh.abs()
    tol["dq"] += e * (out["dq"].abs() + tol["dq"])
    return out, tol


def near(got, want, tol, rounded=True):
    """rounded: to bf16 at the end."""
    err = (got.double() - want).abs()
    room = tol + (2.0 ** -8 * (want.abs() + tol) if rounded else 0.0) + 1e-30
    assert bool((err <= room).all()), float((err / room).max())


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


SHAPES = [(1000, 77, 8, 2, 64), (130, 300, 5, 1, 128), (3, 50, 4, 4, 64), (1, 1, 2, 2, 128), (640, 129, 16, 1, 128),
          (300, 400, 6, 2, 128), (256, 256, 24, 3, 64)]
SIGHTS = [(1, 0), (2, 1), (100, 4), (128, 130), (300, 0), (5000, 7), (64, 500)]


@pytest.mark.gpu
@pytest.mark.parametrize("P,R,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("window,sinks", SIGHTS)
def test_against_float64(P, R, Hq, Hkv, D, window, sinks):
    import long_context_grpo_gb300 as ls
    g = torch.Generator(device="cuda").manual_seed(P + R + window)
    kp, vp, ks, vs = (randn(g, n, Hkv, D) for n in (P, P, R, R))
    q, d = randn(g, R, Hq, D), randn(g, R, Hq, D)
    acc = torch.empty(2, P, Hkv, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=Hq, window=window, sinks=sinks)
    seen = mask(P, R, window, sinks)
    want, tol = reference(q, torch.cat((kp, ks)), torch.cat((vp, vs)), d, seen, D ** -0.5)
    o, lse = p.fwd(q, ks, vs)
    near(o, want["o"], tol["o"] - 2.0 ** -8 * want["o"].abs())
    assert bool(((lse - want["lse"]).abs() <= 2 ** -20 * want["lse"].abs() + 2e-5).all())
    dq, dk, dv = p.bwd(q, ks, vs, o, lse, d)
    near(dq, want["dq"], tol["dq"], rounded=False)
    for x, n, a in ((dk, "dk", acc[0]), (dv, "dv", acc[1])):
        near(x, want[n][P:], tol[n][P:])
        near(a, want[n][:P], tol[n][:P], rounded=False)
        assert not a[~seen.any(0)[:P]].any()         # keys that nobody sees
    # the same bits again, on top of the accumulators
    again = p.bwd(q, ks, vs, o, lse, d)
    assert all(torch.equal(x, y) for x, y in zip(again, (dq, dk, dv)))
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 1], [0, 40, 41, 300], [0, 130, 400, 410, 500]])
@pytest.mark.parametrize("P,window,sinks", [(500, 200, 4), (500, 350, 0), (77, 1, 3), (2, 60, 40), (500, 1 << 40, 0)])
def test_packed_responses(cu, P, window, sinks):
    """Each as by itself; the prompt's accumulators hold their sum."""
    import long_context_grpo_gb300 as ls
    Hq, Hkv, D, T = 10, 2, 128, cu[-1]
    g = torch.Generator(device="cuda").manual_seed(P + T)
    kp, vp, ks, vs = (randn(g, n, Hkv, D) for n in (P, P, T, T))
    q, d = randn(g, T, Hq, D), randn(g, T, Hq, D)
    acc = torch.empty(2, P, Hkv, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=Hq, window=window, sinks=sinks)
    o, lse = p.fwd_packed(cu, q, ks, vs)
    grads = p.bwd_packed(cu, q, ks, vs, o, lse, d)
    total = acc.double()
    want = torch.zeros_like(total)
    tol = torch.zeros_like(total)
    for a, b in zip(cu, cu[1:]):
        i = slice(a, b)
        w, t = reference(q[i], torch.cat((kp, ks[i])), torch.cat((vp, vs[i])), d[i], mask(P, b - a, window, sinks), D ** -0.5)
        want += torch.stack((w["dk"][:P], w["dv"][:P]))
        tol += torch.stack((t["dk"][:P], t["dv"][:P]))
        one = p.fwd(q[i], ks[i], vs[i])
        assert torch.equal(one[0], o[i]) and torch.equal(one[1], lse[i])
        alone = p.bwd(q[i], ks[i], vs[i], o[i], lse[i], d[i])
        assert all(torch.equal(x, y[i]) for x, y in zip(alone, grads))
        near(o[i], w["o"], t["o"] - 2.0 ** -8 * w["o"].abs())
    near(total, want, tol, rounded=False)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("block", [37, 128, 200])
@pytest.mark.parametrize("window,sinks", [(150, 4), (1, 0), (33, 260), (1000, 0)])
def test_blockwise_replay(block, window, sinks):
    """A response replayed block by block in the prefix's own rows, as in one piece."""
    import long_context_grpo_gb300 as ls
    P, R, Hq, Hkv, D = 260, 300, 6, 2, 64
    g = torch.Generator(device="cuda").manual_seed(block)
    k, v = randn(g, P + R, Hkv, D), randn(g, P + R, Hkv, D)
    q, d = randn(g, R, Hq, D), randn(g, R, Hq, D)
    acc = torch.empty(2, P + R, Hkv, D, device="cuda")
    p = ls.Prefix(k, v, acc[0], acc[1], Hq=Hq, window=window, sinks=sinks)
    want, tol = reference(q, k, v, d, mask(P, R, window, sinks), D ** -0.5)
    o, lse, dq = torch.empty_like(q), torch.empty(R, Hq, device="cuda"), torch.empty_like(q)
    for t in range(0, R, block):
        i = slice(t, min(R, t + block))
        p.block_fwd(P + t, q[i], o=o[i], lse=lse[i])
    for t in range(0, R, block):
        i = slice(t, min(R, t + block))
        p.block_bwd(P + t, q[i], o[i], lse[i], d[i], dq=dq[i])
    near(o, want["o"], tol["o"] - 2.0 ** -8 * want["o"].abs())
    near(dq, want["dq"], tol["dq"], rounded=False)
    near(acc[0], want["dk"], tol["dk"], rounded=False)
    near(acc[1], want["dv"], tol["dv"], rounded=False)
    assert ls.device_status() == (0, 0)


@pytest.mark.gpu
def test_gradients_are_differences():
    """One value of a key, a value and a query moved each way: the change of sum d o, in float64 of the
    formula, is the gradient that the kernels give."""
    import long_context_grpo_gb300 as ls
    P, R, H, D, window, sinks = 40, 20, 2, 64, 9, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    kp, vp, ks, vs = (randn(g, n, 1, D) for n in (P, P, R, R))
    q, d = randn(g, R, H, D), randn(g, R, H, D)
    acc = torch.empty(2, P, 1, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=H, window=window, sinks=sinks)
    o, lse = p.fwd(q, ks, vs)
    dq, dk, dv = p.bwd(q, ks, vs, o, lse, d)
    seen = mask(P, R, window, sinks)

    def total(k, v, x):
        s = (torch.einsum("thd,jd->htj", x, k[:, 0]) * D ** -0.5).masked_fill(~seen, -float("inf"))
        return (torch.einsum("htj,jd->thd", torch.softmax(s, -1), v[:, 0]) * d.double()).sum()

    k, v, x = torch.cat((kp, ks)).double(), torch.cat((vp, vs)).double(), q.double()
    _, tol = reference(q, k, v, d, seen, D ** -0.5)
    for which, at, got, room in ((0, (1, 0, 3), acc[0][1, 0, 3], tol["dk"][1, 0, 3]),
                                 (0, (P - 2, 0, 7), acc[0][P - 2, 0, 7], tol["dk"][P - 2, 0, 7]),
                                 (0, (P + 5, 0, 1), dk[5, 0, 1], tol["dk"][P + 5, 0, 1]),
                                 (1, (P + 19, 0, 2), dv[19, 0, 2], tol["dv"][P + 19, 0, 2]),
                                 (2, (11, 1, 5), dq[11, 1, 5], tol["dq"][11, 1, 5])):
        args = [k, v, x]
        ends = []
        for step in (1e-4, -1e-4):
            moved = list(args)
            moved[which] = args[which].clone()
            moved[which][at] += step
            ends.append(total(*moved))
        slope = (ends[0] - ends[1]) / 2e-4
        assert abs(float(got) - float(slope)) <= float(room) + 2.0 ** -8 * abs(float(slope)) + 1e-6


@pytest.mark.gpu
def test_a_window_past_the_sequence_and_taken_away():
    import long_context_grpo_gb300 as ls
    P, R, Hq, Hkv, D = 500, 140, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    kp, vp, ks, vs = (randn(g, n, Hkv, D) for n in (P, P, R, R))
    q, d = randn(g, R, Hq, D), randn(g, R, Hq, D)
    acc = torch.empty(2, P, Hkv, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=Hq)
    plain = p.fwd(q, ks, vs)
    grads = p.bwd(q, ks, vs, *plain, d)
    for window, sinks in ((P + R, 0), (1 << 60, 1 << 60), (1, P + R)):
        p.set_window(window, sinks)
        one = p.fwd(q, ks, vs)
        assert torch.equal(one[0], plain[0]) and torch.equal(one[1], plain[1])
        assert all(torch.equal(x, y) for x, y in zip(p.bwd(q, ks, vs, *one, d), grads))
    p.set_window(7, 1)
    assert not torch.equal(p.fwd(q, ks, vs)[0], plain[0])
    with pytest.raises(ls.LongStrawError) as e:
        p.fwd_prompt_only(q)
    assert e.value.status == 2
    with pytest.raises(ls.LongStrawError) as e:
        p.bwd_prompt_only(q, *plain, d)
    assert e.value.status == 2
    for window, sinks in ((-1, 0), (0, 1), (5, -1)):
        with pytest.raises(ls.LongStrawError) as e:
            p.set_window(window, sinks)
        assert e.value.status == 1
    p.set_window(0)
    assert torch.equal(p.fwd(q, ks, vs)[0], plain[0])
    p.fwd_prompt_only(q)


@pytest.mark.gpu
def test_a_long_prompt_at_sampled_rows():
    """A response far behind a long prompt: the rows' own keys, and nothing written out of sight."""
    import long_context_grpo_gb300 as ls
    P, R, Hq, Hkv, D, window, sinks = 300001, 700, 8, 1, 128, 1111, 5
    g = torch.Generator(device="cuda").manual_seed(2)
    kp, vp, ks, vs = (randn(g, n, Hkv, D) for n in (P, P, R, R))
    q, d = randn(g, R, Hq, D), randn(g, R, Hq, D)
    acc = torch.empty(2, P, Hkv, D, device="cuda")
    p = ls.Prefix(kp, vp, acc[0], acc[1], Hq=Hq, window=window, sinks=sinks)
    o, lse = p.fwd(q, ks, vs)
    dq, dk, dv = p.bwd(q, ks, vs, o, lse, d)
    keep = torch.cat((torch.arange(sinks, device="cuda"), torch.arange(P - window + 1, P, device="cuda")))
    seen = mask(P, R, window, sinks)
    seen = torch.cat((seen[:, keep], seen[:, P:]), 1)
    want, tol = reference(q, torch.cat((kp[keep], ks)), torch.cat((vp[keep], vs)), d, seen, D ** -0.5)
    near(o, want["o"], tol["o"] - 2.0 ** -8 * want["o"].abs())
    near(dq, want["dq"], tol["dq"], rounded=False)
    for x, n, a in ((dk, "dk", acc[0]), (dv, "dv", acc[1])):
        near(x, want[n][len(keep):], tol[n][len(keep):])
        near(a[keep], want[n][:len(keep)], tol[n][:len(keep)], rounded=False)
        a[keep] = 0
        assert not a.any()


def test_refusals_without_a_gpu():
    from long_context_grpo_gb300 import build as lsbuild
    lsbuild.build()
    from long_context_grpo_gb300 import _lib as b
    assert b._lib().ls_prefix_set_window(None, 4, 0) == 3
