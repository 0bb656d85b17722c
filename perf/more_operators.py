"""Measured cases of the operators that a group of a model with head norms and windowed layers adds
to the replay's: norms of queries and keys with the rotation in the same pass, attention through a
sliding window with the first tokens kept in sight (over the cache's pages, and in the replay with
its gradient), and the scores of given tokens.

Every case is a dict of plain values.  `run` computes one pass, either with the library's entry
points (`own`) or in elementary torch operations in 32 bits (64 for angles of far positions and long
sums).  `exact` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one new token of each response of a group: its queries and keys normed and turned (latency)
        dict(name="norm_token", op="norm", T=8, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, scaling="none",
             pos0=32768, fused=False, wide=False, mix=1),
        # a prompt's chunk at a far position, out of the rows of a fused projection
        dict(name="norm_chunk", op="norm", T=8192, Hq=40, Hkv=8, D=128, rot=128, interleaved=False, scaling="ramp",
             pos0=262144, fused=True, wide=False, mix=2),
        # the gradient through norms and a partial interleaved rotation of an odd-sized response
        dict(name="norm_grad", op="norm_grad", T=3001, Hq=40, Hkv=8, D=128, rot=64, interleaved=True, scaling="linear",
             pos0=262144, fused=True, wide=True, mix=3),
        # chunks of four prompts: normed, turned and written into the cache's pages
        dict(name="norm_append", op="norm_append", S=4, q_min=3000, q_max=4096, kv_min=3500, kv_max=60000, Hq=64, Hkv=8,
             D=128, page=64, layout="NHD", scaling="none", mix=4),
        # a windowed layer: one token of one sequence of a toy model (latency)
        dict(name="window_token", op="window", S=1, q_min=1, q_max=1, kv_min=1000, kv_max=1000, Hq=2, Hkv=2, D=64, page=16,
             layout="NHD", window=128, sinks=4, mix=5),
        # one to four tokens of each of many responses, all far behind their window
        dict(name="window_batch", op="window", S=128, q_min=1, q_max=4, kv_min=900, kv_max=20000, Hq=64, Hkv=8, D=128,
             page=64, layout="NHD", window=4096, sinks=4, mix=6),
        # chunks of new tokens behind long cached prompts (prompt capture, scoring)
        dict(name="window_chunk", op="window", S=4, q_min=1500, q_max=2048, kv_min=9000, kv_max=65000, Hq=40, Hkv=8, D=128,
             page=128, layout="HND", window=4096, sinks=64, mix=7),
        # the replay of a short response of a toy model's windowed layer, forward and backward
        dict(name="replay_short", op="replay", P=1000, R=77, Hq=8, Hkv=2, D=64, window=256, sinks=4, mix=8),
        # the replay of a long response of a group on a 32K prompt, forward and backward
        dict(name="replay_long", op="replay", P=32768, R=8192, Hq=40, Hkv=8, D=128, window=4096, sinks=4, mix=9),
        # scores of a handful of response tokens of a toy model (latency)
        dict(name="scores_small", op="scores", T=33, V=1024, pad=0, top=5, temperature=1.0, mix=10),
        # scores of a packed group of a long-context model, padded vocabulary rows, with alternatives
        dict(name="scores_group", op="scores", T=4096, V=151936, pad=64, top=20, temperature=1.0, mix=11),
        # the gradient of log-probabilities and entropies of a response sampled at a temperature
        dict(name="scores_grad", op="scores_grad", T=1279, V=151936, pad=0, temperature=0.8, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_append", "window", "window", "window", "replay", "replay", "scores", "scores",
                     "scores_grad"])
    mix = rng.randrange(1 << 30)
    Hq, Hkv = rng.choice([(2, 2), (32, 8), (40, 8), (48, 8), (64, 8)])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    layout = rng.choice(["NHD", "HND"])
    if op in ("norm", "norm_grad"):
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 32, 20]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ramp"]),
                    pos0=_log(rng, 1, 1 << 21) - 1, fused=rng.random() < 0.5, wide=rng.random() < 0.5, mix=mix)
    if op == "norm_append":
        S = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, 16384 // S))
        kv = _log(rng, hi, 65536)
        return dict(op=op, S=S, q_min=max(0, hi // 2), q_max=hi, kv_min=hi, kv_max=kv, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    layout=layout, scaling=rng.choice(["none", "linear", "ramp"]), mix=mix)
    sinks = rng.choice([0, 1, 4, 64, _log(rng, 1, 300)])
    if op == "window":
        S = _log(rng, 1, 128)
        q_max = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(2048, 8192 // S)))
        # the gathered keys of the plain form stay moderate
        window = _log(rng, 1, min(16384, 480000 // S, max(1, (1 << 25) // (S * q_max))))
        kv_max = _log(rng, 1, min(131072, 2400000 // S))
        kv_min = max(1, kv_max // rng.choice([1, 2, 20]))
        return dict(op=op, S=S, q_min=max(0, q_max // rng.choice([1, 2, 1000])), q_max=q_max, kv_min=kv_min,
                    kv_max=kv_max, Hq=Hq, Hkv=Hkv, D=D, page=page, layout=layout, window=window, sinks=sinks, mix=mix)
    if op == "replay":
        R = _log(rng, 1, 8192)
        window = _log(rng, 1, min(16384, (1 << 25) * 40 // (R * max(Hq, 40))))
        return dict(op=op, P=_log(rng, 1, 65536), R=R, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=sinks, mix=mix)
    V = rng.choice([_log(rng, 500, 151936), _log(rng, 500, 151936) // 8 * 8, 32000, 151936])
    most = 4096 if op == "scores" else 2048
    c = dict(op=op, T=_log(rng, 1, min(16384, most * 151936 // V)), V=V, pad=rng.choice([0, 8, 64, 1]),
             temperature=rng.choice([1.0, 0.6, 1.3]), mix=mix)
    if op == "scores":
        c["top"] = rng.choice([0, 1, 5, 20, 32])
    return c


# --------------------------------------------------------------- sizes that the case alone sets
def _lens(case):
    """(new tokens, lengths with them) of every sequence."""
    rng = random.Random(case["mix"])
    n, kv = [], []
    for _ in range(case["S"]):
        n.append(rng.randint(case["q_min"], case["q_max"]))
        kv.append(max(n[-1], rng.randint(case["kv_min"], case["kv_max"])))
    if sum(n) == 0:
        n[0], kv[0] = 1, max(1, kv[0])
    return n, kv


def _freqs(rot, scaling):
    """(inverse frequencies, factor on the rotated vector) from their definitions, in 64 bits."""
    i = np.arange(rot // 2, dtype=np.float64)
    theta, factor, orig, fast, slow = 1.0e6, 8.0, 32768.0, 32.0, 1.0
    f = theta ** (-2.0 * i / rot)
    if scaling == "none":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    at = lambda turns: rot * math.log(orig / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


EPS = 1.0e-6


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed & 0x7FFFFFFF)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _projected(g, *shape):
    """Rows of a projection before their norm: heads of very different sizes."""
    size = torch.exp(1.5 * torch.randn(*shape[:-1], 1, generator=g, device=DEV))
    return (torch.randn(*shape, generator=g, device=DEV) * size).to(torch.bfloat16)


def _qkv(s, g, case, T, make):
    """q, k (and for the gradient the outputs' gradients) as rows of their own or of a fused projection."""
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case.get("fused"):
        both = make(g, T, Hq + 2 * Hkv, D)
        return both[:, :Hq], both[:, Hq:Hq + Hkv]
    return make(g, T, Hq, D), make(g, T, Hkv, D)


def prepare(case, seed):
    g = _gen(seed * 7919 + 29)
    s = {"case": case}
    op = case["op"]
    if op.startswith("norm"):
        f, s["factor"] = _freqs(case.get("rot", case["D"]), case["scaling"])
        s["freqs"] = torch.from_numpy(f)
        kind = torch.float32 if case.get("wide") else torch.bfloat16
        s["wq"], s["wk"] = ((1.0 + 0.3 * torch.randn(case["D"], generator=g, device=DEV)).to(kind) for _ in range(2))
    if op in ("norm", "norm_grad"):
        T = case["T"]
        s["q"], s["k"] = _qkv(s, g, case, T, _projected)
        s["positions"] = case["pos0"] + torch.randperm(T, generator=g, device=DEV)
        if op == "norm_grad":
            s["dq"], s["dk"] = _normal(g, T, case["Hq"], case["D"]), _normal(g, T, case["Hkv"], case["D"])
        return s
    if op in ("scores", "scores_grad"):
        T, V = case["T"], case["V"]
        x = torch.randn(T, V + case["pad"], generator=g, device=DEV) * 2.0
        s["ids"] = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
        # most sampled tokens are likely ones
        x[torch.arange(T, device=DEV), s["ids"].long()] += 20.0 * torch.rand(T, generator=g, device=DEV)
        s["logits"] = x.to(torch.bfloat16)[:, :V]
        del x
        if op == "scores_grad":
            logp, lse, ent = (torch.empty(T, device=DEV) for _ in range(3))
            for a in range(0, T, 256):
                y = s["logits"][a:a + 256].double() / case["temperature"]
                soft = torch.log_softmax(y, 1)
                logp[a:a + 256] = soft.gather(1, s["ids"][a:a + 256].long()[:, None])[:, 0].float()
                lse[a:a + 256] = torch.logsumexp(y, 1).float()
                ent[a:a + 256] = -(soft.exp() * soft).sum(1).float()
            s["logp"], s["lse"], s["entropy"] = logp, lse, ent
            w = (torch.rand(T, generator=g, device=DEV) >= 0.1).float()
            s["d_logp"] = w * torch.randn(T, generator=g, device=DEV) / T
            s["d_entropy"] = w * -0.01 / T
        return s
    if op == "replay":
        P, R, Hq, Hkv, D = (case[n] for n in ("P", "R", "Hq", "Hkv", "D"))
        s["kp"], s["vp"] = _normal(g, P, Hkv, D), _normal(g, P, Hkv, D)
        s["q"], s["ks"], s["vs"] = _normal(g, R, Hq, D), _normal(g, R, Hkv, D), _normal(g, R, Hkv, D)
        s["d_out"] = _normal(g, R, Hq, D)
        if own:
            import long_context_grpo_gb300 as ls
            acc = torch.empty(2, P, Hkv, D, device=DEV)
            s["prefix"] = ls.Prefix(s["kp"], s["vp"], acc[0], acc[1], Hq=Hq, window=case["window"], sinks=case["sinks"])
            s["work"] = torch.empty(max(16, s["prefix"].bwd_workspace_bytes(R)), dtype=torch.uint8, device=DEV)
        return s
    # the cache: shuffled pages of every sequence in one pool that holds keys and values side by side
    n, kv = _lens(case)
    ps, Hkv, D = case["page"], case["Hkv"], case["D"]
    need = [-(-x // ps) for x in kv]
    pages = sum(need) + 5
    order = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(kv), max(need) + 2), -1, dtype=np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    inner = (ps, Hkv, D) if case["layout"] == "NHD" else (Hkv, ps, D)
    both = torch.empty(pages, 2, *inner, dtype=torch.bfloat16, device=DEV)
    both.normal_(generator=g)
    s["k"], s["v"] = both[:, 0], both[:, 1]
    s["table"] = torch.from_numpy(table).to(DEV)
    s["ref"] = torch.from_numpy(np.bincount(table[table >= 0], minlength=pages).astype(np.int32)).to(DEV)
    s["len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["cu"] = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
    s["T"], s["max_new"], s["max_len"] = sum(n), max(n), max(kv)
    if op == "norm_append":
        s["q"], s["k_new"] = _projected(g, s["T"], case["Hq"], D), _projected(g, s["T"], Hkv, D)
        s["v_new"] = _normal(g, s["T"], Hkv, D)
    else:
        s["q"] = _normal(g, s["T"], case["Hq"], D)
    if own:
        import long_context_grpo_gb300 as ls
        s["cache"] = ls.PagedCache(s["k"], s["v"], s["table"], s["len"], s["ref"], Hq=case["Hq"], layout=case["layout"])
        if op == "window":
            need = s["cache"].attn_workspace_bytes(case["S"], s["T"], s["max_new"], s["max_len"], window=case["window"],
                                                   sinks=case["sinks"])
            s["work"] = torch.empty(max(16, need), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _turn(x, cos, sin, rot, interleaved):
    """x [T, H, D] with its first `rot` values rotated by the angles of cos, sin [T, rot / 2], in their type."""
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _angles(positions, freqs, factor, sign=1.0):
    a = positions.double()[:, None] * freqs.to(positions.device)[None]
    return (torch.cos(a) * factor).float(), (sign * torch.sin(a) * factor).float()


def _normed(x, weight):
    y = x.float()
    return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()


def _own_norm(s):
    import long_context_grpo_gb300 as ls
    c = s["case"]
    q, k = ls.norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["freqs"], eps=EPS, positions=s["positions"],
                        interleaved=c["interleaved"], attn_factor=s["factor"])
    return {"q": q, "k": k}


def _plain_norm(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], s["freqs"], s["factor"])
    return {n: _turn(_normed(s[n], s["w" + n]), cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16) for n in ("q", "k")}


def _own_norm_grad(s):
    import long_context_grpo_gb300 as ls
    c = s["case"]
    r = ls.norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["freqs"], eps=EPS,
                         positions=s["positions"], interleaved=c["interleaved"], attn_factor=s["factor"])
    return {"dq": r.dq, "dk": r.dk, "dwq": r.dq_weight, "dwk": r.dk_weight}


def _plain_norm_grad(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], s["freqs"], s["factor"], -1.0)
    out = {}
    for n in ("q", "k"):
        back = _turn(s["d" + n].float(), cos, sin, c["rot"], c["interleaved"])
        x = s[n].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * r
        out["dw" + n] = (back * x).sum((0, 1), dtype=torch.float64).float()
        back *= s["w" + n].float()
        out["d" + n] = (r * (back - x * (back * x).mean(-1, keepdim=True))).to(torch.bfloat16)
    return out


def _places(s):
    """(sequence, position) of every new token."""
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=s["T"])
    return seq, s["len"].long()[seq] - n[seq] + torch.arange(s["T"], device=DEV) - cu[seq]


def _own_norm_append(s):
    q, _ = s["cache"].append(s["k_new"], s["v_new"], s["cu"], q=s["q"], inv_freq=s["freqs"], attn_factor=s["factor"],
                             q_weight=s["wq"], k_weight=s["wk"], norm_eps=EPS)
    return {"q": q, "k_pages": s["k"], "v_pages": s["v"]}


def _plain_norm_append(s):
    c = s["case"]
    seq, pos = _places(s)
    cos, sin = _angles(pos, s["freqs"], s["factor"])
    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    k = _turn(_normed(s["k_new"], s["wk"]), cos, sin, c["D"], False).to(torch.bfloat16)
    if c["layout"] == "NHD":
        s["k"][page, slot] = k
        s["v"][page, slot] = s["v_new"]
    else:
        s["k"][page, :, slot] = k
        s["v"][page, :, slot] = s["v_new"]
    q = _turn(_normed(s["q"], s["wq"]), cos, sin, c["D"], False).to(torch.bfloat16)
    return {"q": q, "k_pages": s["k"], "v_pages": s["v"]}


def _own_window(s):
    c = s["case"]
    o, lse = s["cache"].attn(s["q"], s["cu"], max_new=s["max_new"], max_len=s["max_len"], window=c["window"],
                             sinks=c["sinks"], workspace=s["work"])
    return {"o": o, "lse": lse}


def _seen(at, pos, window, sinks):
    """Whether a token at `pos` sees the key at `at`."""
    return (at <= pos) & ((at > pos - window) | (at < sinks))


def _plain_window(s):
    """The first keys and the window's union of every sequence gathered, sequences together while their
    scores stay moderate."""
    c = s["case"]
    n, kv = _lens(c)
    Hq, Hkv, D, ps, W = c["Hq"], c["Hkv"], c["D"], c["page"], c["window"]
    o = torch.empty(s["T"], Hq, D, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(s["T"], Hq, device=DEV)
    sinks = min(c["sinks"], s["max_len"])
    L = min(s["max_len"], sinks + W + s["max_new"] - 1)
    seq, pos = _places(s)
    off = torch.arange(s["T"], device=DEV) - s["cu"].long()[seq]
    step = max(1, (1 << 30) // (Hq * s["max_new"] * L))
    first = (s["len"].long() - (s["cu"][1:] - s["cu"][:-1]).long() - W + 1).clamp(min=sinks)
    for a in range(0, c["S"], step):
        S = min(step, c["S"] - a)
        at = torch.arange(L, device=DEV).repeat(S, 1)
        at[:, sinks:] += (first[a:a + S] - sinks)[:, None]
        alive = at < s["len"][a:a + S, None]
        page = s["table"][a:a + S].long().gather(1, (at // ps).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)
        if c["layout"] == "NHD":
            k, v = (x[page, at % ps].permute(0, 2, 1, 3).float() for x in (s["k"], s["v"]))
        else:
            k, v = (x[page, :, at % ps].permute(0, 2, 1, 3).float() for x in (s["k"], s["v"]))
        mine = slice(sum(n[:a]), sum(n[:a + S]))
        who = seq[mine] - a
        q = torch.zeros(S, s["max_new"], Hkv, Hq // Hkv, D, device=DEV)
        where = torch.full((S, s["max_new"]), -1, device=DEV)
        q[who, off[mine]] = s["q"][mine].float().reshape(-1, Hkv, Hq // Hkv, D)
        where[who, off[mine]] = pos[mine]
        hidden = ~(_seen(at[:, None], where[:, :, None], W, sinks) & alive[:, None])
        x = q.permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D) @ k.transpose(-1, -2)
        x = x.reshape(S, Hkv, -1, s["max_new"], L).mul_(D ** -0.5)
        x.masked_fill_(hidden[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        x = x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        y = (x.reshape(S, Hkv, -1, L) @ v).reshape(S, Hkv, -1, s["max_new"], D) / total.clamp(min=1e-30)
        y = y.permute(0, 3, 1, 2, 4).reshape(S, s["max_new"], Hq, D)
        e = (torch.log(total) + top).squeeze(-1).permute(0, 3, 1, 2).reshape(S, s["max_new"], Hq)
        o[mine], lse[mine] = y[who, off[mine]].to(torch.bfloat16), e[who, off[mine]]
    return {"o": o, "lse": lse}


def _touched(case):
    """The runs of prompt rows that a response sees: (first, rows) of the window's and the first tokens'."""
    P = case["P"]
    lo = max(0, P - case["window"] + 1)
    sinks = min(case["sinks"], P)
    if lo <= sinks:
        return [(0, P)]
    return ([(lo, P - lo)] if lo < P else []) + ([(0, sinks)] if sinks else [])


def _own_replay(s):
    p = s["prefix"]
    o, lse = p.fwd(s["q"], s["ks"], s["vs"])
    dq, dk, dv = p.bwd(s["q"], s["ks"], s["vs"], o, lse, s["d_out"], workspace=s["work"])
    out = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    for i, (row, n) in enumerate(_touched(s["case"])):
        a, b = (torch.empty(n, p.Hkv, p.D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        out["dk_prompt%d" % i], out["dv_prompt%d" % i] = p.finalize_rows(row, n, dk_out=a, dv_out=b, reset=True)
    return out


def _replay(s, kind, block):
    """Forward and backward in `kind`, blocks of queries over the keys that they may see."""
    c = s["case"]
    P, R, Hq, Hkv, D, W = (c[n] for n in ("P", "R", "Hq", "Hkv", "D", "window"))
    sinks, g, scale = min(c["sinks"], P + R), Hq // Hkv, D ** -0.5
    k = torch.cat((s["kp"], s["ks"])).to(kind).transpose(0, 1).contiguous()
    v = torch.cat((s["vp"], s["vs"])).to(kind).transpose(0, 1).contiguous()
    o, dq = (torch.empty(R, Hq, D, dtype=kind, device=DEV) for _ in range(2))
    lse = torch.empty(R, Hq, dtype=kind, device=DEV)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    for t0 in range(0, R, block):
        t1 = min(R, t0 + block)
        lo = max(P + t0 - W + 1, 0)
        at = torch.cat((torch.arange(min(sinks, lo), device=DEV), torch.arange(lo, P + t1, device=DEV)))
        hidden = ~_seen(at[None], P + torch.arange(t0, t1, device=DEV)[:, None], W, sinks)
        for h in range(Hkv):
            kh, vh = k[h, at], v[h, at]
            q, d = (x[t0:t1, h * g:(h + 1) * g].to(kind).transpose(0, 1) for x in (s["q"], s["d_out"]))
            x = (q @ kh.T).mul_(scale).masked_fill_(hidden, -math.inf)
            top = x.amax(-1, keepdim=True)
            p = x.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            p = p.div_(total)
            y = p @ vh
            o[t0:t1, h * g:(h + 1) * g] = y.transpose(0, 1)
            lse[t0:t1, h * g:(h + 1) * g] = (torch.log(total) + top)[..., 0].T
            dv[h].index_add_(0, at, p.flatten(0, 1).T @ d.flatten(0, 1))
            ds = (d @ vh.T).sub_((d * y).sum(-1, keepdim=True)).mul_(p)
            dq[t0:t1, h * g:(h + 1) * g] = (ds @ kh).mul_(scale).transpose(0, 1)
            dk[h].index_add_(0, at, (ds.flatten(0, 1).T @ q.flatten(0, 1)).mul_(scale))
    out = {"o": o, "lse": lse, "dq": dq, "dk": dk[:, P:].transpose(0, 1), "dv": dv[:, P:].transpose(0, 1)}
    for i, (row, n) in enumerate(_touched(c)):
        out["dk_prompt%d" % i] = dk[:, row:row + n].transpose(0, 1)
        out["dv_prompt%d" % i] = dv[:, row:row + n].transpose(0, 1)
    return out


def _plain_replay(s):
    out = _replay(s, torch.float32, 1024)
    return {n: x if n == "lse" else x.to(torch.bfloat16) for n, x in out.items()}


def _own_scores(s):
    import long_context_grpo_gb300 as ls
    c = s["case"]
    r = ls.token_scores(s["logits"], s["ids"], top=c["top"], temperature=c["temperature"])
    return {"logp": r.logp, "lse": r.lse, "entropy": r.entropy, "top_ids": r.top_ids, "top_logp": r.top_logp}


def _plain_scores(s):
    c = s["case"]
    T, V, top = c["T"], c["V"], c["top"]
    logp, lse, ent = (torch.empty(T, device=DEV) for _ in range(3))
    ids = torch.empty(T, top, dtype=torch.int32, device=DEV)
    best = torch.empty(T, top, device=DEV)
    rows = max(1, (1 << 27) // V)
    for a in range(0, T, rows):
        i = slice(a, min(T, a + rows))
        x = s["logits"][i].float() / c["temperature"]
        high = x.amax(1, keepdim=True)
        e = torch.exp(x - high)
        total = e.sum(1, dtype=torch.float64)
        z = torch.log(total)
        logp[i] = ((x.gather(1, s["ids"][i].long()[:, None]) - high)[:, 0].double() - z).float()
        lse[i] = (high[:, 0].double() + z).float()
        ent[i] = (z - (e * (x - high)).sum(1, dtype=torch.float64) / total).float()
        if top:
            # the logits' order with ties to the lowest index as whole numbers
            y = s["logits"][i].float() + 0.0
            key = y.view(torch.int32)
            key = torch.where(key < 0, key ^ 0x7FFFFFFF, key).long() * (1 << 31) + (V - 1 - torch.arange(V, device=DEV))
            at = V - 1 - (key.topk(top, 1).values & ((1 << 31) - 1))
            ids[i] = at.int()
            best[i] = ((x.gather(1, at) - high).double() - z[:, None]).float()
    return {"logp": logp, "lse": lse, "entropy": ent, "top_ids": ids, "top_logp": best}


def _own_scores_grad(s):
    import long_context_grpo_gb300 as ls
    return {"dlogits": ls.token_scores_bwd(s["logits"], s["ids"], s["logp"], s["lse"], s["entropy"], s["d_logp"],
                                           s["d_entropy"], temperature=s["case"]["temperature"])}


def _plain_scores_grad(s):
    c = s["case"]
    out = torch.empty(c["T"], c["V"], dtype=torch.bfloat16, device=DEV)
    rows = max(1, (1 << 28) // c["V"])
    for a in range(0, c["T"], rows):
        i = slice(a, min(c["T"], a + rows))
        x = s["logits"][i].float() / c["temperature"] - s["lse"][i, None]
        p = torch.exp(x)
        d = -p * (s["d_logp"][i, None] + s["d_entropy"][i, None] * (x + s["entropy"][i, None]))
        # the given token's own: 1 - p from its log-probability
        y = s["ids"][i].long()[:, None]
        lp = s["logp"][i, None]
        mine = -torch.expm1(lp) * s["d_logp"][i, None] - torch.exp(lp) * s["d_entropy"][i, None] * (lp + s["entropy"][i, None])
        d.scatter_(1, y, mine)
        out[i] = (d / c["temperature"]).to(torch.bfloat16)
    return {"dlogits": out}


_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "norm_append": _own_norm_append, "window": _own_window,
        "replay": _own_replay, "scores": _own_scores, "scores_grad": _own_scores_grad}
_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "norm_append": _plain_norm_append, "window": _plain_window,
          "replay": _plain_replay, "scores": _plain_scores, "scores_grad": _plain_scores_grad}


# ------------------------------------------------------------------- what a pass cannot do without
def _pairs(n, first, window, sinks):
    """(query, key) pairs of n tokens at positions first, first + 1, .. and the keys that any of them sees."""
    pos = np.arange(first, first + n, dtype=np.int64)
    lo = np.maximum(pos - window + 1, 0)
    pairs = int((pos + 1 - lo + np.minimum(sinks, lo)).sum())
    return pairs, int(first + n - lo[0] + min(sinks, lo[0])) if n else 0


def work(case):
    op = case["op"]
    D = case.get("D", 0)
    if op in ("norm", "norm_grad"):
        n = case["T"] * (case["Hq"] + case["Hkv"])
        w = 2 * D * (4 if case["wide"] else 2)
        if op == "norm":
            return {"bytes": 4 * n * D + 8 * case["T"] + w, "flops": 4 * n * D + 3 * n * case["rot"]}
        return {"bytes": 6 * n * D + 8 * case["T"] + w + 8 * D, "flops": 10 * n * D + 3 * n * case["rot"]}
    if op == "norm_append":
        T = sum(_lens(case)[0])
        H = case["Hq"] + 2 * case["Hkv"]
        return {"bytes": 4 * T * H * D + 12 * case["S"] + 4 * D, "flops": 7 * T * (case["Hq"] + case["Hkv"]) * D}
    if op == "window":
        n, kv = _lens(case)
        pairs = keys = 0
        for a, b in zip(n, kv):
            x, y = _pairs(a, b - a, case["window"], case["sinks"])
            pairs, keys = pairs + x, keys + y
        return {"bytes": 4 * keys * case["Hkv"] * D + sum(n) * case["Hq"] * (4 * D + 4), "flops": 4 * D * case["Hq"] * pairs}
    if op == "replay":
        P, R, Hq, Hkv = case["P"], case["R"], case["Hq"], case["Hkv"]
        pairs, _ = _pairs(R, P, case["window"], case["sinks"])
        prompt = sum(n for _, n in _touched(case))
        # forward: q, keys, values in, o and lse out; backward: those again with d_out, five products
        rows, heads = R * Hq * D, Hkv * D
        return {"bytes": 2 * (6 * rows + 8 * (prompt + R) * heads - 2 * prompt * heads) + 8 * R * Hq + 4 * prompt * heads,
                "flops": 14 * D * Hq * pairs}
    T, V = case["T"], case["V"]
    if op == "scores":
        return {"bytes": T * (2 * V + 16 + 8 * case["top"]), "flops": 6 * T * V}
    return {"bytes": T * (4 * V + 24), "flops": 7 * T * V}


# ----------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("window", "replay") and work(case)["flops"] > 4.0e12:
        return None
    s = prepare(case, seed)
    return _exact[op](s)


def _by(positions, freqs, factor, sign):
    """factor exp(+-i angle) of every token and pair."""
    angle = positions.double()[:, None] * freqs.to(positions.device)
    return torch.polar(torch.full_like(angle, factor), sign * angle)[:, None]


def _exact_turn(x, by, rot, interleaved):
    y = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * by
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * by
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_rms(x, w):
    x = x.double()
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


def _exact_norm(s):
    c = s["case"]
    by = _by(s["positions"], s["freqs"], s["factor"], 1.0)
    return {n: _exact_turn(_exact_rms(s[n], s["w" + n]), by, c["rot"], c["interleaved"]) for n in ("q", "k")}


def _exact_norm_grad(s):
    """Automatic differentiation of the definition."""
    c = s["case"]
    by = _by(s["positions"], s["freqs"], s["factor"], 1.0)
    out = {}
    for n in ("q", "k"):
        x, w = s[n].double().requires_grad_(), s["w" + n].double().requires_grad_()
        y = _exact_rms(x, w)
        # the rotation is linear: its transpose is the rotation by minus the angle
        back = _exact_turn(s["d" + n].double(), by.conj(), c["rot"], c["interleaved"])
        out["d" + n], out["dw" + n] = torch.autograd.grad(y, (x, w), back)
    return out


def _exact_norm_append(s):
    c = s["case"]
    seq, pos = _places(s)
    by = _by(pos, s["freqs"], s["factor"], 1.0)
    k_new = _exact_turn(_exact_rms(s["k_new"], s["wk"]), by, c["D"], False)
    out = {"q": _exact_turn(_exact_rms(s["q"], s["wq"]), by, c["D"], False), "k_pages": s["k"].double(),
           "v_pages": s["v"].double()}
    for b, (m, end) in enumerate(zip(*_lens(c))):
        at, places = int(s["cu"][b]), torch.arange(end - m, end, device=DEV)
        pages = s["table"][b].long()[places // c["page"]]
        for n, x in (("k_pages", k_new), ("v_pages", s["v_new"].double())):
            pool = out[n] if c["layout"] == "NHD" else out[n].transpose(1, 2)
            pool[pages, places % c["page"]] = x[at:at + m]
    return out


def _exact_window(s):
    """Sequence by sequence, key head by key head, blocks of tokens over all keys up to theirs."""
    c = s["case"]
    n, kv = _lens(c)
    W, sinks, g = c["window"], c["sinks"], c["Hq"] // c["Hkv"]
    o = torch.zeros(s["T"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b in range(c["S"]):
        pages = s["table"][b, :-(-kv[b] // c["page"])].long()
        k, v = (x[pages] if c["layout"] == "NHD" else x[pages].transpose(1, 2) for x in (s["k"], s["v"]))
        k, v = (x.reshape(-1, c["Hkv"], c["D"])[:kv[b]] for x in (k, v))
        for t in range(0, n[b], 512):
            m = min(512, n[b] - t)
            pos = kv[b] - n[b] + t + torch.arange(m, device=DEV)
            places = torch.arange(kv[b], device=DEV)
            near = torch.nonzero((places < sinks) | ((places > int(pos[0]) - W) & (places <= int(pos[-1]))))[:, 0]
            back = pos[:, None] - near[None]
            hidden = (back < 0) | ((back >= W) & (near >= sinks)[None])
            kn, vn = k[near].double(), v[near].double()
            for h in range(c["Hkv"]):
                i = slice(at + t, at + t + m), slice(h * g, (h + 1) * g)
                x = (s["q"][i].double().transpose(0, 1) @ kn[:, h].T / math.sqrt(c["D"])).masked_fill(hidden, -math.inf)
                lse[i] = torch.logsumexp(x, -1).T
                o[i] = (torch.softmax(x, -1) @ vn[:, h]).transpose(0, 1)
        at += n[b]
    return {"o": o, "lse": lse}


def _exact_replay(s):
    """Automatic differentiation of the softmax over the visible keys, blocks of 512 queries."""
    c = s["case"]
    P, R, W, g, D = c["P"], c["R"], c["window"], c["Hq"] // c["Hkv"], c["D"]
    o, dq = (torch.empty(R, c["Hq"], D, dtype=torch.float64, device=DEV) for _ in range(2))
    lse = torch.empty(R, c["Hq"], dtype=torch.float64, device=DEV)
    keys, values = (torch.cat((s[a], s[b])) for a, b in (("kp", "ks"), ("vp", "vs")))
    dk, dv = (torch.zeros(keys.shape, dtype=torch.float64, device=DEV) for _ in range(2))
    places = torch.arange(P + R, device=DEV)
    for t in range(0, R, 512):
        pos = P + torch.arange(t, min(R, t + 512), device=DEV)
        near = torch.nonzero((places < c["sinks"]) & (places <= pos[-1]) | (places > pos[0] - W) & (places <= pos[-1]))[:, 0]
        back = pos[:, None] - near[None]
        hidden = (back < 0) | ((back >= W) & (near >= c["sinks"])[None])
        for h in range(c["Hkv"]):
            i = slice(t, t + len(pos)), slice(h * g, (h + 1) * g)
            q = s["q"][i].double().transpose(0, 1).requires_grad_()
            k, v = (x[near, h].double().requires_grad_() for x in (keys, values))
            x = (q @ k.T / math.sqrt(D)).masked_fill(hidden, -math.inf)
            y = torch.softmax(x, -1) @ v
            grads = torch.autograd.grad(y, (q, k, v), s["d_out"][i].double().transpose(0, 1))
            lse[i] = torch.logsumexp(x.detach(), -1).T
            o[i], dq[i] = y.detach().transpose(0, 1), grads[0].transpose(0, 1)
            dk[near, h] += grads[1]
            dv[near, h] += grads[2]
    out = {"o": o, "lse": lse, "dq": dq, "dk": dk[P:], "dv": dv[P:]}
    for j, (row, n) in enumerate(_touched(c)):
        out["dk_prompt%d" % j], out["dv_prompt%d" % j] = dk[row:row + n], dv[row:row + n]
    return out


def _exact_scores(s):
    c = s["case"]
    out = {n: [] for n in ("logp", "lse", "entropy", "top_logp")}
    for a in range(0, c["T"], 256):
        x = s["logits"][a:a + 256].double() / c["temperature"]
        soft = torch.log_softmax(x, 1)
        out["logp"].append(soft.gather(1, s["ids"][a:a + 256].long()[:, None])[:, 0])
        out["lse"].append(torch.logsumexp(x, 1))
        out["entropy"].append(torch.special.entr(soft.exp()).sum(1))
        out["top_logp"].append(soft.topk(c["top"], 1).values)
    out = {n: torch.cat(x) for n, x in out.items()}
    out["top_ids"] = None
    return {n: out[n] for n in ("logp", "lse", "entropy", "top_ids", "top_logp")}


def _exact_scores_grad(s):
    """From the logits alone: the saved log-probabilities and entropies are roundings of what this computes."""
    c = s["case"]
    out = torch.empty(c["T"], c["V"], dtype=torch.float64, device=DEV)
    for a in range(0, c["T"], 128):
        i = slice(a, min(c["T"], a + 128))
        soft = torch.log_softmax(s["logits"][i].double() / c["temperature"], 1)
        p = soft.exp()
        mean = (p * soft).sum(1, keepdim=True)
        one = torch.zeros_like(p).scatter_(1, s["ids"][i].long()[:, None], 1.0)
        out[i] = ((one - p) * s["d_logp"][i, None].double() - p * (soft - mean) * s["d_entropy"][i, None].double()) / c["temperature"]
    return {"dlogits": out}


_exact = {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "norm_append": _exact_norm_append, "window": _exact_window,
          "replay": _exact_replay, "scores": _exact_scores, "scores_grad": _exact_scores_grad}
