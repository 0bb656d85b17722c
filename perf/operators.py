"""Measured cases of the operators around branch replay: the policy loss with a KL term, rotary
positions, the paged cache of a group's keys and values, and attention over it.

Every case is a dict of plain values.  `run` computes one pass, either with the library's
entry points (`own`) or in elementary torch operations in 32 bits (64 for angles of far
positions, log-sum-exps next to a clip border and long sums).  `exact` is the definition in
64 bits.
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
        # the policy loss: a handful of response tokens of a toy model (latency)
        dict(name="loss_small", op="loss", T=33, V=1024, pad=0, kl="k3", beta=0.04, masked=0.1, mix=1),
        # one ordinary response of a group on a 32K prompt, all tokens trained on, no KL term
        dict(name="loss_response", op="loss", T=1279, V=32000, pad=0, kl="none", beta=0.0, masked=0.0, mix=2),
        # a packed group of a long-context model, padded vocabulary rows, a tenth of the tokens masked
        dict(name="loss_group", op="loss", T=4096, V=151936, pad=64, kl="k3", beta=0.01, masked=0.1, mix=3),
        # rotary positions of one new token per response of a group (latency)
        dict(name="rope_token", op="rope", T=8, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, scaling="none",
             inverse=False, pos0=32768, fused=False, mix=4),
        # the gradient through a partial interleaved rotation of an odd-sized response
        dict(name="rope_grad", op="rope", T=3001, Hq=40, Hkv=8, D=128, rot=64, interleaved=True, scaling="linear",
             inverse=True, pos0=262144, fused=True, mix=5),
        # a chunk of a far prompt: rotated and written into the cache's pages
        dict(name="append_chunk", op="append", S=4, q_min=3000, q_max=4096, kv_min=3500, kv_max=60000, Hq=64, Hkv=8,
             D=128, page=64, layout="NHD", scaling="ramp", mix=6),
        # attention: one token of one short sequence (latency)
        dict(name="attn_token", op="attn", S=1, q_min=1, q_max=1, kv_min=257, kv_max=257, Hq=2, Hkv=2, D=64, page=16,
             layout="NHD", group=1, shared=0, mix=7),
        # one token of each response of a group forked from a 32K prompt: the prompt's pages are shared
        dict(name="attn_group", op="attn", S=8, q_min=1, q_max=1, kv_min=33300, kv_max=34700, Hq=32, Hkv=8, D=128,
             page=64, layout="NHD", group=8, shared=32768, mix=8),
        # one to four tokens of many unrelated sequences of very different lengths
        dict(name="attn_batch", op="attn", S=40, q_min=1, q_max=4, kv_min=900, kv_max=65000, Hq=64, Hkv=8, D=128,
             page=32, layout="HND", group=1, shared=0, mix=9),
        # a chunk of new tokens behind 128K cached ones (prompt capture, scoring)
        dict(name="attn_chunk", op="attn", S=1, q_min=1024, q_max=1024, kv_min=131072, kv_max=131072, Hq=40, Hkv=8,
             D=128, page=128, layout="NHD", group=1, shared=0, mix=10),
        # the next group: its rows retired and forked again from the prompts' rows
        dict(name="pages_fork", op="fork", P=8, G=16, kv_min=20000, kv_max=33000, Hkv=8, D=128, page=64,
             layout="NHD", mix=11),
        # a fragmented pool's live pages gathered into another one
        dict(name="pages_compact", op="compact", S=24, kv_min=500, kv_max=40000, Hkv=8, D=128, page=64, layout="HND",
             spare=0.6, mix=12),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["loss", "loss", "rope", "append", "attn", "attn", "attn", "fork", "compact"])
    mix = rng.randrange(1 << 30)
    Hq, Hkv = rng.choice([(2, 2), (32, 8), (40, 8), (48, 8), (64, 8)])
    D = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    layout = rng.choice(["NHD", "HND"])
    if op == "loss":
        V = rng.choice([_log(rng, 500, 151936), _log(rng, 500, 151936) // 8 * 8, 32000, 151936])
        kl = rng.choice(["none", "k1", "k2", "k3"])
        return dict(op=op, T=_log(rng, 1, min(16384, 4096 * 151936 // V)), V=V, pad=rng.choice([0, 8, 64, 1]), kl=kl,
                    beta=0.0 if kl == "none" else rng.choice([0.001, 0.04, 0.2]), masked=rng.choice([0.0, 0.1, 0.5]), mix=mix)
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 32, 20]),
                    interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ramp"]),
                    inverse=rng.random() < 0.5, pos0=_log(rng, 1, 1 << 21) - 1, fused=rng.random() < 0.5, mix=mix)
    if op == "append":
        S = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, 16384 // S))
        kv = _log(rng, hi, 65536)
        return dict(op=op, S=S, q_min=max(0, hi // 2), q_max=hi, kv_min=hi, kv_max=kv, Hq=Hq, Hkv=Hkv, D=D, page=page,
                    layout=layout, scaling=rng.choice(["none", "linear", "ramp"]), mix=mix)
    if op == "attn":
        group = rng.choice([1, 1, 2, 8])
        S = group * _log(rng, 1, max(1, 48 // group))
        q_max = 1 if rng.random() < 0.4 else _log(rng, 1, 2048)
        # the plain form's scores, S x Hq x q_max x kv_max in 32 bits, and its gathered keys stay moderate
        kv_most = min(131072, (1 << 27) // max(1, S * q_max * Hq // 40), 1300000 // S)
        kv_max = _log(rng, 1, max(2, kv_most))
        kv_min = max(1, kv_max // rng.choice([1, 2, 20]))
        shared = 0 if group == 1 else max(0, kv_min - q_max) // rng.choice([1, 2]) // page * page
        return dict(op=op, S=S, q_min=max(0, q_max // rng.choice([1, 2, 1000])), q_max=q_max, kv_min=kv_min,
                    kv_max=kv_max, Hq=Hq, Hkv=Hkv, D=D, page=page, layout=layout, group=group, shared=shared, mix=mix)
    if op == "fork":
        P = _log(rng, 1, 12)
        G = _log(rng, 1, 64)
        kv = _log(rng, 2, 33000)
        return dict(op=op, P=P, G=G, kv_min=max(1, kv // 2), kv_max=kv, Hkv=Hkv, D=D, page=page, layout=layout, mix=mix)
    kv = _log(rng, 16, 40000)
    return dict(op=op, S=_log(rng, 1, 24), kv_min=max(1, kv // 8), kv_max=kv, Hkv=Hkv, D=D, page=page, layout=layout,
                spare=rng.choice([0.1, 0.6, 1.0]), mix=mix)


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
    # frequencies that turn more than `fast` times over the original length stay, those that turn
    # less than `slow` times are divided by the factor, in between both are mixed by the index
    at = lambda turns: rot * math.log(orig / (turns * 2.0 * math.pi)) / (2.0 * math.log(theta))  # noqa: E731
    lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed & 0x7FFFFFFF)


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16) * std


def _pool(g, pages, case):
    """Keys' and values' pages in one allocation, as views [pages, ...] of the case's layout."""
    inner = (case["page"], case["Hkv"], case["D"]) if case["layout"] == "NHD" else (case["Hkv"], case["page"], case["D"])
    both = torch.empty(pages, 2, *inner, dtype=torch.bfloat16, device=DEV)
    both.normal_(generator=g)
    return both[:, 0], both[:, 1]


def _tables(case, seed, lens, extra, shared=0, group=1):
    """Shuffled page tables of rows with these lengths: (table, refcount), on the host."""
    rng = np.random.default_rng(seed)
    ps = case["page"]
    need = [-(-n // ps) for n in lens]
    keep = shared // ps
    total = sum(need) - sum((group - 1) * keep for _ in range(len(lens) // group) if group > 1)
    pages = total + extra
    order = rng.permutation(pages)
    width = max(need) + 2
    table = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        first = 0
        if group > 1 and b % group:
            table[b, :keep] = table[b - b % group, :keep]
            first = keep
        table[b, first:n] = order[at:at + n - first]
        at += n - first
    ref = np.bincount(table[table >= 0], minlength=pages).astype(np.int32)
    return table, ref


def prepare(case, seed):
    g = _gen(seed * 7919 + 17)
    s = {"case": case}
    op = case["op"]
    if op == "loss":
        T, V = case["T"], case["V"]
        s["logits"] = (torch.randn(T, V + case["pad"], generator=g, device=DEV) * 2.0).to(torch.bfloat16)[:, :V]
        s["ids"] = torch.randint(0, V, (T,), generator=g, device=DEV, dtype=torch.int32)
        logp = torch.empty(T, device=DEV)
        for a in range(0, T, 512):
            x = s["logits"][a:a + 512].float()
            logp[a:a + 512] = x.gather(1, s["ids"][a:a + 512].long()[:, None])[:, 0] - torch.logsumexp(x, 1)
        s["old"] = logp + 0.2 * torch.randn(T, generator=g, device=DEV)
        s["ref"] = logp + 0.3 * torch.randn(T, generator=g, device=DEV)
        s["adv"] = torch.randn(T, generator=g, device=DEV)
        w = (torch.rand(T, generator=g, device=DEV) >= case["masked"]).float()
        s["weight"] = w / w.sum().clamp(min=1.0)
        s["eps"] = (0.2, 0.28)
        return s
    if op == "rope":
        T, D = case["T"], case["D"]
        if case["fused"]:  # rows of a projection that holds queries, keys and values side by side
            qkv = _normal(g, T, case["Hq"] + 2 * case["Hkv"], D)
            s["q"], s["k"] = qkv[:, :case["Hq"]], qkv[:, case["Hq"]:case["Hq"] + case["Hkv"]]
        else:
            s["q"], s["k"] = _normal(g, T, case["Hq"], D), _normal(g, T, case["Hkv"], D)
        s["positions"] = case["pos0"] + torch.randperm(T, generator=g, device=DEV)
        f, s["factor"] = _freqs(case["rot"], case["scaling"])
        s["freqs"] = torch.from_numpy(f)
        return s
    if op in ("append", "attn"):
        n, kv = _lens(case)
        table, ref = _tables(case, seed, kv, 5, case.get("shared", 0), case.get("group", 1))
        T = sum(n)
        s["k"], s["v"] = _pool(g, len(ref), case)
        s["table"], s["ref"] = torch.from_numpy(table).to(DEV), torch.from_numpy(ref).to(DEV)
        s["len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        s["cu"] = torch.tensor([0] + list(np.cumsum(n)), dtype=torch.int32, device=DEV)
        s["T"], s["max_new"], s["max_len"] = T, max(n), max(kv)
        s["q"] = _normal(g, T, case["Hq"], case["D"])
        if op == "append":
            s["k_new"], s["v_new"] = _normal(g, T, case["Hkv"], case["D"]), _normal(g, T, case["Hkv"], case["D"])
            f, s["factor"] = _freqs(case["D"], case["scaling"])
            s["freqs"] = torch.from_numpy(f)
        elif case["group"] > 1:
            s["shared"] = torch.full((case["S"] // case["group"],), case["shared"], dtype=torch.int32, device=DEV)
        else:
            s["shared"] = None
    elif op == "fork":
        rng = random.Random(case["mix"])
        P, G, ps = case["P"], case["G"], case["page"]
        kv = [rng.randint(case["kv_min"], case["kv_max"]) for _ in range(P)]
        mine, ref = _tables(case, seed, kv, P * G + 7)
        table = np.full((P + P * G, mine.shape[1]), -1, dtype=np.int32)
        table[:P] = mine
        s["k"], s["v"] = _pool(g, len(ref), case)
        free = list(np.nonzero(ref == 0)[0][::-1])
        length = kv + [0] * (P * G)
        for c in range(P * G):  # the last group's rows, forked from the same prompts
            p, row = c // G, P + c
            table[row] = table[p]
            length[row] = kv[p]
            full, part = divmod(kv[p], ps)
            ref[table[p, :full]] += 1
            if part:
                table[row, full] = free.pop(0)
                ref[table[row, full]] = 1
        s["table"], s["ref"] = torch.from_numpy(table).to(DEV), torch.from_numpy(ref).to(DEV)
        s["len"] = torch.tensor(length, dtype=torch.int32, device=DEV)
        s["parents"] = torch.arange(P, device=DEV, dtype=torch.int32).repeat_interleave(G)
        s["children"] = P + torch.arange(P * G, device=DEV, dtype=torch.int32)
    else:
        rng = random.Random(case["mix"])
        kv = [rng.randint(case["kv_min"], case["kv_max"]) for _ in range(case["S"])]
        live = sum(-(-x // case["page"]) for x in kv)
        table, ref = _tables(case, seed, kv, 1 + int(case["spare"] * live))
        s["k"], s["v"] = _pool(g, len(ref), case)
        s["table"], s["ref"] = torch.from_numpy(table).to(DEV), torch.from_numpy(ref).to(DEV)
        s["len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        # the pool that the live pages move into: pages past them stay as they are
        both = torch.zeros(live + 3, 2, *s["k"].shape[1:], dtype=torch.bfloat16, device=DEV)
        s["k2"], s["v2"] = both[:, 0], both[:, 1]
        s["table2"], s["ref2"] = torch.empty_like(s["table"]), torch.empty(live + 3, dtype=torch.int32, device=DEV)
        s["len2"] = torch.empty_like(s["len"])
    if own:
        import long_context_grpo_gb300 as ls
        Hq = case.get("Hq", case["Hkv"])
        s["cache"] = ls.PagedCache(s["k"], s["v"], s["table"], s["len"], s["ref"], Hq=Hq, layout=case["layout"])
        if op == "compact":
            s["cache2"] = ls.PagedCache(s["k2"], s["v2"], s["table2"], s["len2"], s["ref2"], Hq=Hq, layout=case["layout"])
        if op == "attn":
            s["work"] = torch.empty(s["cache"].attn_workspace_bytes(case["S"], s["T"], s["max_new"], s["max_len"]),
                                    dtype=torch.uint8, device=DEV)
        else:
            s["work"] = torch.empty(s["cache"].pages_workspace_bytes(), dtype=torch.uint8, device=DEV)
    return s


# --------------------------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    return (_own if own else _plain)[op](s)


def _own_loss(s):
    import long_context_grpo_gb300 as ls
    c = s["case"]
    r = ls.policy_loss(s["logits"], s["ids"], s["old"], s["adv"], s["weight"], eps_low=s["eps"][0], eps_high=s["eps"][1],
                       logp_ref=None if c["kl"] == "none" else s["ref"], beta=c["beta"], kl=c["kl"])
    return {"loss": r.loss, "dlogits": r.dlogits, "logp": r.logp, "kl": r.kl, "clip": r.clip_mask}


def _plain_loss(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(1, dtype=torch.float64)
    lse = top[:, 0].double() + torch.log(total)
    y = s["ids"].long()[:, None]
    logp = x.gather(1, y)[:, 0].double() - lse
    d = logp - s["old"].double()
    rho, A = torch.exp(d), s["adv"].double()
    lo, hi = 1.0 - s["eps"][0], 1.0 + s["eps"][1]
    clipped = ((A > 0) & (rho > hi)) | ((A < 0) & (rho < lo))
    surr = torch.where(clipped, rho.clamp(lo, hi) * A, rho * A)
    kl, dkl = _kl(c["kl"], logp, s["ref"].double())
    used = s["weight"] != 0
    w = s["weight"].double()
    term = torch.where(used, w * (c["beta"] * kl - surr), 0.0)
    g = torch.where(used, w * (c["beta"] * dkl - torch.where(clipped, 0.0, rho * A)), 0.0).float()
    # softmax in 32 bits; the sampled token's column has the one
    p *= (-g / total.float())[:, None]
    p.scatter_add_(1, y, g[:, None])
    zero = torch.zeros_like(logp, dtype=torch.float32)
    return {"loss": term.sum().float().reshape(1), "dlogits": torch.where(used[:, None], p, 0.0).to(torch.bfloat16),
            "logp": torch.where(used, logp.float(), zero), "kl": torch.where(used, kl.float(), zero),
            "clip": (clipped & used).to(torch.uint8)}


def _kl(kind, logp, ref):
    """(estimate, its derivative by logp)."""
    d = logp - ref
    if kind == "k1":
        return d, torch.ones_like(d)
    if kind == "k2":
        return d * d / 2, d
    if kind == "k3":
        return torch.expm1(-d) + d, -torch.expm1(-d)
    return torch.zeros_like(d), torch.zeros_like(d)


def _own_rope(s):
    import long_context_grpo_gb300 as ls
    c = s["case"]
    q, k = ls.rope(s["q"], s["k"], s["freqs"], positions=s["positions"], interleaved=c["interleaved"],
                   attn_factor=s["factor"], inverse=c["inverse"])
    return {"q": q, "k": k}


def _turn(x, cos, sin, rot, interleaved):
    """x [T, H, D] with its first `rot` values rotated by the angles of cos, sin [T, rot / 2], in their type."""
    y = x.to(cos.dtype)
    c, n = cos[:, None], sin[:, None]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _angles(positions, freqs, factor, inverse, kind):
    a = positions.double()[:, None] * freqs.to(positions.device)[None]
    return (torch.cos(a) * factor).to(kind), ((-1.0 if inverse else 1.0) * torch.sin(a) * factor).to(kind)


def _plain_rope(s):
    c = s["case"]
    cos, sin = _angles(s["positions"], s["freqs"], s["factor"], c["inverse"], torch.float32)
    return {n: _turn(s[n], cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16) for n in ("q", "k")}


def _places(s):
    """(sequence, position) of every new token."""
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n, output_size=s["T"])
    return seq, s["len"].long()[seq] - n[seq] + torch.arange(s["T"], device=DEV) - cu[seq]


def _own_append(s):
    q, _ = s["cache"].append(s["k_new"], s["v_new"], s["cu"], q=s["q"], inv_freq=s["freqs"], attn_factor=s["factor"])
    return {"q": q, "k_pages": s["k"], "v_pages": s["v"]}


def _plain_append(s):
    c = s["case"]
    seq, pos = _places(s)
    cos, sin = _angles(pos, s["freqs"], s["factor"], False, torch.float32)
    page, slot = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    k = _turn(s["k_new"], cos, sin, c["D"], False).to(torch.bfloat16)
    if c["layout"] == "NHD":
        s["k"][page, slot] = k
        s["v"][page, slot] = s["v_new"]
    else:
        s["k"][page, :, slot] = k
        s["v"][page, :, slot] = s["v_new"]
    return {"q": _turn(s["q"], cos, sin, c["D"], False).to(torch.bfloat16), "k_pages": s["k"], "v_pages": s["v"]}


def _own_attn(s):
    c = s["case"]
    o, lse = s["cache"].attn(s["q"], s["cu"], max_new=s["max_new"], max_len=s["max_len"], group=c["group"],
                             shared_len=s["shared"], workspace=s["work"])
    return {"o": o, "lse": lse}


def _gathered(pages, s, kind):
    """The sequences' keys or values, [S, Hkv, L, D], zero behind each one's length."""
    c = s["case"]
    n = -(-s["max_len"] // c["page"])
    x = pages[s["table"][:, :n].clamp(min=0).long()]
    x = x.movedim(3, 1) if c["layout"] == "NHD" else x.movedim(2, 1)
    x = x.reshape(c["S"], c["Hkv"], n * c["page"], c["D"]).to(kind)
    return x * (torch.arange(n * c["page"], device=DEV) < s["len"].long()[:, None])[:, None, :, None]


def _attend(s, kind):
    """Attention of every new token over its sequence's keys up to its own, in `kind`."""
    c = s["case"]
    seq, pos = _places(s)
    at = torch.arange(s["T"], device=DEV) - s["cu"].long()[seq]
    k, v = _gathered(s["k"], s, kind), _gathered(s["v"], s, kind)
    S, Hkv, L, D = k.shape
    q = torch.zeros(S, s["max_new"], Hkv, c["Hq"] // Hkv, D, dtype=kind, device=DEV)
    last = torch.full((S, s["max_new"]), -1, device=DEV)
    q[seq, at] = s["q"].to(kind).reshape(s["T"], Hkv, -1, D)
    last[seq, at] = pos
    x = q.permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, D) @ k.transpose(-1, -2)
    x = x.reshape(S, Hkv, -1, s["max_new"], L).mul_(D ** -0.5)
    x.masked_fill_(torch.arange(L, device=DEV) > last[:, None, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.reshape(S, Hkv, -1, L) @ v).reshape(S, Hkv, -1, s["max_new"], D)
    o = (o / total.clamp(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(S, s["max_new"], c["Hq"], D)
    lse = (torch.log(total) + top).squeeze(-1).permute(0, 3, 1, 2).reshape(S, s["max_new"], c["Hq"])
    return o[seq, at], torch.where(pos[:, None] >= 0, lse[seq, at], -math.inf)


def _plain_attn(s):
    o, lse = _attend(s, torch.float32)
    return {"o": o.to(torch.bfloat16), "lse": lse}


def _own_fork(s):
    s["cache"].free(s["children"])
    s["cache"].fork(s["parents"], s["children"], workspace=s["work"])
    return {"table": s["table"], "len": s["len"], "ref": s["ref"], "k_pages": s["k"], "v_pages": s["v"]}


def _plain_fork(s):
    ps = s["case"]["page"]
    pa, ch, width = s["parents"].long(), s["children"].long(), s["table"].shape[1]
    old = s["table"][ch].long().flatten()
    gone = torch.zeros(len(s["ref"]) + 1, dtype=torch.int32, device=DEV)
    gone.scatter_add_(0, torch.where(old < 0, len(s["ref"]), old), torch.ones_like(old, dtype=torch.int32))
    s["ref"] -= gone[:-1]
    # whole pages shared, a part-filled last page copied into the lowest free ones in the pairs' order
    n = s["len"].long()[pa]
    full, part = n // ps, n % ps
    col = torch.arange(width, device=DEV)
    rows = torch.where(col < full[:, None], s["table"][pa].long(), -1)
    free = torch.argsort((s["ref"] > 0).to(torch.int8), stable=True)
    page = free[torch.cumsum((part > 0).long(), 0) - (part > 0).long()]
    rows = torch.where((col == full[:, None]) & (part > 0)[:, None], page[:, None], rows)
    now = rows.flatten()
    s["ref"] += torch.zeros_like(gone).scatter_add_(
        0, torch.where(now < 0, len(s["ref"]), now), torch.ones_like(now, dtype=torch.int32))[:-1]
    s["table"][ch], s["len"][ch] = rows.int(), n.int()
    src = s["table"][pa, full.clamp(max=width - 1)].long()
    # the whole page is taken along here; only its first tokens are the row's
    has = part > 0
    keep = torch.arange(ps, device=DEV) < part[has][:, None]
    keep = keep[:, :, None, None] if s["case"]["layout"] == "NHD" else keep[:, None, :, None]
    for x in (s["k"], s["v"]):
        x[page[has]] = torch.where(keep, x[src[has]], x[page[has]])
    return {"table": s["table"], "len": s["len"], "ref": s["ref"], "k_pages": s["k"], "v_pages": s["v"]}


def _own_compact(s):
    s["cache"].compact(s["cache2"], workspace=s["work"])
    return {"table": s["table2"], "len": s["len2"], "ref": s["ref2"], "k_pages": s["k2"], "v_pages": s["v2"]}


def _plain_compact(s):
    live = s["ref"] > 0
    to = torch.cumsum(live.long(), 0) - 1
    pages = torch.nonzero(live)[:, 0]
    s["k2"][:len(pages)], s["v2"][:len(pages)] = s["k"][pages], s["v"][pages]
    s["ref2"].zero_()
    s["ref2"][:len(pages)] = s["ref"][pages]
    s["table2"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()], -1))
    s["len2"].copy_(s["len"])
    return {"table": s["table2"], "len": s["len2"], "ref": s["ref2"], "k_pages": s["k2"], "v_pages": s["v2"]}


_own = {"loss": _own_loss, "rope": _own_rope, "append": _own_append, "attn": _own_attn, "fork": _own_fork,
        "compact": _own_compact}
_plain = {"loss": _plain_loss, "rope": _plain_rope, "append": _plain_append, "attn": _plain_attn, "fork": _plain_fork,
          "compact": _plain_compact}


# ------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "loss":
        T, V = case["T"], case["V"]
        return {"bytes": T * (4 * V + 4 * (4 + (case["kl"] != "none")) + 9) + 4, "flops": 8 * T * V}
    if op == "rope":
        n = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": 4 * n * case["D"] + 8 * case["T"], "flops": 3 * n * case["rot"]}
    if op == "append":
        n, _ = _lens(case)
        T = sum(n)
        H = case["Hq"] + 2 * case["Hkv"]
        return {"bytes": 4 * T * H * case["D"] + 12 * case["S"], "flops": 3 * T * (case["Hq"] + case["Hkv"]) * case["D"]}
    if op == "attn":
        n, kv = _lens(case)
        keys = sum(kv) - (case["group"] - 1) * case["shared"] * (case["S"] // case["group"])
        pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(n, kv))
        return {"bytes": 4 * keys * case["Hkv"] * case["D"] + sum(n) * case["Hq"] * (4 * case["D"] + 4),
                "flops": 4 * case["D"] * case["Hq"] * pairs}
    rng = random.Random(case["mix"])
    kv = [rng.randint(case["kv_min"], case["kv_max"]) for _ in range(case["P"] if op == "fork" else case["S"])]
    token = 4 * case["Hkv"] * case["D"]
    if op == "fork":  # a parent's part-filled page read once and written for each child; the table rows and counts
        part = sum(x % case["page"] for x in kv)
        full = sum(x // case["page"] for x in kv)
        return {"bytes": part * token * (1 + case["G"]) + full * (4 + 12 * case["G"]), "flops": full * case["G"]}
    live = sum(-(-x // case["page"]) for x in kv)
    return {"bytes": 2 * live * case["page"] * token + 24 * live, "flops": live}


# ----------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    op = case["op"]
    if op in ("fork", "compact"):
        return None
    if op == "attn" and work(case)["flops"] > 3.0e12:
        return None
    s = prepare(case, seed)
    if op == "loss":
        return _exact_loss(s)
    if op == "attn":
        return _exact_attn(s)
    if op == "rope":
        q, k = (_exact_turn(s[n], s["positions"], s["freqs"], s["factor"], case["rot"], case["interleaved"],
                            case["inverse"]) for n in ("q", "k"))
        return {"q": q, "k": k}
    seq, pos = _places(s)
    q = _exact_turn(s["q"], pos, s["freqs"], s["factor"], case["D"], False, False)
    # the cache's pages, token by token of each sequence
    k_new = _exact_turn(s["k_new"], pos, s["freqs"], s["factor"], case["D"], False, False)
    out = {"q": q, "k_pages": s["k"].double(), "v_pages": s["v"].double()}
    for b, (m, end) in enumerate(zip(*_lens(case))):
        at, places = int(s["cu"][b]), torch.arange(end - m, end, device=DEV)
        pages = s["table"][b].long()[places // case["page"]]
        for n, x in (("k_pages", k_new), ("v_pages", s["v_new"].double())):
            pool = out[n] if case["layout"] == "NHD" else out[n].transpose(1, 2)
            pool[pages, places % case["page"]] = x[at:at + m]
    return out


def _exact_loss(s):
    c = s["case"]
    out = {n: [] for n in ("dlogits", "logp", "kl")}
    loss = 0.0
    for a in range(0, c["T"], 256):
        i = slice(a, a + 256)
        x = s["logits"][i].double()
        soft = torch.log_softmax(x, 1)
        y = s["ids"][i].long()[:, None]
        logp = soft.gather(1, y)[:, 0]
        A, w = s["adv"][i].double(), s["weight"][i].double()
        rho = torch.exp(logp - s["old"][i].double())
        inside = torch.minimum(rho * A, rho.clamp(1 - s["eps"][0], 1 + s["eps"][1]) * A)
        r = torch.exp(s["ref"][i].double() - logp)
        kl, slope = {"none": (0 * r, 0 * r), "k1": (-torch.log(r), 0 * r + 1), "k2": (torch.log(r) ** 2 / 2, -torch.log(r)),
                     "k3": (r - 1 - torch.log(r), 1 - r)}[c["kl"]]
        moves = (inside == rho * A).double()
        g = w * (c["beta"] * slope - moves * rho * A)
        loss += float((w * (c["beta"] * kl - inside)).sum())
        used = (w != 0).double()
        soft = soft.exp_().mul_(-g[:, None])
        soft.scatter_add_(1, y, g[:, None])
        out["dlogits"].append(soft)
        out["logp"].append(logp * used)
        out["kl"].append(kl * used)
    return {"loss": torch.tensor([loss], dtype=torch.float64), "dlogits": torch.cat(out["dlogits"]),
            "logp": torch.cat(out["logp"]), "kl": torch.cat(out["kl"]), "clip": None}


def _exact_turn(x, positions, freqs, factor, rot, interleaved, inverse):
    """The pairs as complex numbers times factor exp(+-i angle)."""
    x = x.double()
    angle = positions.double()[:, None] * freqs.to(x.device)
    by = torch.polar(torch.full_like(angle, factor), -angle if inverse else angle)[:, None]
    y = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (rot // 2, 2)).contiguous()) * by
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * by
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def _exact_attn(s):
    """Sequence by sequence and key head by key head, with the softmax over the visible keys."""
    c = s["case"]
    n, kv = _lens(c)
    o = torch.zeros(s["T"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((s["T"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
    g, at = c["Hq"] // c["Hkv"], 0
    for b in range(c["S"]):
        pages = s["table"][b, :-(-kv[b] // c["page"])].long()
        k, v = (x[pages] if c["layout"] == "NHD" else x[pages].transpose(1, 2) for x in (s["k"], s["v"]))
        k, v = (x.reshape(-1, c["Hkv"], c["D"])[:kv[b]] for x in (k, v))
        hidden = torch.arange(kv[b], device=DEV)[None] > (kv[b] - n[b] + torch.arange(n[b], device=DEV))[:, None]
        for h in range(c["Hkv"] if n[b] else 0):
            q = s["q"][at:at + n[b], h * g:(h + 1) * g].double().transpose(0, 1)
            x = (q @ k[:, h].double().T / math.sqrt(c["D"])).masked_fill(hidden, -math.inf)
            lse[at:at + n[b], h * g:(h + 1) * g] = torch.logsumexp(x, -1).T
            o[at:at + n[b], h * g:(h + 1) * g] = (torch.softmax(x, -1) @ v[:, h].double()).transpose(0, 1)
        at += n[b]
    return {"o": o, "lse": lse}
