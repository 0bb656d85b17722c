"""Clipped policy loss with a KL term over packed tokens, float64, row by row.  TEST
INFRASTRUCTURE ONLY."""
import numpy as np

from ._np import to_np


def policy_loss(logits, ids, logp_old, advantages, weights, eps_low, eps_high, logp_ref=None, beta=0.0,
                kl="none"):
    """loss, and per token: g = d loss / d logp, p (softmax row), dlogits, logp, kl, clip, terms."""
    x = to_np(logits)
    ids, A, w, old = (np.asarray(to_np(v)) for v in (ids, advantages, weights, logp_old))
    ids = ids.astype(np.int64)
    T, V = x.shape
    out = dict(logp=np.zeros(T), kl=np.zeros(T), clip=np.zeros(T, dtype=bool), terms=np.zeros(T),
               g=np.zeros(T), p=np.zeros((T, V)), dlogits=np.zeros((T, V)), d=np.zeros(T))
    ref = None if logp_ref is None else to_np(logp_ref)
    for t in range(T):
        if w[t] == 0 or not 0 <= ids[t] < V:
            continue
        m = x[t].max()
        e = np.exp(x[t] - m)
        logp = x[t, ids[t]] - m - np.log(e.sum())
        d = logp - old[t]
        rho = np.exp(d)
        clip = (A[t] > 0 and rho > 1 + eps_high) or (A[t] < 0 and rho < 1 - eps_low)
        surr = min(rho * A[t], min(max(rho, 1 - eps_low), 1 + eps_high) * A[t])
        k = dk = 0.0
        if kl != "none":
            r = logp - ref[t]
            k, dk = {"k1": (r, 1.0), "k2": (r * r / 2, r), "k3": (np.exp(-r) + r - 1, 1 - np.exp(-r))}[kl]
        out["logp"][t], out["kl"][t], out["clip"][t], out["d"][t] = logp, k, clip, d
        out["terms"][t] = w[t] * (beta * k - surr)
        g = w[t] * (beta * dk - (0.0 if clip else A[t] * rho))
        out["g"][t] = g
        out["p"][t] = e / e.sum()
        out["dlogits"][t] = -g * out["p"][t]
        out["dlogits"][t, ids[t]] += g
    out["loss"] = out["terms"].sum()
    return out
