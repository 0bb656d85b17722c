"""Scores of given tokens on the host, float64: log-probability, log-sum-exp, entropy, alternatives, gradient.
TEST INFRASTRUCTURE ONLY."""
import numpy as np


def scores(x, ids, top=0, temperature=1.0):
    """(logp, lse, entropy, top_ids, top_logp) of logits x [T, V]."""
    z = np.asarray(x, dtype=np.float64) / temperature
    T, V = z.shape
    bad = np.isnan(z).any(1) | np.isposinf(z).any(1) | np.isneginf(z).all(1)
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        e = np.exp(z - m)
        lse = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
        p = e / e.sum(1, keepdims=True)
        ent = -np.where(p > 0, p * np.log(np.where(p > 0, p, 1.0)), 0.0).sum(1)
        ok = (ids >= 0) & (ids < V)
        # (by the difference to the maximum: exact where the row's logits are far from zero)
        logp = np.where(ok, z[np.arange(T), np.where(ok, ids, 0)] - m[:, 0] - np.log(e.sum(1)), 0.0)
        order = np.argsort(-z, axis=1, kind="stable")[:, :top]
        tl = np.take_along_axis(z, order, 1) - m - np.log(e.sum(1, keepdims=True))
    lse[bad] = ent[bad] = np.nan
    logp[bad & ok] = np.nan
    order[bad], tl[bad] = -1, np.nan
    return logp, lse, ent, order, tl


def scores_grad(x, ids, d_logp, d_entropy, temperature=1.0):
    """d loss / d x."""
    z = np.asarray(x, dtype=np.float64) / temperature
    logp = z - z.max(1, keepdims=True)
    logp = logp - np.log(np.exp(logp).sum(1, keepdims=True))
    p = np.exp(logp)
    pl = np.where(p > 0, p * np.where(p > 0, logp, 0.0), 0.0)
    one = np.zeros_like(p)
    one[np.arange(len(z)), ids] = 1.0
    return (d_logp[:, None] * (one - p) - d_entropy[:, None] * (pl - p * pl.sum(1, keepdims=True))) / temperature
