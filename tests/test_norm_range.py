"""Norms of heads near the largest squares that fp32 holds, beside ordinary heads, against float64: right up to there, NaN (not
0) past it.  Tolerances as in test_norm_rope.py."""
import numpy as np
import pytest
import torch

from oracle.norm_rope import norm, norm_rope, norm_rope_grad
from test_cache_attn import build, cu
from test_norm_rope import EPS, dbl

# tokens, query and key heads, head size, rotated values, pairs: 16-byte paths of every width, then the element path
SHAPES = [(40, 5, 2, 128, 128, False), (33, 4, 1, 64, 32, True), (70, 3, 1, 256, 256, False), (9, 2, 2, 16, 16, False),
          (21, 3, 0, 48, 0, False), (15, 3, 2, 72, 40, True)]
SCALES = [1e-30, 1e-20, 1e-13, 1.0, 1e10, 1e17]


def heads(T, H, D, seed):
    """Heads of all sizes, neighbours of one another; tokens 2 and 3 have one whose squares pass fp32, token 4 one of
    which they just do not."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g)
    x *= torch.tensor(SCALES)[torch.randint(0, len(SCALES), (T, H, 1), generator=g)]
    x[1], x[2, 0, 3], x[3, -1, D - 1] = 0.0, 3e38, 1.9e19
    x[4, 0], x[4, 0, 5] = 1.0, 1.8e19        # 3.24e38
    far = torch.zeros(T, H, dtype=torch.bool)
    far[2, 0] = far[3, -1] = True
    return x.to(torch.bfloat16).cuda(), far.numpy()


def inputs(T, Hq, Hk, D, rot):
    import long_context_grpo_gb300 as ls
    g = torch.Generator().manual_seed(D)
    (q, qf), (k, kf) = (heads(T, H, D, T + H) if H else (None, None) for H in (Hq, Hk))
    w = (1.0 + 0.5 * torch.randn(D, generator=g)).cuda()
    return q, qf, k, kf, w, ls.rope_freqs(rot)[0] if rot else None


def paired(size, f, inter, D):
    if f is not None:
        re = np.arange(len(f)) * 2 if inter else np.arange(len(f))
        im = re + 1 if inter else re + len(f)
        size[..., re] = size[..., im] = size[..., re] + size[..., im]
    return size


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", SHAPES)
def test_norms_of_large_heads(T, Hq, Hk, D, rot, inter):
    import long_context_grpo_gb300 as ls
    q, qf, k, kf, w, f = inputs(T, Hq, Hk, D, rot)
    for x, far, y in zip((q, k), (qf, kf), ls.norm_rope(q, k, w, w, f, eps=EPS, interleaved=inter)):
        if x is None:
            continue
        want = norm_rope(dbl(x), dbl(w), EPS, np.arange(T), None if f is None else f.numpy(), inter)
        size = paired(np.abs(norm(dbl(x), dbl(w), EPS)), f, inter, D)
        y = dbl(y)
        assert np.isnan(y[far]).all()
        err = np.abs(y - want)[~far]
        assert (err <= (2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 2.0 ** -133)[~far]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", SHAPES)
def test_gradients_of_large_heads(T, Hq, Hk, D, rot, inter):
    import long_context_grpo_gb300 as ls
    q, qf, k, kf, w, f = inputs(T, Hq, Hk, D, rot)
    dq, dk = (None if x is None else torch.randn(x.shape, device="cuda").to(torch.bfloat16) for x in (q, k))
    r = ls.norm_rope_bwd(dq, dk, q, k, w, w, f, eps=EPS, interleaved=inter)
    for dy, x, far, gx, gw in ((dq, q, qf, r.dq, r.dq_weight), (dk, k, kf, r.dk, r.dk_weight)):
        if x is None:
            continue
        dx, _, part, _ = norm_rope_grad(dbl(dy), dbl(x), dbl(w), EPS, np.arange(T), None if f is None else f.numpy(), inter)
        if f is not None:
            part = part + 0.5 * np.abs(part).max(-1, keepdims=True)
        gx = dbl(gx)
        assert np.isnan(gx[far]).all() and torch.isnan(gw).all()
        err = np.abs(gx - dx)[~far]
        assert (err <= (2.0 ** -8 * np.abs(dx) + 2.0 ** -17 * part + 2.0 ** -133)[~far]).all()


@pytest.mark.gpu
def test_appended_large_heads():
    import long_context_grpo_gb300 as ls
    make, table = build([40], 16, 2, 64, seed=3)
    c = make(4)
    (k, far), (v, _) = heads(40, 2, 64, 5), heads(40, 2, 64, 6)
    w = torch.ones(64, device="cuda")
    f = ls.rope_freqs(64)[0]
    _, want = ls.norm_rope(None, k, None, w, f)
    c.append(k, v, cu([40]), inv_freq=f, k_weight=w, norm_eps=EPS)
    pages = [int(p) for p in table[0][:3]]
    got = c.k_pages[pages].reshape(-1, 2, 64)[:40]
    assert torch.isnan(got[torch.from_numpy(far)]).all()
    assert torch.equal(got[~torch.from_numpy(far)], want[~torch.from_numpy(far)])
    assert torch.equal(c.v_pages[pages].reshape(-1, 2, 64)[:40], v)
