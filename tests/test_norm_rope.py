"""Norms of queries and keys with the rotation in the same pass, and the gradient, against float64.

Tolerances.  An output is rounded once to bf16 (2^-8 of it, twice the half step); the norm's sum, root and products and
the rotation's angle and products in fp32 are within 2^-18 of the pair's length (rope alone 2^-20).  A gradient is off
by its own rounding and 2^-17 of its two parts' sizes.  Weight gradients are fp32 sums of at most 2^8 additions
in a row on any term's way (a lane's heads, lanes, warps, blocks): 2^-16 of the terms' sizes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.norm_rope import norm, norm_rope, norm_rope_grad
from test_cache_attn import build, cu

EPS = 1e-6


def dbl(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, x, w, pos, f, inter, factor, offset=0.0):
    want = norm_rope(dbl(x), dbl(w), EPS, pos, f, inter, factor, offset)
    size = np.abs(norm(dbl(x), dbl(w), EPS, offset))
    if f is not None:
        n = len(f)
        re = np.arange(n) * 2 if inter else np.arange(n)
        im = re + 1 if inter else re + n
        size[..., re] = size[..., im] = size[..., re] + size[..., im]
    err = np.abs(dbl(got) - want)
    room = 2.0 ** -8 * np.abs(want) + max(factor, 1.0) * size * 2.0 ** -18
    assert (err <= room).all(), (err / np.maximum(room, 1e-300)).max()


def make(T, H, D, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(2.0 * torch.randn(T, H, 1, generator=g))
    return (torch.randn(T, H, D, generator=g) * size).to(torch.bfloat16).cuda()


CASES = [(1, 2, 2, 64, 64, False), (7, 3, 1, 64, 32, False), (130, 8, 2, 128, 128, True), (33, 40, 8, 128, 20, False),
         (5, 1, 1, 128, 2, True), (12, 2, 1, 96, 48, True), (9, 4, 2, 6, 6, False), (65, 64, 8, 128, 128, False),
         (3, 2, 1, 256, 256, False), (3, 5, 1, 72, 40, True), (2000, 4, 1, 128, 64, False), (11, 3, 5, 80, 32, False),
         (40, 7, 0, 16, 16, False), (17, 0, 3, 48, 24, True), (6, 2, 2, 256, 128, True), (4, 3, 1, 32, 0, False),
         (2600, 5, 2, 64, 64, False), (9, 3, 2, 18, 0, False)]


def inputs(T, Hq, Hk, D, rot, kind, offset=0):
    import long_context_grpo_gb300 as ls
    g = torch.Generator().manual_seed(T + D + Hq)
    q, k = (make(T, H, D, T + H + i) if H else None for i, H in enumerate((Hq, Hk)))
    wq, wk = ((1.0 - offset + 0.5 * torch.randn(D, generator=g)).to(kind).cuda() for _ in range(2))
    pos = torch.randint(0, 1 << 21, (T,), generator=g).cuda()
    f, a = ls.rope_freqs(rot, 1e6, "ramp", 4.0, 32768) if rot else (None, 1.0)
    return q, k, wq, wk, pos, f, a


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", CASES)
@pytest.mark.parametrize("kind,offset", [(torch.bfloat16, 0.0), (torch.float32, 1.0)])
def test_against_float64(T, Hq, Hk, D, rot, inter, kind, offset):
    import long_context_grpo_gb300 as ls
    q, k, wq, wk, pos, f, a = inputs(T, Hq, Hk, D, rot, kind, offset)
    qo, ko = ls.norm_rope(q, k, wq, wk, f, eps=EPS, positions=pos, interleaved=inter, attn_factor=a, weight_offset=offset)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        if x is None:
            assert y is None
        else:
            close(y, x, w, dbl(pos), None if f is None else f.numpy(), inter, a, offset)
    # without weights: 1, whatever the offset
    qo, ko = ls.norm_rope(q, k, None, None, f, eps=EPS, positions=pos, interleaved=inter, attn_factor=a, weight_offset=offset)
    for x, y in ((q, qo), (k, ko)):
        if x is not None:
            close(y, x, None, dbl(pos), None if f is None else f.numpy(), inter, a)


def grad_close(got, dy, x, w, pos, f, inter, factor, offset=0.0):
    dx, dw, size, terms = norm_rope_grad(dbl(dy), dbl(x), dbl(w), EPS, pos, f, inter, factor, offset)
    gx, gw = got
    if f is not None:            # (a pair's values are of the pair's length)
        size = size + 2.0 ** 7 * 2.0 ** -8 * np.abs(size).max(-1, keepdims=True)
    err = np.abs(dbl(gx) - dx)
    room = 2.0 ** -8 * np.abs(dx) + 2.0 ** -17 * size
    assert (err <= room).all(), (err / np.maximum(room, 1e-300)).max()
    if w is None:
        assert gw is None
    else:
        assert (np.abs(dbl(gw) - dw) <= 2.0 ** -16 * terms + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", CASES)
@pytest.mark.parametrize("kind,offset", [(torch.float32, 0.0), (torch.bfloat16, 1.0)])
def test_gradient_against_float64(T, Hq, Hk, D, rot, inter, kind, offset):
    import long_context_grpo_gb300 as ls
    q, k, wq, wk, pos, f, a = inputs(T, Hq, Hk, D, rot, kind, offset)
    dq, dk = (None if x is None else torch.randn(x.shape, device="cuda").to(torch.bfloat16) for x in (q, k))
    kw = dict(eps=EPS, positions=pos, interleaved=inter, attn_factor=a)
    r = ls.norm_rope_bwd(dq, dk, q, k, wq, wk, f, weight_offset=offset, **kw)
    fn = None if f is None else f.numpy()
    for dy, x, w, got in ((dq, q, wq, (r.dq, r.dq_weight)), (dk, k, wk, (r.dk, r.dk_weight))):
        if x is None:
            assert got == (None, None)
        else:
            grad_close(got, dy, x, w, dbl(pos), fn, inter, a, offset)
    again = ls.norm_rope_bwd(dq, dk, q, k, wq, wk, f, weight_offset=offset, **kw)
    assert all(x is None or torch.equal(x, y) for x, y in zip(r, again))
    r = ls.norm_rope_bwd(dq, dk, q, k, None, None, f, **kw)
    for dy, x, got in ((dq, q, (r.dq, r.dq_weight)), (dk, k, (r.dk, r.dk_weight))):
        if x is not None:
            grad_close(got, dy, x, None, dbl(pos), fn, inter, a)


@pytest.mark.gpu
def test_gradients_are_differences():
    """One input and one weight moved each way, in float64 of the formula."""
    import long_context_grpo_gb300 as ls
    T, H, D = 4, 3, 64
    q, _, w, _, pos, f, a = inputs(T, H, 0, D, D, torch.float32)
    dy = torch.randn(T, H, D, device="cuda").to(torch.bfloat16)
    r = ls.norm_rope_bwd(dy, None, q, None, w, None, f, eps=EPS, positions=pos, attn_factor=a)
    X, W, G, P = dbl(q), dbl(w), dbl(dy), dbl(pos)
    total = lambda x, v: (norm_rope(x, v, EPS, P, f.numpy(), False, a) * G).sum()  # noqa: E731
    _, _, size, terms = norm_rope_grad(G, X, W, EPS, P, f.numpy(), False, a)
    for at in ((0, 0, 0), (1, 2, 40), (3, 1, 63)):
        h = 1e-5 * np.abs(X[at[:2]]).max()
        ends = []
        for s in (h, -h):
            y = X.copy()
            y[at] += s
            ends.append(total(y, W))
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(float(r.dq[at]) - slope) <= 2.0 ** -7 * abs(slope) + 2.0 ** -15 * size[at[:2]].max()
    for d in (0, 33):
        ends = []
        for s in (1e-5, -1e-5):
            v = W.copy()
            v[d] += s
            ends.append(total(X, v))
        assert abs(float(r.dq_weight[d]) - (ends[0] - ends[1]) / 2e-5) <= 2.0 ** -15 * terms[d] + 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("offset,stride_extra", [(0, 0), (8, 16), (1, 3), (2, 0)])
def test_strided_rows_of_a_fused_projection_and_in_place(offset, stride_extra):
    import long_context_grpo_gb300 as ls
    T, H, D = 19, 3, 64
    flat = torch.randn(T, 2 * H * D + stride_extra + offset, device="cuda").to(torch.bfloat16)
    dflat = torch.randn(flat.shape, device="cuda").to(torch.bfloat16)
    keep, dkeep = flat.clone(), dflat.clone()
    view = lambda t: (t[:, offset:offset + H * D].unflatten(1, (H, D)),  # noqa: E731
                      t[:, offset + H * D:offset + 2 * H * D].unflatten(1, (H, D)))
    (q, k), (dq, dk) = view(flat), view(dflat)
    w = torch.randn(D, device="cuda")
    f, _ = ls.rope_freqs(32, 1e4)
    kw = dict(pos0=77)
    # (a contiguous copy may take the other path: equal up to the order of fp32 sums, one bf16 step)
    want = ls.norm_rope(q.contiguous(), k.contiguous(), w, w, f, **kw)
    grads = ls.norm_rope_bwd(dq.contiguous(), dk.contiguous(), q.contiguous(), k.contiguous(), w, w, f, **kw)
    r = ls.norm_rope_bwd(dq, dk, q, k, w, w, f, dq_out=dq, dk_out=dk, **kw)
    assert r.dq is dq
    ls.norm_rope(q, k, w, w, f, q_out=q, k_out=k, **kw)
    for a, b in ((q, want[0]), (k, want[1]), (dq, grads.dq), (dk, grads.dk)):
        err = (a.double() - b.double()).abs()
        assert bool((err <= 2.0 ** -7 * b.double().abs() + 2.0 ** -16 * b.double().abs().amax(-1, keepdim=True)).all())
    for a, b in ((flat, keep), (dflat, dkeep)):
        assert torch.equal(a[:, :offset], b[:, :offset])
        assert torch.equal(a[:, offset + 2 * H * D:], b[:, offset + 2 * H * D:])


@pytest.mark.gpu
def test_heads_of_zeros_and_of_infinities():
    import long_context_grpo_gb300 as ls
    q = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    q[0, 1] = 0
    q[2, 0, 5] = float("nan")
    q[3, 1, 7] = float("inf")
    w = torch.ones(64, device="cuda")
    y, none = ls.norm_rope(q, None, w, None, ls.rope_freqs(64)[0])
    assert none is None
    assert not y[0, 1].any() and torch.isnan(y[2, 0]).all() and torch.isnan(y[3, 1, 7])
    ok = torch.ones(4, 2, dtype=torch.bool, device="cuda")
    ok[0, 1] = ok[2, 0] = ok[3, 1] = False
    assert torch.isfinite(y[ok]).all()
    dy = torch.randn(4, 2, 64, device="cuda").to(torch.bfloat16)
    r = ls.norm_rope_bwd(dy[:1], None, q[:1], None, w, None, ls.rope_freqs(64)[0])
    assert torch.isfinite(r.dq).all() and float(r.dq[0, 1].float().abs().max()) > 100.0     # 1 / sqrt(eps) there


@pytest.mark.gpu
@pytest.mark.parametrize("layout,ps", [("NHD", 16), ("HND", 64), ("NHD", 256)])
@pytest.mark.parametrize("rot,inter", [(128, False), (64, True), (20, False), (None, False)])
@pytest.mark.parametrize("weighted", [True, False])
def test_append_with_norms(layout, ps, rot, inter, weighted):
    import long_context_grpo_gb300 as ls
    lens, new = [5, 400, 0, 77, 260], [5, 130, 0, 3, 1]
    mk, table = build(lens, ps, 2, 128, layout, seed=4, width=30)
    c = mk(6)
    T = sum(new) + 2
    k, v = make(T, 2, 128, 1), make(T, 2, 128, 2)
    q = make(T, 6, 128, 3)
    wq, wk = (torch.randn(128, device="cuda").to(torch.bfloat16) if weighted else None for _ in range(2))
    before = c.k_pages.clone(), c.v_pages.clone()
    f, a = ls.rope_freqs(rot, 1e4) if rot else (None, 1.0)
    q_out = torch.full_like(q, 7.0)
    c.append(k, v, cu(new, 1), q=q, q_out=q_out, inv_freq=f, interleaved=inter, attn_factor=a, q_weight=wq, k_weight=wk,
             norm_eps=EPS)
    assert ls.device_status() == (0, 0)
    want_k, want_v = before
    at = 1
    for b, n in enumerate(new):
        pos = torch.arange(lens[b] - n, lens[b], device="cuda")
        if n:
            # the bits of the pass without pages
            qb, kb = ls.norm_rope(q[at:at + n], k[at:at + n], wq, wk, f, eps=EPS, positions=pos, interleaved=inter, attn_factor=a)
            assert torch.equal(q_out[at:at + n], qb)
            close(kb, k[at:at + n], wk, dbl(pos), None if f is None else f.numpy(), inter, a)
        for i in range(n):
            p, s = int(table[b, int(pos[i]) // ps]), int(pos[i]) % ps
            sl = (p, s) if layout == "NHD" else (p, slice(None), s)
            want_k[sl], want_v[sl] = kb[i], v[at + i]
        at += n
    assert torch.equal(c.k_pages, want_k) and torch.equal(c.v_pages, want_v)
    assert (q_out[0] == 7).all() and (q_out[T - 1] == 7).all()


@pytest.mark.gpu
def test_append_with_norms_leaves_out_what_has_no_place():
    import long_context_grpo_gb300 as ls
    mk, table = build([3, 40, 20], 16, 1, 64, seed=5, width=4)
    c = mk(2)
    k, v, q = make(9, 1, 64, 1), make(9, 1, 64, 2), make(9, 2, 64, 3)
    f = ls.rope_freqs(64)[0]
    before, out = c.k_pages.clone(), torch.full_like(q, 7.0)
    call = lambda n, **kw: c.append(k[:n], v[:n], cu([n]), q=q[:n], q_out=out[:n], inv_freq=f, norm_eps=EPS, **kw)  # noqa: E731
    want = ls.norm_rope(q[:5], k[:5], None, None, f, pos0=-2)
    call(5)                       # five new tokens of a length of three: two are left out
    before[table[0, 0], :3] = want[1][2:]
    assert torch.equal(c.k_pages, before) and (out[:2] == 7).all() and torch.equal(out[2:5], want[0][2:])
    assert ls.device_status() == (0, 0)
    for offsets in ((0, 9, 4, 9), (-1, 3, 6, 9), (0, 3, 6, 10)):
        out.fill_(7.0)
        c.append(k, v, torch.tensor(offsets, dtype=torch.int32, device="cuda"), q=q, q_out=out, inv_freq=f, norm_eps=EPS)
        assert ls.device_status() == (7, 2) and torch.equal(c.k_pages, before) and bool((out == 7).all())
    c.append(k, v, cu([9]), rows=torch.tensor([3], dtype=torch.int32, device="cuda"), norm_eps=EPS)
    assert torch.equal(c.k_pages, before) and ls.device_status() == (7, 2)


@pytest.mark.gpu
def test_captured_with_a_workspace_on_two_streams():
    import long_context_grpo_gb300 as ls
    T, D = 700, 128
    q, k, wq, wk, pos, f, a = inputs(T, 8, 2, D, D, torch.float32)
    dq, dk = torch.randn(T, 8, D, device="cuda").to(torch.bfloat16), torch.randn(T, 2, D, device="cuda").to(torch.bfloat16)
    kw = dict(positions=pos, attn_factor=a)
    want = [t.clone() for t in ls.norm_rope_bwd(dq, dk, q, k, wq, wk, f, **kw)]
    ws = torch.empty(ls.norm_rope_bwd_workspace_bytes(T, D), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = ls.norm_rope_bwd(dq, dk, q, k, wq, wk, f, workspace=ws, **kw)
    side = torch.cuda.Stream()
    for _ in range(3):
        ws.fill_(0xFF)
        for t in got:
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = ls.norm_rope_bwd(dq, dk, q, k, wq, wk, f, **kw)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and all(torch.equal(x, y) for x, y in zip(other, want))


def test_refusals():
    from long_context_grpo_gb300 import build as lsbuild
    lsbuild.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    f = (ctypes.c_double * 64)(*([0.1] * 64))
    base = dict(T=4, Hq=2, Hk=1, D=64, rot_dim=64, inv_freq=ctypes.addressof(f), attn_factor=1.0, q=0x1000, q_stride=128,
                q_out=0x2000, q_out_stride=128, k=0x3000, k_stride=64, k_out=0x4000, k_out_stride=64)
    nbase = dict(q_weight=0x5000, k_weight=0x6000, weight_fp32=0, weight_offset=0.0, eps=1e-6)
    gbase = dict(q_in=0x7000, q_in_stride=128, k_in=0x8000, k_in_stride=64, dq_weight=0x9000, dk_weight=0xa000)

    def call(n=None, **kw):
        return L.ls_norm_rope(ctypes.byref(b.RopeDesc(**{**base, **kw})), ctypes.byref(b.HeadNorm(**{**nbase, **(n or {})})), None)

    def back(n=None, g=None, ws=0xb000, size=1 << 24, **kw):
        return L.ls_norm_rope_bwd(ctypes.byref(b.RopeDesc(**{**base, **kw})), ctypes.byref(b.HeadNorm(**{**nbase, **(n or {})})),
                                  ctypes.byref(b.HeadNormGrad(**{**gbase, **(g or {})})), ws, size, None)

    nan, inf = float("nan"), float("inf")
    ok = b.RopeDesc(**base)
    assert L.ls_norm_rope(None, ctypes.byref(b.HeadNorm(**nbase)), None) == 1
    assert L.ls_norm_rope(ctypes.byref(ok), None, None) == 1
    assert L.ls_norm_rope_bwd(ctypes.byref(ok), ctypes.byref(b.HeadNorm(**nbase)), None, 0xb000, 1 << 24, None) == 1
    for fn in (call, back):
        for kw in (dict(T=0), dict(Hq=0, Hk=0), dict(Hq=-1), dict(inv_freq=None), dict(rot_dim=0), dict(q=None), dict(k_out=None),
                   dict(q_stride=127), dict(k_out_stride=63), dict(rot_dim=66), dict(rot_dim=31), dict(attn_factor=nan),
                   dict(q_out=0x1000, q_out_stride=256), dict(inverse=1)):
            assert fn(**kw) == 1, kw
        for n in (dict(eps=0.0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(eps=1e-60), dict(weight_offset=nan),
                  dict(weight_offset=inf)):
            assert fn(n=n) == 1, n
        assert fn(D=258, q_stride=600, q_out_stride=600, k_stride=300, k_out_stride=300) == 2
        assert fn(T=1 << 31) == 2 and fn(q=0x1001) == 4
        assert fn(n=dict(q_weight=0x5001)) == 4 and fn(n=dict(k_weight=0x6002, weight_fp32=1)) == 4
    for g in (dict(q_in=None), dict(k_in=None), dict(q_in_stride=127), dict(k_in_stride=63)):
        assert back(g=g) == 1, g
    assert back(Hk=0) == 1                                # a weight gradient of no heads
    assert back(ws=None) == 8 and back(size=100) == 8 and back(ws=0xb008) == 4
    assert back(g=dict(dq_weight=0x9002)) == 4 and back(g=dict(q_in=0x7001)) == 4
    assert L.ls_norm_rope_bwd_workspace_bytes(0, 64) == 0 and L.ls_norm_rope_bwd_workspace_bytes(4, 300) == 0
    assert L.ls_cache_append_norm(None, None, None, None) == 3


def test_packed_descriptors_have_the_structures_layout():
    from long_context_grpo_gb300 import _lib as b
    from long_context_grpo_gb300 import _ops
    for s, D in ((_ops._NORM, b.HeadNorm), (_ops._NORM_GRAD, b.HeadNormGrad)):
        values = [float(i + 1) if k is ctypes.c_double else i + 1 for i, (_, k) in enumerate(D._fields_)]
        got = D.from_buffer_copy(s.pack(*values).ljust(ctypes.sizeof(D), b"\0"))
        assert [getattr(got, n) for n, _ in D._fields_] == values
