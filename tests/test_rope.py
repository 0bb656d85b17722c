"""Rotary positions against float64: layouts, parts of the head, strides, far positions, scaling,
the gradient.  One rounding to bf16 (2^-8 of the value) of an fp32 rotation whose angle is right
to 2^-23 half turns (2^-20 of the pair's length in all)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.rope import freqs as ref_freqs
from oracle.rope import rope as ref_rope


def _close(got, x, want, rot, interleaved, factor=1.0):
    x = np.abs(np.asarray(x.double().cpu()))
    size = x.copy()
    n = rot // 2
    re = np.arange(n) * 2 if interleaved else np.arange(n)
    im = re + 1 if interleaved else re + n
    size[..., re] = size[..., im] = x[..., re] + x[..., im]
    tol = np.abs(want) * 2 ** -8 + factor * size * 2 ** -20
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


CASES = [(1, 2, 2, 64, 64, False), (7, 3, 1, 64, 32, False), (130, 8, 2, 128, 128, True), (33, 40, 8, 128, 20, False),
         (5, 1, 1, 128, 2, True), (12, 2, 1, 96, 48, True), (9, 4, 2, 6, 6, False), (65, 64, 8, 128, 128, False),
         (3, 2, 1, 256, 256, False), (3, 5, 1, 72, 40, True), (2000, 4, 1, 128, 64, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,D,rot,inter", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_against_float64(T, Hq, Hk, D, rot, inter, inverse):
    import long_context_grpo_gb300 as ls
    g = torch.Generator().manual_seed(T + D)
    q = torch.randn(T, Hq, D, generator=g).to(torch.bfloat16)
    k = torch.randn(T, Hk, D, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 21, (T,), generator=g)
    f, a = ls.rope_freqs(rot, 1e6, "ramp", 4.0, 32768)
    qo, ko = ls.rope(q.cuda(), k.cuda(), f, positions=pos.cuda(), interleaved=inter, attn_factor=a, inverse=inverse)
    for x, y in ((q, qo), (k, ko)):
        want = ref_rope(x.double().numpy(), pos.numpy(), f.numpy(), inter, a, inverse)
        _close(y, x, want, rot, inter, a)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


@pytest.mark.gpu
@pytest.mark.parametrize("pos0", [0, 1, -5, (1 << 21) + 3, (1 << 31) - 300, -(1 << 31)])
def test_far_and_negative_positions(pos0):
    import long_context_grpo_gb300 as ls
    x = torch.randn(200, 1, 128).to(torch.bfloat16)
    f, _ = ls.rope_freqs(128, 10000.0)
    y, none = ls.rope(x.cuda(), None, f, pos0=pos0)
    assert none is None
    pos = pos0 + np.arange(200)
    # the angle of the definition, reduced in integers: pos * f in float64 is off by 2^-53 pos
    _close(y, x, ref_rope(x.double().numpy(), pos, f.numpy()), 128, False, 1.0 + 2 ** -53 * abs(pos0) * 2 ** 20)


@pytest.mark.gpu
@pytest.mark.parametrize("offset,stride_extra", [(0, 0), (8, 16), (1, 3), (2, 0)])
def test_strided_rows_of_a_fused_projection_and_in_place(offset, stride_extra):
    import long_context_grpo_gb300 as ls
    T, H, D = 19, 3, 64
    flat = torch.randn(T, 2 * H * D + stride_extra + offset, device="cuda").to(torch.bfloat16)
    keep = flat.clone()
    q = flat[:, offset:offset + H * D].unflatten(1, (H, D))
    k = flat[:, offset + H * D:offset + 2 * H * D].unflatten(1, (H, D))
    f, _ = ls.rope_freqs(32, 1e4)
    want = [t.clone() for t in ls.rope(q.contiguous(), k.contiguous(), f, pos0=77)]
    ls.rope(q, k, f, pos0=77, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(flat[:, :offset], keep[:, :offset]) and torch.equal(flat[:, offset + 2 * H * D:], keep[:, offset + 2 * H * D:])


@pytest.mark.gpu
def test_gradient_is_the_transposed_map():
    """<dy, R x> = <R^T dy, x> in float64 of the rounded values, up to the roundings of both."""
    import long_context_grpo_gb300 as ls
    x, dy = (torch.randn(50, 4, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
    f, a = ls.rope_freqs(128, 1e6, "ramp", 8.0, 4096)
    y, _ = ls.rope(x, None, f, pos0=100000, attn_factor=a)
    dx, _ = ls.rope(None, dy, f, pos0=100000, attn_factor=a, inverse=True)[::-1]
    lhs, rhs = (y.double() * dy.double()).sum(), (x.double() * dx.double()).sum()
    assert abs(lhs - rhs) <= 2 ** -8 * ((y.double() * dy.double()).norm() + (x.double() * dx.double()).norm()) * 4
    # and against a difference along one input value: the map is linear
    e = torch.zeros_like(x)
    e[7, 2, 5] = 1.0
    step, _ = ls.rope(e, None, f, pos0=100000, attn_factor=a)
    assert abs((step.double() * dy.double()).sum() - dx[7, 2, 5].double()) <= 2 ** -6 * dy[7, 2].double().abs().max()


@pytest.mark.parametrize("kind", ["none", "linear", "ramp"])
@pytest.mark.parametrize("rot,theta,factor,orig", [(128, 1e6, 8.0, 32768), (64, 1e4, 2.5, 4096), (2, 5.0, 1.0, 7)])
def test_frequencies(kind, rot, theta, factor, orig):
    import long_context_grpo_gb300 as ls
    from long_context_grpo_gb300 import build
    build.build()
    f, a = ls.rope_freqs(rot, theta, kind, factor, orig)
    want, wa = ref_freqs(rot, theta, kind, factor, orig)
    np.testing.assert_allclose(f.numpy(), want, rtol=1e-14)
    assert abs(a - wa) <= 1e-15 * abs(wa)


def test_turns_in_fixed_point():
    """position * turns modulo 2^64 is the fraction of a turn: checked through the library's own
    conversion, compiled here, with exact rational arithmetic."""
    import os
    import subprocess
    import tempfile
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = ('#include <cstdio>\n#include <cstdlib>\n#include "%s/long_context_grpo_gb300/csrc/ls_rope_host.h"\n'
           'int main(int c, char** v) { for (int i = 1; i < c; ++i) { double f = atof(v[i]); static ls::RopeArgs a;'
           ' if (!ls::rope_turns(&f, 2, 1.0, &a)) { puts("refused"); continue; }'
           ' printf("%%llu\\n", (unsigned long long)a.turns[0]); } }' % root)
    values = [1.0, 0.5, 1e-6, 3.0, 6.283185307179586, 123.456, -0.25, 1e5, 0.8659643233600653, 2.0 ** -60]
    with tempfile.TemporaryDirectory() as d:
        open(d + "/t.cpp", "w").write(src)
        subprocess.run(["g++", "-std=c++17", "-O1", "-I/usr/local/cuda/include", d + "/t.cpp", "-o", d + "/t"], check=True)
        out = subprocess.run([d + "/t"] + [repr(v) for v in values] + ["inf", "nan", "1e9"], capture_output=True, text=True,
                             check=True).stdout.split()
    assert out[-3:] == ["refused"] * 3
    for v, u in zip(values, out):
        want = Decimal(v) / two_pi * 2 ** 64
        err = Decimal(int((Decimal(int(u)) - want) * 1024) % (2 ** 74)) / 1024
        # 1e5 / 2 pi has its fma error (2^-53 of 2^14, squared away) well below these units
        assert min(err, 2 ** 64 - err) <= 2, (v, u)


def test_refusals():
    from long_context_grpo_gb300 import build
    build.build()
    from long_context_grpo_gb300 import _lib as b
    L = b._lib()
    f = (ctypes.c_double * 64)(*([0.1] * 64))
    base = dict(T=4, Hq=2, Hk=1, D=64, rot_dim=64, inv_freq=ctypes.addressof(f), attn_factor=1.0, q=0x1000, q_stride=128,
                q_out=0x2000, q_out_stride=128, k=0x3000, k_stride=64, k_out=0x4000, k_out_stride=64)
    call = lambda **kw: L.ls_rope(ctypes.byref(b.RopeDesc(**{**base, **kw})), None)  # noqa: E731
    assert L.ls_rope(None, None) == 1
    for kw in (dict(T=0), dict(Hq=0, Hk=0), dict(Hq=-1), dict(inv_freq=None), dict(q=None), dict(k_out=None), dict(q_stride=127),
               dict(k_out_stride=63), dict(rot_dim=0), dict(rot_dim=66), dict(rot_dim=31), dict(attn_factor=float("nan")),
               dict(q_out=0x1000, q_out_stride=256)):
        assert call(**kw) == 1, kw
    assert call(D=258, rot_dim=64, q_stride=600, q_out_stride=600, k_stride=300, k_out_stride=300) == 2
    assert call(D=63) == 2 and call(T=1 << 31) == 2
    assert call(q=0x1001) == 4 and call(positions=0x1004) == 4
    f[3] = float("inf")
    assert call() == 1
    k = ctypes.c_double()
    fr = lambda *a: L.ls_rope_freqs(*a, ctypes.addressof(f), ctypes.addressof(k))  # noqa: E731
    assert fr(64, 1.0, 0, 1.0, 0, 32.0, 1.0) == 1 and fr(63, 1e4, 0, 1.0, 0, 32.0, 1.0) == 1
    assert fr(64, 1e4, 3, 1.0, 0, 32.0, 1.0) == 1 and fr(64, 1e4, 1, 0.5, 0, 32.0, 1.0) == 1
    assert fr(64, 1e4, 2, 2.0, 0, 32.0, 1.0) == 1 and fr(64, 1e4, 2, 2.0, 10, 1.0, 2.0) == 1
    assert fr(258, 1e4, 0, 1.0, 0, 32.0, 1.0) == 1
