"""Host side of the group operators: descriptor layouts as the binding packs them, refusals of the
policy loss, binding checks that need no GPU."""
import ctypes

import pytest

from long_context_grpo_gb300 import build as lsbuild


@pytest.fixture(scope="module")
def b():
    lsbuild.build()
    from long_context_grpo_gb300 import _lib
    _lib._lib()
    return _lib


@pytest.mark.parametrize("packed,desc", [("_POLICY", "PolicyLossDesc"), ("_ROPE", "RopeDesc"), ("_APPEND", "CacheAppendDesc"),
                                         ("_ATTN", "CacheAttnDesc")])
def test_packed_descriptors_have_the_structures_layout(b, packed, desc):
    from long_context_grpo_gb300 import _ops
    s, D = getattr(_ops, packed), getattr(b, desc)
    kinds = [k for _, k in D._fields_]
    values = [float(i + 1) if k is ctypes.c_double else i + 1 for i, k in enumerate(kinds)]
    raw = s.pack(*values)
    assert len(raw) <= ctypes.sizeof(D)
    got = D.from_buffer_copy(raw.ljust(ctypes.sizeof(D), b"\0"))
    assert [getattr(got, n) for n, _ in D._fields_] == values


def test_structures_match_the_header(b, tmp_path):
    """sizeof and the last field's offset of every descriptor, from the header itself."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    last = {"ls_policy_loss_desc": ("kl_out", "PolicyLossDesc"), "ls_rope_desc": ("k_out_stride", "RopeDesc"),
            "ls_cache_desc": ("refcount", "CacheDesc"), "ls_cache_append_desc": ("attn_factor", "CacheAppendDesc"),
            "ls_cache_attn_desc": ("shared_len", "CacheAttnDesc")}
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "%s/include/longstraw.h"\nint main(void){\n' % root
    for c, (f, _) in last.items():
        src += 'printf("%%zu %%zu\\n", sizeof(%s), offsetof(%s, %s));\n' % (c, c, f)
    (tmp_path / "t.c").write_text(src + "return 0;}\n")
    subprocess.run(["gcc", "-std=c99", str(tmp_path / "t.c"), "-o", str(tmp_path / "t")], check=True)
    out = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout.split()
    for i, (f, py) in enumerate(last.values()):
        D = getattr(b, py)
        assert (ctypes.sizeof(D), getattr(D, f).offset) == (int(out[2 * i]), int(out[2 * i + 1])), py


def test_policy_loss_refusals(b):
    L = b._lib()
    ws = L.ls_policy_loss_workspace_bytes(100)
    assert ws >= 800 and ws % 256 == 0 and L.ls_policy_loss_workspace_bytes(0) == 0
    base = dict(T=100, V=64, logits_stride=64, dlogits_stride=64, logits=0x1000, ids=0x2000, logp_old=0x3000, logp_ref=0x4000,
                advantages=0x5000, weights=0x6000, eps_low=0.2, eps_high=0.2, beta=0.1, kl=3, loss=0x7000, dlogits=0x8000,
                clip_mask=0x9001, logp_out=0xa000, kl_out=0xb000)
    call = lambda wsp=0xc000, n=ws, **kw: L.ls_policy_loss(ctypes.byref(b.PolicyLossDesc(**{**base, **kw})), wsp, n, None)  # noqa: E731
    assert L.ls_policy_loss(None, 0xc000, ws, None) == 1
    nan, inf = float("nan"), float("inf")
    for kw in (dict(logits=None), dict(ids=None), dict(logp_old=None), dict(advantages=None), dict(weights=None), dict(loss=None),
               dict(dlogits=None), dict(clip_mask=None), dict(T=0), dict(V=0), dict(T=-1), dict(logits_stride=63),
               dict(dlogits_stride=63), dict(eps_low=1.0), dict(eps_low=-0.1), dict(eps_low=nan), dict(eps_high=-0.1),
               dict(eps_high=inf), dict(beta=nan), dict(beta=inf), dict(kl=4), dict(kl=-1), dict(logp_ref=None),
               dict(dlogits=0x1000, dlogits_stride=72)):
        assert call(**kw) == 1, kw
    for kw in (dict(T=1 << 31), dict(V=1 << 31, logits_stride=1 << 31, dlogits_stride=1 << 31), dict(logits_stride=1 << 31)):
        assert call(**kw) == 2, kw
    assert call(wsp=None) == 8 and call(n=ws - 1) == 8
    for kw in (dict(logits=0x1001), dict(ids=0x2002), dict(loss=0x7002), dict(logp_out=0xa001), dict(wsp=0xc008)):
        assert call(**kw) == 4, kw


def test_binding_refuses_before_the_library(b):
    import torch

    import long_context_grpo_gb300 as ls
    x = torch.zeros(2, 8)
    with pytest.raises(TypeError):
        ls.rope(x, None, [0.1])
    with pytest.raises(TypeError):
        ls.policy_loss(None, None, None, None, None)
    with pytest.raises(ValueError):
        ls.policy_loss(x, None, None, None, None, kl="k4")
    with pytest.raises(ValueError):
        ls.rope_freqs(64, scaling="cubic")
    with pytest.raises(ls.LongStrawError):
        ls.rope_freqs(63)
    with pytest.raises(ValueError):
        ls.PagedCache(x, x, x, x, x, Hq=1, layout="DHN")
