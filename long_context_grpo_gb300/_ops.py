"""Binding of the operators around the replay: the policy loss with a KL term, rotary
positions and the paged cache.  Argument marshalling only, as in _lib.py: every tensor is
checked (device, dtype, shape, strides) and passed as a raw pointer with torch's current
stream; outputs and workspaces that are not given are allocated on it.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib as b

_KL = {"none": 0, "k1": 1, "k2": 2, "k3": 3}
_SCALING = {"none": 0, "linear": 1, "ramp": 2}
_LAYOUT = {"NHD": 0, "HND": 1}


def _ptr(t, name, dtype, shape=None):
    """As _lib._ptr, and on the current device (whose stream the call goes to)."""
    p = b._ptr(t, name, dtype, shape)
    if t is not None and t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d"
                         % (name, t.device, torch.cuda.current_device()))
    return p


def _strided(t, name, shape, strides, width):
    """(pointer, elements between rows) of a bf16 tensor of this shape whose dimensions behind
    the first have these strides; the rows hold `width` values each."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != torch.bfloat16:
        raise TypeError("%s must be %s, got %s" % (name, torch.bfloat16, t.dtype))
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    st = t.stride()
    for n, have, want in zip(shape[1:], st[1:], strides):
        if n > 1 and have != want:
            raise ValueError("%s must be contiguous behind its first dimension" % name)
    if t.device.index != torch.cuda.current_device():
        raise ValueError("%s is on %s, the current device is cuda:%d"
                         % (name, t.device, torch.cuda.current_device()))
    # one row: whatever stride torch keeps for it
    return t.data_ptr(), (st[0] if shape[0] > 1 else max(width, (width + 7) // 8 * 8))


def _heads(t, name, T, H, D):
    return _strided(t, name, (T, H, D), (D, 1), H * D)


def _host_doubles(x, name):
    """(pointer, count, keep-alive) of float64 values on the host."""
    if isinstance(x, torch.Tensor):
        if x.is_cuda or x.dtype != torch.float64 or x.dim() != 1 or not x.is_contiguous():
            raise TypeError("%s must be a contiguous 1-D float64 tensor on the CPU" % name)
        return x.data_ptr(), x.numel(), x
    v = [float(e) for e in x]
    a = (ctypes.c_double * len(v))(*v)
    return ctypes.addressof(a), len(v), a


class PolicyLoss(NamedTuple):
    loss: torch.Tensor        # fp32 [1]
    dlogits: torch.Tensor     # bf16 [T, V]
    logp: torch.Tensor        # fp32 [T]
    kl: torch.Tensor          # fp32 [T]
    clip_mask: torch.Tensor   # uint8 [T]


def policy_loss_workspace_bytes(T: int) -> int:
    return int(b._lib().ls_policy_loss_workspace_bytes(T))


def policy_loss(logits, ids, logp_old, advantages, weights, eps_low=0.2, eps_high=0.2,
                logp_ref=None, beta=0.0, kl="none", loss=None, dlogits=None, logp_out=None,
                kl_out=None, clip_mask=None, workspace=None) -> PolicyLoss:
    """Clipped policy loss over packed tokens with per-token advantages and weights and a KL
    term to a reference policy (kl = "none", "k1", "k2" or "k3", weighted by beta), with its
    gradient:  loss = sum_t w_t (beta kl_t - min(rho A, clip(rho, 1-eps_low, 1+eps_high) A)).
    logits: bf16 [T, V], rows may be strided; dlogits may be the logits themselves.  A token
    of weight 0 is left out (its inputs are not looked at)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise TypeError("logits must be a 2-D CUDA tensor")
    if kl not in _KL:
        raise ValueError("kl must be one of %s" % (tuple(_KL),))
    T, V = logits.shape
    x, ldx = _strided(logits, "logits", (T, V), (1,), V)
    dev = logits.device
    if dlogits is None:
        dlogits = torch.empty((T, V), dtype=torch.bfloat16, device=dev)
    dx, ldd = _strided(dlogits, "dlogits", (T, V), (1,), V)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    logp_out = torch.empty(T, dtype=torch.float32, device=dev) if logp_out is None else logp_out
    kl_out = torch.empty(T, dtype=torch.float32, device=dev) if kl_out is None else kl_out
    clip_mask = torch.empty(T, dtype=torch.uint8, device=dev) if clip_mask is None else clip_mask
    if workspace is None:
        workspace = torch.empty(max(policy_loss_workspace_bytes(T), 16), dtype=torch.uint8, device=dev)
    f32 = torch.float32
    d = b.PolicyLossDesc(
        T, V, ldx, ldd, x, _ptr(ids, "ids", torch.int32, (T,)), _ptr(logp_old, "logp_old", f32, (T,)),
        _ptr(logp_ref, "logp_ref", f32, (T,)), _ptr(advantages, "advantages", f32, (T,)),
        _ptr(weights, "weights", f32, (T,)), float(eps_low), float(eps_high), float(beta), _KL[kl],
        _ptr(loss, "loss", f32, (1,)), dx, _ptr(clip_mask, "clip_mask", torch.uint8, (T,)),
        _ptr(logp_out, "logp_out", f32, (T,)), _ptr(kl_out, "kl_out", f32, (T,)))
    b._check(b._lib().ls_policy_loss(ctypes.byref(d), _ptr(workspace, "workspace", torch.uint8),
                                     workspace.numel(), b._stream()), "ls_policy_loss")
    return PolicyLoss(loss, dlogits, logp_out, kl_out, clip_mask)


def rope_freqs(rot_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               orig_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inverse frequencies as a float64 CPU tensor [rot_dim / 2], attention factor) for rope()
    and PagedCache.append(); scaling "linear" or "ramp" for contexts `factor` times orig_len."""
    if scaling not in _SCALING:
        raise ValueError("scaling must be one of %s" % (tuple(_SCALING),))
    f = torch.empty(max(rot_dim // 2, 1), dtype=torch.float64)
    k = ctypes.c_double()
    b._check(b._lib().ls_rope_freqs(rot_dim, float(theta), _SCALING[scaling], float(factor), orig_len,
                                    float(beta_fast), float(beta_slow), f.data_ptr(),
                                    ctypes.addressof(k)), "ls_rope_freqs")
    return f, k.value


def rope(q, k, inv_freq, positions=None, pos0: int = 0, interleaved: bool = False,
         attn_factor: float = 1.0, inverse: bool = False, q_out=None, k_out=None):
    """Rotary positions of q [T, Hq, D] and k [T, Hk, D] (bf16; either may be None; rows may be
    strided views): the first 2 len(inv_freq) values of every head are turned by position *
    inv_freq, token t at positions[t] (int64) or pos0 + t.  inverse=True is the gradient:
    give it d loss / d output.  q_out / k_out may be the inputs.  Returns (q_out, k_out)."""
    some = q if q is not None else k
    if not isinstance(some, torch.Tensor) or some.dim() != 3:
        raise TypeError("q or k must be a 3-D CUDA tensor")
    T, _, D = some.shape
    f, n, keep = _host_doubles(inv_freq, "inv_freq")
    d = b.RopeDesc(T=T, D=D, rot_dim=2 * n, interleaved=int(interleaved), inverse=int(inverse),
                   inv_freq=f, attn_factor=float(attn_factor), pos0=pos0,
                   positions=_ptr(positions, "positions", torch.int64, (T,)))
    if q is not None:
        d.Hq = q.shape[1]
        d.q, d.q_stride = _heads(q, "q", T, d.Hq, D)
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
        d.q_out, d.q_out_stride = _heads(q_out, "q_out", T, d.Hq, D)
    if k is not None:
        d.Hk = k.shape[1]
        d.k, d.k_stride = _heads(k, "k", T, d.Hk, D)
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device) if k_out is None else k_out
        d.k_out, d.k_out_stride = _heads(k_out, "k_out", T, d.Hk, D)
    b._check(b._lib().ls_rope(ctypes.byref(d), b._stream()), "ls_rope")
    return q_out, k_out


class PagedCache:
    """Keys and values of one attention layer in pages that sequences may share.

    k_pages, v_pages: bf16 [pages, page_size, Hkv, D] ("NHD") or [pages, Hkv, page_size, D]
    ("HND"), contiguous behind the first dimension (both may be views of one pool).
    page_table int32 [rows, width], seq_len int32 [rows], refcount int32 [pages].  All are
    borrowed and must outlive the handle; reset() makes every row empty.  Calls are ordered
    on one stream.  See include/longstraw.h for each call's contract.
    """

    def __init__(self, k_pages, v_pages, page_table, seq_len, refcount, Hq: int, layout: str = "NHD",
                 softmax_scale: float = 0.0):
        if layout not in _LAYOUT:
            raise ValueError("layout must be one of %s" % (tuple(_LAYOUT),))
        if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
            raise TypeError("k_pages must be a 4-D CUDA tensor")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise TypeError("page_table must be a 2-D CUDA tensor")
        shape = tuple(k_pages.shape)
        N, D = shape[0], shape[3]
        ps, Hkv = (shape[1], shape[2]) if layout == "NHD" else (shape[2], shape[1])
        inner = (shape[2] * D, D, 1)
        kp, stride = _strided(k_pages, "k_pages", shape, inner, ps * Hkv * D)
        vp, vstride = _strided(v_pages, "v_pages", shape, inner, ps * Hkv * D)
        if stride != vstride:
            raise ValueError("k_pages and v_pages must have the same page stride")
        rows, width = page_table.shape
        self.num_pages, self.page_size, self.Hq, self.Hkv, self.D = N, ps, Hq, Hkv, D
        self.k_pages, self.v_pages = k_pages, v_pages
        self.page_table, self.seq_len, self.refcount = page_table, seq_len, refcount
        i32 = torch.int32
        d = b.CacheDesc(N, ps, Hq, Hkv, D, _LAYOUT[layout], softmax_scale, stride, kp, vp, rows, width,
                        _ptr(page_table, "page_table", i32, (rows, width)),
                        _ptr(seq_len, "seq_len", i32, (rows,)), _ptr(refcount, "refcount", i32, (N,)))
        h = ctypes.c_void_p()
        b._check(b._lib().ls_cache_create(ctypes.byref(d), ctypes.byref(h)), "ls_cache_create")
        self._h = h

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value is not None:
            b._check(b._lib().ls_cache_destroy(self._h), "ls_cache_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _list(self, t, name, n=None):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            raise TypeError("%s must be a 1-D CUDA tensor" % name)
        return _ptr(t, name, torch.int32, None if n is None else (n,))

    def _pages_ws(self, workspace):
        if workspace is None:
            workspace = torch.empty(self.pages_workspace_bytes(), dtype=torch.uint8,
                                    device=self.refcount.device)
        return workspace

    def pages_workspace_bytes(self) -> int:
        return int(b._lib().ls_cache_pages_workspace_bytes(self._h))

    def reset(self):
        """Every row empty, every page free."""
        b._check(b._lib().ls_cache_reset(self._h, b._stream()), "ls_cache_reset")

    def extend(self, rows, add, workspace=None):
        """Lengths of `rows` grow by `add` (int32), with free pages for the new tokens."""
        ws = self._pages_ws(workspace)
        b._check(b._lib().ls_cache_extend(
            self._h, rows.numel(), self._list(rows, "rows"), self._list(add, "add", rows.numel()),
            _ptr(ws, "workspace", torch.uint8), ws.numel(), b._stream()), "ls_cache_extend")

    def fork(self, parents, children, workspace=None):
        """Empty rows `children` become copies of rows `parents`: whole pages are shared, a
        part-filled last page is copied."""
        ws = self._pages_ws(workspace)
        b._check(b._lib().ls_cache_fork(
            self._h, parents.numel(), self._list(parents, "parents"),
            self._list(children, "children", parents.numel()), _ptr(ws, "workspace", torch.uint8),
            ws.numel(), b._stream()), "ls_cache_fork")

    def free(self, rows):
        """Empties `rows`; pages that no row lists any more become free."""
        b._check(b._lib().ls_cache_free(self._h, rows.numel(), self._list(rows, "rows"), b._stream()),
                 "ls_cache_free")

    def compact(self, into=None, n_live=None, workspace=None):
        """Moves the live pages together: in place, or into another PagedCache's pool."""
        ws = self._pages_ws(workspace)
        dst = self if into is None else into
        b._check(b._lib().ls_cache_compact(
            self._h, dst._h, _ptr(n_live, "n_live", torch.int32, (1,)),
            _ptr(ws, "workspace", torch.uint8), ws.numel(), b._stream()), "ls_cache_compact")

    def append(self, k_new, v_new, cu_new, rows=None, q=None, q_out=None, inv_freq=None,
               interleaved: bool = False, attn_factor: float = 1.0):
        """Writes the last new tokens of each sequence (packed by cu_new, int32 [S + 1]; lengths
        already extended) into their pages, rotated with inv_freq on the way, and rotates q
        [T, Hq, D] in the same pass.  Returns (q_out, None) or, without q, (None, None)."""
        if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3:
            raise TypeError("k_new must be a 3-D CUDA tensor")
        T = k_new.shape[0]
        S = cu_new.numel() - 1
        d = b.CacheAppendDesc(S=S, T=T, cu_new=self._list(cu_new, "cu_new"),
                              rows=None if rows is None else self._list(rows, "rows", S),
                              interleaved=int(interleaved), attn_factor=float(attn_factor))
        d.k_new, d.k_stride = _heads(k_new, "k_new", T, self.Hkv, self.D)
        d.v_new, d.v_stride = _heads(v_new, "v_new", T, self.Hkv, self.D)
        keep = None
        if inv_freq is not None:
            d.inv_freq, n, keep = _host_doubles(inv_freq, "inv_freq")
            d.rot_dim = 2 * n
        if q is not None:
            d.q, d.q_stride = _heads(q, "q", T, self.Hq, self.D)
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else q_out
            d.q_out, d.q_out_stride = _heads(q_out, "q_out", T, self.Hq, self.D)
        b._check(b._lib().ls_cache_append(self._h, ctypes.byref(d), b._stream()), "ls_cache_append")
        del keep
        return (q_out if q is not None else None), None

    def attn_workspace_bytes(self, S: int, T: int, max_new: int, max_len: int) -> int:
        return int(b._lib().ls_cache_attn_workspace_bytes(self._h, S, T, max_new, max_len))

    def attn(self, q, cu_new, max_new: int, max_len: int, rows=None, group: int = 1,
             shared_len=None, o=None, lse=None, workspace=None):
        """Attention of the new tokens q [T, Hq, D] over their sequences' pages, causal within
        the sequence (append first).  group > 1: runs of `group` entries share their first
        shared_len[i] tokens' pages, which are read once.  Returns (o, lse)."""
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise TypeError("q must be a 3-D CUDA tensor")
        T = q.shape[0]
        S = cu_new.numel() - 1
        if o is None:
            o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if lse is None:
            lse = torch.empty((T, self.Hq), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = torch.empty(max(self.attn_workspace_bytes(S, T, max_new, max_len), 16),
                                    dtype=torch.uint8, device=q.device)
        qp, qs = _heads(q, "q", T, self.Hq, self.D)
        d = b.CacheAttnDesc(
            S, T, None if rows is None else self._list(rows, "rows", S), self._list(cu_new, "cu_new"),
            max_new, max_len, qp, qs, _ptr(o, "o", torch.bfloat16, (T, self.Hq, self.D)),
            _ptr(lse, "lse", torch.float32, (T, self.Hq)), group,
            None if shared_len is None else self._list(shared_len, "shared_len", S // max(group, 1)))
        b._check(b._lib().ls_cache_attn(self._h, ctypes.byref(d), _ptr(workspace, "workspace", torch.uint8),
                                        workspace.numel(), b._stream()), "ls_cache_attn")
        return o, lse
