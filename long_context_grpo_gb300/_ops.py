"""Binding of the operators around the replay: the policy loss with a KL term, rotary
positions and the paged cache.  Argument marshalling only, as in _lib.py: every tensor is
checked (device, dtype, shape, strides) and passed as a raw pointer with torch's current
stream; outputs and workspaces that are not given are allocated on it.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import torch

from . import _lib as b

_KL = {"none": 0, "k1": 1, "k2": 2, "k3": 3}
_SCALING = {"none": 0, "linear": 1, "ramp": 2}
_LAYOUT = {"NHD": 0, "HND": 1}


# The descriptors of include/longstraw.h as native struct layouts: packing one is several times
# cheaper than filling a ctypes.Structure, and small calls are bound by the host.
_POLICY = struct.Struct("@qqqqPPPPPPdddiPPPPP")
_ROPE = struct.Struct("@qiiiiiiPdPqPqPqPqPq")
_APPEND = struct.Struct("@iqPPPqPqPqPqPiid")
_ATTN = struct.Struct("@iqPPiqPqPPiP")

_Tensor = torch.Tensor
_bf16, _f32, _i32, _i64, _u8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _ptr(t, name, dtype, shape, dev):
    """Address of a contiguous tensor of this type and shape (None: any) on device `dev`, the
    current one, whose stream the call goes to."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    b._ptr(t, name, dtype, shape)          # says what is wrong with it
    if t is None:
        raise TypeError("%s must be a CUDA tensor" % name)
    raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, dev))


def _opt(t, name, dtype, shape, dev):
    return 0 if t is None else _ptr(t, name, dtype, shape, dev)


def _strided(t, name, shape, strides, width, dev):
    """(pointer, elements between rows) of a bf16 tensor of this shape whose dimensions behind
    the first have these strides; the rows hold `width` values each."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype is not _bf16:
        raise TypeError("%s must be %s, got %s" % (name, _bf16, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    st = t.stride()
    if st[1:] != strides:
        for n, have, want in zip(shape[1:], st[1:], strides):
            if n > 1 and have != want:
                raise ValueError("%s must be contiguous behind its first dimension" % name)
    if t.get_device() != dev:
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, dev))
    # one row: whatever stride torch keeps for it
    return t.data_ptr(), (st[0] if shape[0] > 1 else (width + 7) // 8 * 8)


def _heads(t, name, T, H, D, dev):
    return _strided(t, name, (T, H, D), (D, 1), H * D, dev)


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _host_doubles(x, name):
    """(pointer, count, keep-alive) of float64 values on the host."""
    if isinstance(x, _Tensor):
        if x.is_cuda or x.dtype is not torch.float64 or x.dim() != 1 or not x.is_contiguous():
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
    dev = torch.cuda.current_device()
    at = logits.device
    x, ldx = _strided(logits, "logits", (T, V), (1,), V, dev)
    if dlogits is None:
        dlogits = torch.empty((T, V), dtype=_bf16, device=at)
        dx, ldd = dlogits.data_ptr(), V
    else:
        dx, ldd = _strided(dlogits, "dlogits", (T, V), (1,), V, dev)
    n = (T,)
    if clip_mask is None:
        clip_mask = torch.empty(n, dtype=_u8, device=at)
        cm = clip_mask.data_ptr()
    else:
        cm = _ptr(clip_mask, "clip_mask", _u8, n, dev)
    nbytes = b._lib().ls_policy_loss_workspace_bytes(T)
    # (one allocation an output: views of a fresh tensor cost the host more than its allocation)
    if loss is None:
        loss = torch.empty(1, dtype=_f32, device=at)
        sp = loss.data_ptr()
    else:
        sp = _ptr(loss, "loss", _f32, (1,), dev)
    if logp_out is None:
        logp_out = torch.empty(n, dtype=_f32, device=at)
        lp = logp_out.data_ptr()
    else:
        lp = _ptr(logp_out, "logp_out", _f32, n, dev)
    if kl_out is None:
        kl_out = torch.empty(n, dtype=_f32, device=at)
        kp = kl_out.data_ptr()
    else:
        kp = _ptr(kl_out, "kl_out", _f32, n, dev)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=_u8, device=at)
        wp = workspace.data_ptr()
    else:
        wp, nbytes = _ptr(workspace, "workspace", _u8, None, dev), workspace.numel()
    d = _POLICY.pack(
        T, V, ldx, ldd, x, _ptr(ids, "ids", _i32, n, dev), _ptr(logp_old, "logp_old", _f32, n, dev),
        _opt(logp_ref, "logp_ref", _f32, n, dev), _ptr(advantages, "advantages", _f32, n, dev),
        _ptr(weights, "weights", _f32, n, dev), eps_low, eps_high, beta, _KL[kl], sp, dx, cm, lp, kp)
    b._check(b._lib().ls_policy_loss(d, wp, nbytes, _raw_stream(dev)), "ls_policy_loss")
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
    for t in (some, k):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dim() != 3):
            raise TypeError("q and k must be 3-D CUDA tensors")
    if some is None:
        raise TypeError("q or k must be a 3-D CUDA tensor")
    T, _, D = some.shape
    dev = torch.cuda.current_device()
    f, n, keep = _host_doubles(inv_freq, "inv_freq")
    Hq = Hk = qp = qs = qo = qos = kp = ks = ko = kos = 0
    if q is not None:
        Hq = q.shape[1]
        qp, qs = _heads(q, "q", T, Hq, D, dev)
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=_bf16, device=q.device)
            qo, qos = q_out.data_ptr(), Hq * D
        else:
            qo, qos = _heads(q_out, "q_out", T, Hq, D, dev)
    if k is not None:
        Hk = k.shape[1]
        kp, ks = _heads(k, "k", T, Hk, D, dev)
        if k_out is None:
            k_out = torch.empty((T, Hk, D), dtype=_bf16, device=k.device)
            ko, kos = k_out.data_ptr(), Hk * D
        else:
            ko, kos = _heads(k_out, "k_out", T, Hk, D, dev)
    d = _ROPE.pack(T, Hq, Hk, D, 2 * n, bool(interleaved), bool(inverse), f, attn_factor,
                   _opt(positions, "positions", _i64, (T,), dev), pos0, qp, qs, qo, qos, kp, ks, ko, kos)
    b._check(b._lib().ls_rope(d, _raw_stream(dev)), "ls_rope")
    return q_out, k_out


class PagedCache:
    """Keys and values of one attention layer in pages that sequences may share.

    k_pages, v_pages: bf16 [pages, page_size, Hkv, D] ("NHD") or [pages, Hkv, page_size, D]
    ("HND"), contiguous behind the first dimension (both may be views of one pool).
    page_table int32 [rows, width], seq_len int32 [rows], refcount int32 [pages].  All are
    borrowed and must outlive the handle; reset() makes every row empty.  Every layer of a model
    has a handle and table, lengths and counts of its own.  Calls are ordered on one stream.  See
    include/longstraw.h for each call's contract.
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
        dev = torch.cuda.current_device()
        kp, stride = _strided(k_pages, "k_pages", shape, inner, ps * Hkv * D, dev)
        vp, vstride = _strided(v_pages, "v_pages", shape, inner, ps * Hkv * D, dev)
        if stride != vstride:
            raise ValueError("k_pages and v_pages must have the same page stride")
        rows, width = page_table.shape
        self.num_pages, self.page_size, self.Hq, self.Hkv, self.D = N, ps, Hq, Hkv, D
        self.k_pages, self.v_pages = k_pages, v_pages
        self.page_table, self.seq_len, self.refcount = page_table, seq_len, refcount
        d = b.CacheDesc(N, ps, Hq, Hkv, D, _LAYOUT[layout], softmax_scale, stride, kp, vp, rows, width,
                        _ptr(page_table, "page_table", _i32, (rows, width), dev),
                        _ptr(seq_len, "seq_len", _i32, (rows,), dev),
                        _ptr(refcount, "refcount", _i32, (N,), dev))
        h = ctypes.c_void_p()
        b._check(b._lib().ls_cache_create(ctypes.byref(d), ctypes.byref(h)), "ls_cache_create")
        self._h = h
        self._pages_bytes = int(b._lib().ls_cache_pages_workspace_bytes(h))

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value is not None:
            b._check(b._lib().ls_cache_destroy(self._h), "ls_cache_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _list(t, name, dev, n=None):
        if not isinstance(t, _Tensor) or t.dim() != 1:
            raise TypeError("%s must be a 1-D CUDA tensor" % name)
        return _ptr(t, name, _i32, None if n is None else (n,), dev)

    def _pages_ws(self, workspace, dev):
        if workspace is None:
            workspace = torch.empty(self._pages_bytes, dtype=_u8, device=self.refcount.device)
        return workspace, _ptr(workspace, "workspace", _u8, None, dev)

    def pages_workspace_bytes(self) -> int:
        return self._pages_bytes

    def reset(self):
        """Every row empty, every page free."""
        b._check(b._lib().ls_cache_reset(self._h, b._stream()), "ls_cache_reset")

    def extend(self, rows, add, workspace=None):
        """Lengths of `rows` grow by `add` (int32), with free pages for the new tokens."""
        dev = torch.cuda.current_device()
        ws, wp = self._pages_ws(workspace, dev)
        rp, n = self._list(rows, "rows", dev), rows.numel()
        b._check(b._lib().ls_cache_extend(self._h, n, rp, self._list(add, "add", dev, n), wp, ws.numel(),
                                          _raw_stream(dev)), "ls_cache_extend")

    def fork(self, parents, children, workspace=None):
        """Empty rows `children` become copies of rows `parents`: whole pages are shared, a
        part-filled last page is copied."""
        dev = torch.cuda.current_device()
        ws, wp = self._pages_ws(workspace, dev)
        pp, n = self._list(parents, "parents", dev), parents.numel()
        b._check(b._lib().ls_cache_fork(self._h, n, pp, self._list(children, "children", dev, n), wp, ws.numel(),
                                        _raw_stream(dev)), "ls_cache_fork")

    def free(self, rows):
        """Empties `rows`; pages that no row lists any more become free."""
        dev = torch.cuda.current_device()
        rp = self._list(rows, "rows", dev)
        b._check(b._lib().ls_cache_free(self._h, rows.numel(), rp, _raw_stream(dev)), "ls_cache_free")

    def compact(self, into=None, n_live=None, workspace=None):
        """Moves the live pages together: in place, or into another PagedCache's pool."""
        dev = torch.cuda.current_device()
        ws, wp = self._pages_ws(workspace, dev)
        dst = self if into is None else into
        b._check(b._lib().ls_cache_compact(self._h, dst._h, _opt(n_live, "n_live", _i32, (1,), dev), wp, ws.numel(),
                                           _raw_stream(dev)), "ls_cache_compact")

    def append(self, k_new, v_new, cu_new, rows=None, q=None, q_out=None, inv_freq=None,
               interleaved: bool = False, attn_factor: float = 1.0):
        """Writes the last new tokens of each sequence (packed by cu_new, int32 [S + 1]; lengths
        already extended) into their pages, rotated with inv_freq on the way, and rotates q
        [T, Hq, D] in the same pass.  Returns (q_out, None) or, without q, (None, None)."""
        if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3:
            raise TypeError("k_new must be a 3-D CUDA tensor")
        T = k_new.shape[0]
        dev = torch.cuda.current_device()
        cp, S = self._list(cu_new, "cu_new", dev), cu_new.numel() - 1
        kp, ks = _heads(k_new, "k_new", T, self.Hkv, self.D, dev)
        vp, vs = _heads(v_new, "v_new", T, self.Hkv, self.D, dev)
        f = n = qp = qs = qo = qos = 0
        keep = None
        if inv_freq is not None:
            f, n, keep = _host_doubles(inv_freq, "inv_freq")
        if q is not None:
            qp, qs = _heads(q, "q", T, self.Hq, self.D, dev)
            if q_out is None:
                q_out = torch.empty((T, self.Hq, self.D), dtype=_bf16, device=q.device)
                qo, qos = q_out.data_ptr(), self.Hq * self.D
            else:
                qo, qos = _heads(q_out, "q_out", T, self.Hq, self.D, dev)
        d = _APPEND.pack(S, T, 0 if rows is None else self._list(rows, "rows", dev, S), cp,
                         kp, ks, vp, vs, qp, qs, qo, qos, f, 2 * n, bool(interleaved), attn_factor)
        b._check(b._lib().ls_cache_append(self._h, d, _raw_stream(dev)), "ls_cache_append")
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
        dev = torch.cuda.current_device()
        cp, S = self._list(cu_new, "cu_new", dev), cu_new.numel() - 1
        at = q.device
        if o is None:
            o = torch.empty((T, self.Hq, self.D), dtype=_bf16, device=at)
            op = o.data_ptr()
        else:
            op = _ptr(o, "o", _bf16, (T, self.Hq, self.D), dev)
        if lse is None:
            lse = torch.empty((T, self.Hq), dtype=_f32, device=at)
            lp = lse.data_ptr()
        else:
            lp = _ptr(lse, "lse", _f32, (T, self.Hq), dev)
        if workspace is None:
            workspace = torch.empty(max(self.attn_workspace_bytes(S, T, max_new, max_len), 16), dtype=_u8,
                                    device=at)
        qp, qs = _heads(q, "q", T, self.Hq, self.D, dev)
        d = _ATTN.pack(S, T, 0 if rows is None else self._list(rows, "rows", dev, S), cp,
                       max_new, max_len, qp, qs, op, lp, group,
                       0 if shared_len is None else self._list(shared_len, "shared_len", dev, S // max(group, 1)))
        b._check(b._lib().ls_cache_attn(self._h, d, _ptr(workspace, "workspace", _u8, None, dev), workspace.numel(),
                                        _raw_stream(dev)), "ls_cache_attn")
        return o, lse
