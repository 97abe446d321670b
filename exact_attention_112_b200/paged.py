"""Rotary positions and the paged key/value cache: argument marshalling of
``fa_rope``, ``fa_rope_bwd``, ``fa_paged_append`` and ``fa_paged_fwd`` (see
``include/fa.h``).

    rope = fa.Rope(*fa.rope_inv_freq(128, base=500000.0))
    q, k = fa.rope_forward(q, k, rope)                       # training, before attention_forward
    dq, dk = fa.rope_backward(dq, dk, rope)                  # after attention_backward

    kv = fa.PagedKV(k_cache, v_cache, page_table, seq_lens)  # serving: one handle per cache and batch
    o, lse = fa.paged_step(kv, q, k, v, cu_seqlens_q, max_seqlen_q, rope)

``Rope`` and ``PagedKV`` check their tensors once, when they are made, and keep
them alive; the tables' values may change between calls, their storage may not.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import struct

from . import FA_ERR_UNSUPPORTED, FA_OK, FaError, _bad, _check, _dtype_code, lib

__all__ = ["Rope", "PagedKV", "rope_inv_freq", "fa_rope", "fa_rope_bwd", "rope_forward", "rope_backward",
           "fa_paged_append", "fa_paged_fwd", "fa_paged_fwd_workspace_bytes", "paged_attention", "paged_step",
           "rope_attention_forward", "rope_attention_backward"]

_LL3 = ctypes.c_longlong * 3
# host arrays of strides, as the bytes that the C side reads during the call (of
# four strides the first three)
_strides2 = struct.Struct("2q").pack
_strides3 = struct.Struct("3q").pack
_strides4 = struct.Struct("4q").pack


class _RopeSpec(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("scale", ctypes.c_float)]


class _PagedSpec(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("k_strides", _LL3), ("v_strides", _LL3), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_longlong), ("seq_lens", ctypes.c_void_p),
                ("num_seqs", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("num_kv_heads", ctypes.c_int), ("page_size", ctypes.c_int), ("D", ctypes.c_int),
                ("dtype", ctypes.c_int)]


def _declare(L):
    """Argument types of the C entry points (called once, by lib())."""
    vp, i, ll, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    rope_args = [vp, vp, vp, vp, i, vp, vp, vp, vp, i, i, i, i, vp, vp, ll, i, i, vp]
    for f in (L.fa_rope, L.fa_rope_bwd):
        f.argtypes = rope_args
        f.restype = i
    L.fa_paged_append.argtypes = [vp, vp, vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, i, vp]
    L.fa_paged_append.restype = i
    L.fa_paged_fwd_workspace_bytes.argtypes = [vp, i, i]
    L.fa_paged_fwd_workspace_bytes.restype = sz
    L.fa_paged_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, ctypes.c_float, vp, sz, vp]
    L.fa_paged_fwd.restype = i


def rope_inv_freq(rot_dim, base=10000.0, scaling=None, factor=1.0, original_max_position=8192,
                  low_freq_factor=1.0, high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """(frequencies, attention factor) of a rotary embedding: float64
    [rot_dim/2] radians per position, base ** (-2i / rot_dim), scaled for
    contexts ``factor`` times ``original_max_position`` by

      None     not at all
      "linear" every frequency divided by the factor
      "ntk"    the base raised, so that the lowest frequency is divided by it
      "bands"  frequencies that turn more than high_freq_factor times within
               the original context kept, those that turn less than
               low_freq_factor times divided, a linear blend in between
      "yarn"   the same blend over the index of the frequency, between those
               that turn beta_fast and beta_slow times, and the attention factor
               0.1 ln(factor) + 1 on cosine and sine
    """
    import torch
    if rot_dim < 16 or rot_dim % 16 != 0:
        _bad("rope_inv_freq", f"rot_dim must be a multiple of 16, got {rot_dim}")
    if not (base > 1.0 and math.isfinite(base)) or not (factor >= 1.0 and math.isfinite(factor)):
        _bad("rope_inv_freq", "base must be > 1 and factor >= 1")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -i / rot_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if not high_freq_factor > low_freq_factor:
            _bad("rope_inv_freq", "high_freq_factor must exceed low_freq_factor")
        turns = original_max_position * f / (2 * math.pi)
        keep = ((turns - low_freq_factor) / (high_freq_factor - low_freq_factor)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    elif scaling == "yarn":
        at = lambda turns: rot_dim * math.log(original_max_position / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rot_dim - 1)
        keep = 1.0 - ((i / 2 - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        _bad("rope_inv_freq", f"unknown scaling {scaling!r}")
    return f.to(device), scale


class Rope:
    """A rotary embedding: float64 frequencies [rot_dim/2] on the GPU (radians
    per position, as from rope_inv_freq), the factor on cosine and sine, and
    which values form a pair: (i, i + rot_dim/2), or (2i, 2i + 1) when
    ``interleaved``."""

    def __init__(self, inv_freq, scale=1.0, interleaved=False):
        import torch
        if inv_freq.dim() != 1 or inv_freq.dtype != torch.float64 or not inv_freq.is_contiguous():
            _bad("Rope", "inv_freq must be a contiguous float64 vector [rot_dim / 2]")
        if inv_freq.numel() < 8 or inv_freq.numel() % 8 != 0:
            _bad("Rope", f"inv_freq must have a multiple of 8 entries, got {inv_freq.numel()}")
        if not inv_freq.is_cuda:
            _bad("Rope", f"inv_freq must be on a CUDA device, got {inv_freq.device}")
        if not (scale > 0.0 and math.isfinite(scale)):
            _bad("Rope", "scale must be finite and > 0")
        self.inv_freq, self.scale, self.interleaved = inv_freq, float(scale), bool(interleaved)
        self.rot_dim = 2 * inv_freq.numel()
        self.device = inv_freq.device
        self._spec = _RopeSpec(inv_freq.data_ptr(), self.rot_dim, int(self.interleaved), self.scale)
        self._ref = ctypes.byref(self._spec)


class PagedKV:
    """A paged cache and the sequences in it: k_cache, v_cache f16/bf16
    [num_pages, num_kv_heads, page_size, D] (any strides with contiguous rows, so
    a [num_pages, page_size, num_kv_heads, D] cache is passed transposed),
    page_table int32 [num_seqs, max_pages], seq_lens int32 [num_seqs] (the keys
    of each sequence, the new ones of the current call included)."""

    def __init__(self, k_cache, v_cache, page_table, seq_lens):
        import torch
        what = "PagedKV"
        if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
            _bad(what, "k_cache and v_cache must be [num_pages, num_kv_heads, page_size, D] of one shape")
        self.dtype, self._code = k_cache.dtype, _dtype_code(k_cache)
        if v_cache.dtype != k_cache.dtype:
            _bad(what, f"v_cache must be {k_cache.dtype}, got {v_cache.dtype}")
        self.num_pages, self.num_kv_heads, self.page_size, self.D = k_cache.shape
        if self.D not in (64, 128):
            raise FaError(FA_ERR_UNSUPPORTED, f"{what}: D must be 64 or 128, got {self.D}")
        if self.page_size < 8 or self.page_size % 8 != 0 or self.page_size > 65536:
            _bad(what, f"page_size must be a multiple of 8 up to 65536, got {self.page_size}")
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.numel() == 0:
            _bad(what, "page_table must be an int32 [num_seqs, max_pages] table")
        self.num_seqs, self.max_pages = page_table.shape
        if seq_lens.dim() != 1 or seq_lens.dtype != torch.int32 or seq_lens.numel() != self.num_seqs:
            _bad(what, f"seq_lens must be an int32 vector of {self.num_seqs} entries")
        if (self.max_pages > 1 and page_table.stride(1) != 1) or (self.num_seqs > 1 and
                                                                  page_table.stride(0) < self.max_pages):
            _bad(what, "page_table rows must be contiguous and apart")
        if self.num_seqs > 1 and seq_lens.stride(0) != 1:
            _bad(what, "seq_lens must be contiguous")
        if self.num_pages < 1 or self.num_kv_heads < 1 or self.max_pages * self.page_size > 1 << 30:
            _bad(what, "the cache needs a page and a head, and max_pages * page_size must be at most 2^30")
        for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
            if t.stride(3) != 1 or any(n > 1 and (s % 8 or s < self.D) for n, s in zip(t.shape[:3], t.stride()[:3])):
                _bad(what, f"{name} rows must be contiguous, with strides that are multiples of 8 and at least D")
            if t.data_ptr() % 16:
                _bad(what, f"{name} must start 16-byte aligned")
        for t in (k_cache, v_cache, page_table, seq_lens):
            if not t.is_cuda:
                _bad(what, f"every tensor must be on a CUDA device, got {t.device}")
            if t.device != k_cache.device:
                _bad(what, f"every tensor must be on {k_cache.device}, got {t.device}")
        self.k_cache, self.v_cache, self.page_table, self.seq_lens = k_cache, v_cache, page_table, seq_lens
        self.device = k_cache.device
        self._spec = _PagedSpec(
            k_cache.data_ptr(), v_cache.data_ptr(), _LL3(*k_cache.stride()[:3]), _LL3(*v_cache.stride()[:3]),
            page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), self.num_seqs, self.max_pages,
            self.num_pages, self.num_kv_heads, self.page_size, self.D, self._code)
        self._ref = ctypes.byref(self._spec)


def _on_current(what, device):
    """Refuse tensors of another device than the current one; returns its index."""
    import torch
    index = torch._C._cuda_getDevice()
    if device.index != index:
        _bad(what, f"every tensor must be on the current device cuda:{index}, got {device}")
    return index


def _stream_of(stream, device_index):
    """Handle of ``stream``: a torch stream, a raw handle or None (the current one)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(device_index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _rows(what, name, t, shape, dtype, device, low=0):
    """Check a 16-bit tensor whose last dimension is contiguous; its other
    strides must be multiples of 8 elements and at least `low` (an output's rows
    must not overlap, so D).  Returns its address and strides."""
    if t is None:
        _bad(what, f"{name} is required")
    if t.shape != shape:
        _bad(what, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        _bad(what, f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        _bad(what, f"{name} must be on {device}, got {t.device}")
    st, ptr = t.stride(), t.data_ptr()
    # rows, heads and batches at once (a packed tensor has no batches); what one of
    # them is wrong about is found below, where extents of 1 are let through
    if st[-1] != 1 or (st[-2] | st[-3] | st[0]) & 7 or st[-2] < low or st[-3] < low or st[0] < low or ptr & 15:
        if st[-1] != 1:
            _bad(what, f"{name} rows must be contiguous")
        for n, s in zip(shape, st[:-1]):
            if (s & 7 or s < low) and n > 1:
                _bad(what, f"{name} strides must be multiples of 8" + (" and at least D" if low else ""))
        if ptr & 15:
            _bad(what, f"{name} must start 16-byte aligned")
    return ptr, st


def _int32(what, name, x):
    """`x` as an int that a C int holds: ctypes would take it modulo 2^32."""
    x = int(x)
    if not -2147483648 <= x <= 2147483647:
        _bad(what, f"{name} must fit in 32 bits, got {x}")
    return x


_AS_IT_IS = contextlib.nullcontext()


def _allocating_on(stream):
    """Context in which torch allocates for ``stream`` (the current one if None):
    memory that a kernel of another stream fills must not come from, nor go back
    to, the pool of the current one."""
    if stream is None:
        return _AS_IT_IS
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)


def _need_rope(what, rope):
    if not isinstance(rope, Rope):
        _bad(what, "rope must be a Rope")


def _positions(what, positions, B, N, device):
    """(pointer, stride between batches) of int32 positions [B, N], or [N] for every batch."""
    if positions is None:
        return None, 0
    import torch
    if positions.dtype is not torch.int32:
        _bad(what, f"positions must be torch.int32, got {positions.dtype}")
    shape, st = positions.shape, positions.stride()
    if shape != (B, N) and shape != (N,):
        _bad(what, f"positions must have shape {(B, N)} or {(N,)}, got {tuple(shape)}")
    if st[-1] != 1 and N > 1:
        _bad(what, "positions must be contiguous along the rows")
    if positions.device != device:
        _bad(what, f"positions must be on {device}, got {positions.device}")
    bstride = st[0] if len(st) == 2 and B > 1 else 0
    if bstride < 0:
        _bad(what, "positions must not have negative strides")
    return positions.data_ptr(), bstride


def _rope_call(what, q, k, q_out, k_out, rope, positions, offset, stream, fresh=False):
    """fresh: the outputs come from empty_like, so they are as they have to be."""
    if q is None or q.dim() not in (3, 4):
        _bad(what, "q must be [B, H, N, D] or [H, total, D]")
    code = _dtype_code(q)
    _need_rope(what, rope)
    shape = q.shape
    D, N, B = shape[-1], shape[-2], shape[0] if len(shape) == 4 else 1
    if rope.rot_dim > D:
        _bad(what, f"rot_dim {rope.rot_dim} exceeds D {D}")
    if D % 8 or D < 16 or D > 512:
        raise FaError(FA_ERR_UNSUPPORTED, f"{what}: D must be a multiple of 8 from 16 to 512, got {D}")
    offset = _int32(what, "offset", offset)
    if not q.is_cuda:
        _bad(what, f"every tensor must be on a CUDA device, got {q.device}")
    current = _on_current(what, q.device)
    if rope.device != q.device:
        _bad(what, f"rope must be on {q.device}, got {rope.device}")
    dtype, device = q.dtype, q.device
    qp, qs = _rows(what, "q", q, shape, dtype, device)
    qop, qos = (q_out.data_ptr(), q_out.stride()) if fresh else _rows(what, "q_out", q_out, shape, dtype, device, D)
    Hk, kp, kop, ks, kos = 0, None, None, None, None
    if k is not None:
        if k.dim() != len(shape):
            _bad(what, "k must have as many dimensions as q")
        Hk = k.shape[-3]
        kshape = (*shape[:-3], Hk, N, D)
        kp, ks = _rows(what, "k", k, kshape, dtype, device)
        kop, kos = (k_out.data_ptr(), k_out.stride()) if fresh else _rows(what, "k_out", k_out, kshape, dtype, device, D)
        if Hk == 0:
            kp = kop = ks = kos = None
    elif k_out is not None:
        _bad(what, "k_out without k")
    pp, pstride = _positions(what, positions, B, N, device)
    f = lib().fa_rope if what == "fa_rope" else lib().fa_rope_bwd
    if len(shape) == 4:     # three strides beside the values', packed rows [H, total, D] have two
        qs, qos = _strides4(*qs), _strides4(*qos)
        if Hk:
            ks, kos = _strides4(*ks), _strides4(*kos)
    else:
        qs, qos = _strides3(0, qs[0], qs[1]), _strides3(0, qos[0], qos[1])
        if Hk:
            ks, kos = _strides3(0, ks[0], ks[1]), _strides3(0, kos[0], kos[1])
    st = f(qp, qs, qop, qos, shape[-3], kp, ks, kop, kos, Hk, B, N, D, rope._ref, pp, pstride, offset, code,
           _stream_of(stream, current))
    if st != FA_OK:
        _check(st, what)


def fa_rope(q, k, q_out, k_out, rope, positions=None, offset=0, stream=None):
    """Rotate q [B,Hq,N,D] and k [B,Hk,N,D] (or packed [H,total,D]; k may be
    None) into caller-owned q_out, k_out (which may be q and k).  Row n is at
    ``positions[b, n]`` (int32 [B,N] or [N]) or at ``offset + n``."""
    _rope_call("fa_rope", q, k, q_out, k_out, rope, positions, offset, stream)


def fa_rope_bwd(dq_out, dk_out, dq, dk, rope, positions=None, offset=0, stream=None):
    """Gradients of fa_rope with respect to q and k into caller-owned dq, dk."""
    _rope_call("fa_rope_bwd", dq_out, dk_out, dq, dk, rope, positions, offset, stream)


def rope_forward(q, k, rope, positions=None, offset=0, stream=None):
    """Allocate the rotated q and k with torch and run ``fa_rope``."""
    import torch
    with _allocating_on(stream):
        q_out = torch.empty_like(q)
        k_out = None if k is None else torch.empty_like(k)
    _rope_call("fa_rope", q, k, q_out, k_out, rope, positions, offset, stream, fresh=True)
    return q_out, k_out


def rope_backward(dq_out, dk_out, rope, positions=None, offset=0, stream=None):
    """Allocate dq and dk with torch and run ``fa_rope_bwd``."""
    import torch
    with _allocating_on(stream):
        dq = torch.empty_like(dq_out)
        dk = None if dk_out is None else torch.empty_like(dk_out)
    _rope_call("fa_rope_bwd", dq_out, dk_out, dq, dk, rope, positions, offset, stream, fresh=True)
    return dq, dk


def rope_attention_forward(q, k, v, rope, positions=None, offset=0, causal=False, scale=None, key_bias=None,
                           stream=None):
    """attention_forward of the rotated q and k; returns (o, lse, q_rot, k_rot),
    the last two for rope_attention_backward.  Like attention_forward it takes as
    many heads of k and v as of q; grouped ones are rotated by rope_forward."""
    from . import attention_forward
    with _allocating_on(stream):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        q_rot, k_rot = rope_forward(q, k, rope, positions=positions, offset=offset, stream=stream)
        o, lse = attention_forward(q_rot, k_rot, v, causal=causal, scale=scale, key_bias=key_bias, stream=stream)
    return o, lse, q_rot, k_rot


def rope_attention_backward(q_rot, k_rot, v, o, lse, dO, rope, positions=None, offset=0, causal=False, scale=None,
                            key_bias=None, stream=None):
    """Gradients of rope_attention_forward with respect to q, k (before the
    rotation) and v."""
    from . import attention_backward
    with _allocating_on(stream):
        dq, dk, dv = attention_backward(q_rot, k_rot, v.contiguous(), o, lse, dO, causal=causal, scale=scale,
                                        key_bias=key_bias, stream=stream)
    fa_rope_bwd(dq, dk, dq, dk, rope, positions=positions, offset=offset, stream=stream)
    return dq, dk, dv


def _cu(what, kv, cu):
    import torch
    if cu is None or cu.dtype is not torch.int32 or cu.dim() != 1 or not cu.is_contiguous():
        _bad(what, "cu_seqlens_q must be a contiguous int32 vector [num_seqs + 1]")
    if cu.shape[0] != kv.num_seqs + 1:
        _bad(what, f"cu_seqlens_q must have num_seqs + 1 = {kv.num_seqs + 1} entries, got {cu.shape[0]}")
    if cu.device != kv.device:
        _bad(what, f"cu_seqlens_q must be on {kv.device}, got {cu.device}")
    return cu.data_ptr()


def _need_kv(what, kv):
    if not isinstance(kv, PagedKV):
        _bad(what, "kv must be a PagedKV")
    return _on_current(what, kv.device)


def fa_paged_append(kv, k, v, cu_seqlens_q, rope=None, positions=None, q=None, q_out=None, stream=None):
    """Store the new keys (rotated by ``rope``) and values [num_kv_heads,
    total_q, D] of a ragged batch in the cache, and, with q [Hq, total_q, D],
    write the rotated queries to q_out (see include/fa.h)."""
    what = "fa_paged_append"
    current = _need_kv(what, kv)
    if k is None or k.dim() != 3:
        _bad(what, "k must be [num_kv_heads, total_q, D]")
    T, D = k.shape[1], kv.D
    shape = (kv.num_kv_heads, T, D)
    kp, ks = _rows(what, "k", k, shape, kv.dtype, kv.device)
    vp, vs = _rows(what, "v", v, shape, kv.dtype, kv.device)
    cup = _cu(what, kv, cu_seqlens_q)
    ref, pp = None, None
    if rope is not None:
        _need_rope(what, rope)
        if rope.rot_dim > D:
            _bad(what, f"rot_dim {rope.rot_dim} exceeds D {D}")
        if rope.device != kv.device:
            _bad(what, f"rope must be on {kv.device}, got {rope.device}")
        ref = rope._ref
        if positions is not None:
            pp, _ = _positions(what, positions, 1, T, kv.device)
    elif positions is not None or q is not None:
        _bad(what, "positions and q need a rope")
    H, qp, qop, qs, qos = 0, None, None, None, None
    if q is not None:
        if q.dim() != 3:
            _bad(what, "q must be [Hq, total_q, D]")
        H = q.shape[0]
        qp, st = _rows(what, "q", q, (H, T, D), kv.dtype, kv.device)
        qs = _strides2(st[0], st[1])
        qop, st = _rows(what, "q_out", q_out, (H, T, D), kv.dtype, kv.device, D)
        qos = _strides2(st[0], st[1])
    elif q_out is not None:
        _bad(what, "q_out without q")
    st = lib().fa_paged_append(kv._ref, kp, _strides2(ks[0], ks[1]), vp, _strides2(vs[0], vs[1]), cup, T, ref, pp, qp, qs, qop,
                               qos, H, _stream_of(stream, current))
    if st != FA_OK:
        _check(st, what)


def fa_paged_fwd_workspace_bytes(kv, Hq, max_seqlen_q) -> int:
    what = "fa_paged_fwd_workspace_bytes"
    if not isinstance(kv, PagedKV):
        _bad(what, "kv must be a PagedKV")
    Hq, max_seqlen_q = _int32(what, "Hq", Hq), _int32(what, "max_seqlen_q", max_seqlen_q)
    return int(lib().fa_paged_fwd_workspace_bytes(kv._ref, Hq, max_seqlen_q))


def _heads(what, kv, H):
    if H % kv.num_kv_heads or not 1 <= H // kv.num_kv_heads <= 128:
        _bad(what, f"Hq must be 1 to 128 times the cache's {kv.num_kv_heads} heads, got {H}")


def _bound(what, max_seqlen_q):
    max_seqlen_q = _int32(what, "max_seqlen_q", max_seqlen_q)
    if max_seqlen_q < 0:
        _bad(what, f"max_seqlen_q must be >= 0, got {max_seqlen_q}")
    return max_seqlen_q


def fa_paged_fwd(kv, q, o, lse, cu_seqlens_q, max_seqlen_q, workspace, causal=True, scale=None, stream=None):
    """Attention of the new rows q [Hq, total_q, D] of a ragged batch over the
    paged cache into caller-owned o (same shape) and lse float32 [Hq, total_q],
    with a caller-owned workspace of fa_paged_fwd_workspace_bytes() bytes (see
    include/fa.h).  ``causal`` is on by default: a new row sees the keys up to
    its own."""
    import torch
    what = "fa_paged_fwd"
    current = _need_kv(what, kv)
    if q is None or q.dim() != 3:
        _bad(what, "q must be [Hq, total_q, D]")
    H, T, D = q.shape
    _heads(what, kv, H)
    shape = (H, T, kv.D)
    qp, qs = _rows(what, "q", q, shape, kv.dtype, kv.device, D)
    op, os_ = _rows(what, "o", o, shape, kv.dtype, kv.device, D)
    if lse is None or lse.shape != (H, T) or lse.dtype is not torch.float32 or not lse.is_contiguous():
        _bad(what, f"lse must be a contiguous torch.float32 tensor of shape {(H, T)}")
    if lse.device != kv.device:
        _bad(what, f"lse must be on {kv.device}, got {lse.device}")
    if workspace is None or not workspace.is_contiguous() or workspace.device != kv.device:
        _bad(what, f"workspace must be a contiguous tensor on {kv.device}")
    max_seqlen_q = _bound(what, max_seqlen_q)
    cup = _cu(what, kv, cu_seqlens_q)
    st = lib().fa_paged_fwd(kv._ref, qp, _strides2(qs[0], qs[1]), op, _strides2(os_[0], os_[1]), lse.data_ptr(), cup, T,
                            max_seqlen_q, H, int(bool(causal)),
                            1.0 / math.sqrt(D) if scale is None else float(scale), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream_of(stream, current))
    if st != FA_OK:
        _check(st, what)


def paged_attention(kv, q, cu_seqlens_q, max_seqlen_q, causal=True, scale=None, stream=None):
    """Allocate O, LSE and the workspace with torch and run ``fa_paged_fwd``."""
    import torch
    if q is None or q.dim() != 3:
        _bad("fa_paged_fwd", "q must be [Hq, total_q, D]")
    _need_kv("fa_paged_fwd", kv)
    with _allocating_on(stream):
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        ws = torch.empty(fa_paged_fwd_workspace_bytes(kv, q.shape[0], max_seqlen_q), dtype=torch.uint8, device=kv.device)
    fa_paged_fwd(kv, q, o, lse, cu_seqlens_q, max_seqlen_q, ws, causal=causal, scale=scale, stream=stream)
    return o, lse


def paged_step(kv, q, k, v, cu_seqlens_q, max_seqlen_q, rope=None, positions=None, causal=True, scale=None,
               stream=None):
    """One layer's attention of a serving step: store the new keys and values
    (rotated, and q with them, when there is a rope), then attend over the
    cache.  Returns (o, lse).  A call that is refused has stored nothing."""
    import torch
    what = "paged_step"
    # what the attention would refuse, ahead of the append (which checks the rest)
    _need_kv(what, kv)
    if q is None or q.dim() != 3:
        _bad(what, "q must be [Hq, total_q, D]")
    H, T = q.shape[:2]
    _heads(what, kv, H)
    _rows(what, "q", q, (H, T, kv.D), kv.dtype, kv.device, kv.D if rope is None else 0)
    if H * T > 2147483647:
        _bad(what, f"Hq * total_q must fit in 31 bits, got {H} * {T}")
    _bound(what, max_seqlen_q)
    if scale is not None and not 0.0 < ctypes.c_float(float(scale)).value < math.inf:
        _bad(what, f"scale must be finite and > 0 in float32, got {scale}")
    if rope is None and positions is not None:
        _bad(what, "positions need a rope")
    q_rot = q
    if rope is not None:
        with _allocating_on(stream):
            q_rot = torch.empty_like(q)
        fa_paged_append(kv, k, v, cu_seqlens_q, rope=rope, positions=positions, q=q, q_out=q_rot, stream=stream)
    else:
        fa_paged_append(kv, k, v, cu_seqlens_q, stream=stream)
    return paged_attention(kv, q_rot, cu_seqlens_q, max_seqlen_q, causal=causal, scale=scale, stream=stream)
