"""Thin Python binding of the calls around the layer: head norm and rotation,
the paged KV cache and its attention, draft verification (include/pw.h).

Only argument marshalling and shape checks happen here and in the compiled
module ``_pw_torch`` (csrc/pw_torch.cpp); every step runs in libpw.so's kernels
on the given (or the tensors' device's current) stream, and no call
synchronises.  A wrong shape, type or device raises ValueError, what the
library refuses raises PwError.
"""
from __future__ import annotations

import ctypes as C

import torch

from . import _pw_torch
from ._lib import Heads, KvDesc, RotaryDesc, check, lib
from .api import _p, _s

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


class Rotary:
    """Norm and rotation parameters (pw_rotary): cos_sin fp32 [max_pos, rot_dim] (cosines, then sines) or None for
    no rotation; q_weight / k_weight [head_dim] RMS norm weights or None."""

    def __init__(self, cos_sin, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False):
        if cos_sin is not None and (cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or not cos_sin.is_contiguous()):
            raise ValueError("cos_sin must be a contiguous float32 [max_pos, rot_dim] tensor")
        max_pos, rot = (0, 0) if cos_sin is None else cos_sin.shape
        weights = [w for w in (q_weight, k_weight) if w is not None]
        for w in weights:
            if w.dim() != 1 or not w.is_contiguous() or w.shape != weights[0].shape or w.dtype != weights[0].dtype:
                raise ValueError("norm weights must be contiguous [head_dim] tensors of one type")
        given = [t for t in (cos_sin, q_weight, k_weight) if t is not None]
        if any(t.device != given[0].device for t in given):
            raise ValueError("cos_sin and the norm weights must be on one device")
        self._keep = (cos_sin, q_weight, k_weight)
        self.desc = RotaryDesc(_p(cos_sin), max_pos, rot, 1 if interleaved else 0, _p(q_weight), _p(k_weight), eps)
        self._key = (C.addressof(self.desc), _DTYPES.get(weights[0].dtype, len(_DTYPES)) if weights else -1,
                     weights[0].shape[0] if weights else 0, given[0] if given else None)


def qk_norm_rope(rotary: Rotary, q, k, positions, q_out, k_out, err=None, stream=None):
    """RMS norm and rotation of query heads q [T, Hq, D] into q_out and key heads k [T, Hkv, D] into k_out, in one
    pass (pw_qk_norm_rope).  Either side may be None; outputs may be the inputs.  positions int32 [T]; err: optional
    int32 [1] error word."""
    st = _pw_torch.qk_norm_rope(rotary._key, q, k, positions, q_out, k_out, err, stream)
    if st:
        check(st, "pw_qk_norm_rope")


class KvCache:
    """Paged KV cache (pw_kv_create) over tensors k, v [n_pages, n_kv_heads, page_tokens, head_dim] of any strides
    with contiguous head rows (a [pages, tokens, heads, dim] cache is passed as its transpose(1, 2))."""

    def __init__(self, k, v, n_heads: int):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.stride(3) != 1 \
                or k.device != v.device:
            raise ValueError("k and v must be [pages, kv heads, page tokens, head_dim] tensors of one layout")
        if k.dtype not in _DTYPES:
            raise ValueError(f"heads are float16 or bfloat16, not {k.dtype}")
        _pw_torch.check_cache(k)
        self.k, self.v = k, v
        n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = k.shape
        self.n_heads, self.dtype = n_heads, k.dtype
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        desc = KvDesc(Heads(_DTYPES[k.dtype], n_heads, self.n_kv_heads, self.head_dim), self.page_tokens, n_pages,
                      k.stride(0), k.stride(1), k.stride(2))
        handle = C.c_void_p()
        check(lib.pw_kv_create(C.byref(desc), k.data_ptr(), v.data_ptr(), self.err.data_ptr(), C.byref(handle)),
              "pw_kv_create")
        self.handle = handle.value

    def __del__(self):
        self.close()

    def close(self):
        if getattr(self, "handle", None):
            lib.pw_kv_destroy(self.handle)
            self.handle = 0  # calls on a closed cache answer PW_ERR_INVALID_ARG

    def check_device(self, stream=None) -> int:
        """Read and clear the error word (synchronises): 0 or PW_ERR_DEVICE_CHECK (7)."""
        return lib.pw_kv_check_device(self.handle, _s(stream))

    def append(self, k, v, slots, rotary: Rotary = None, positions=None, q=None, q_out=None, stream=None):
        """Append keys (normed and rotated when rotary is given) and values [T, Hkv, D] at int32 slots [T], and norm
        and rotate the queries q [T, Hq, D] into q_out in the same launch (pw_kv_append)."""
        st = _pw_torch.append(self.handle, self.k, self.n_heads, k, v, slots, None if rotary is None else rotary._key,
                              positions, q, q_out, stream)
        if st:
            check(st, "pw_kv_append")

    def attend_workspace_size(self, batch: int, q_len: int = 1, n_groups: int = 0) -> int:
        n = C.c_size_t(0)
        check(lib.pw_kv_attend_workspace_size(self.handle, batch, q_len, n_groups, C.byref(n)),
              "pw_kv_attend_workspace_size")
        return n.value

    def attend(self, q, table, lens, out, ws, q_len: int = 1, scale: float = None, prefix_table=None,
               prefix_lens=None, group_offsets=None, lse=None, stream=None):
        """Attention of q [B * q_len, Hq, D] over each sequence's own pages table int32 [B, pages] (lens int32 [B])
        behind its group's shared prefix (prefix_table int32 [groups, pages], prefix_lens int32 [groups],
        group_offsets int32 [groups + 1]; one group over the whole batch needs no offsets; no prefix: all three None),
        into out and, when given, lse fp32 [B * q_len, Hq] (pw_kv_attend).  ws: uint8 scratch of attend_workspace_size bytes."""
        st = _pw_torch.attend(self.handle, self.k, self.n_heads, q, table, lens, out, ws, q_len,
                              self.head_dim ** -0.5 if scale is None else scale, prefix_table, prefix_lens,
                              group_offsets, lse, stream)
        if st:
            check(st, "pw_kv_attend")


def verify_draft(target_p, draft_p, tokens, n_draft, u, noise, out, accepted, err=None, stream=None):
    """Verify drafted tokens int32 [B, K] (n_draft int32 [B] of them each) with target probabilities fp32 [B, K+1, V],
    draft probabilities fp32 [B, K, V], uniforms u [B, K] and exponential noise [B, V]: accepted int32 [B] tokens are
    kept, out int32 [B, K+1] holds them, the next token and -1s (pw_verify_draft)."""
    st = _pw_torch.verify_draft(target_p, draft_p, tokens, n_draft, u, noise, out, accepted, err, stream)
    if st:
        check(st, "pw_verify_draft")
