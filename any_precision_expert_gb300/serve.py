"""Thin Python binding of the calls around the layer: head norm and rotation,
the paged KV cache and its attention, draft verification (include/pw.h).

Only argument marshalling and shape checks happen here; every step runs in
libpw.so's kernels on the given (or current) stream, and no call synchronises.
"""
from __future__ import annotations

import ctypes as C

import torch

from ._lib import AttendDesc, Heads, KvDesc, RotaryDesc, Rows, check, lib
from .api import _p, _s

_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


def _dtype(t) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"heads are float16 or bfloat16, not {t.dtype}")
    return _DTYPES[t.dtype]


def _rows(t, T, H, D, dtype, what):
    """A [T, H, D] tensor of contiguous head rows as pw_rows."""
    if t is None:
        return None
    if tuple(t.shape) != (T, H, D) or t.dtype != dtype:
        raise ValueError(f"{what} must be [{T}, {H}, {D}] of {dtype}, not {tuple(t.shape)} of {t.dtype}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{what}: a head's values must be contiguous")
    return Rows(t.data_ptr(), st, sh)


def _vec(t, shape, dtype, what):
    """Device address of a contiguous tensor of a given shape and type."""
    if t is None:
        return None
    if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {list(shape)} tensor of {dtype}, not {tuple(t.shape)} of {t.dtype}")
    return t.data_ptr()


def _ref(s):
    return None if s is None else C.byref(s)


class Rotary:
    """Norm and rotation parameters (pw_rotary): cos_sin fp32 [max_pos, rot_dim] (cosines, then sines) or None for
    no rotation; q_weight / k_weight [head_dim] RMS norm weights or None."""

    def __init__(self, cos_sin, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False):
        max_pos, rot = (0, 0) if cos_sin is None else cos_sin.shape
        for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None and (w.dim() != 1 or not w.is_contiguous()):
                raise ValueError(f"{what} must be a contiguous [head_dim] tensor")
        self._keep = (cos_sin, q_weight, k_weight)
        self.desc = RotaryDesc(_vec(cos_sin, (max_pos, rot), torch.float32, "cos_sin"), max_pos, rot,
                               1 if interleaved else 0, _p(q_weight), _p(k_weight), eps)
        self._ref = C.byref(self.desc)

    def _check(self, dtype, D):
        for w in self._keep[1:]:
            if w is not None and (w.dtype != dtype or w.shape[0] != D):
                raise ValueError(f"norm weights must be [{D}] of {dtype}, not {list(w.shape)} of {w.dtype}")


def qk_norm_rope(rotary: Rotary, q, k, positions, q_out, k_out, err=None, stream=None):
    """RMS norm and rotation of query heads q [T, Hq, D] into q_out and key heads k [T, Hkv, D] into k_out, in one
    pass (pw_qk_norm_rope).  Either side may be None; outputs may be the inputs.  positions int32 [T]; err: optional
    int32 [1] error word."""
    some = q if q is not None else k
    if some is None or some.dim() != 3:
        raise ValueError("q or k must be [T, heads, head_dim]")
    T, H, D = some.shape
    hq, hk = (H if q is not None else k.shape[1]), (k.shape[1] if k is not None else H)
    if k is None:
        hk = hq
    rotary._check(some.dtype, D)
    heads = Heads(_dtype(some), hq, hk, D)
    check(lib.pw_qk_norm_rope(C.byref(heads), rotary._ref, _vec(positions, (T,), torch.int32, "positions"), T,
                              _ref(_rows(q, T, hq, D, some.dtype, "q")), _ref(_rows(k, T, hk, D, some.dtype, "k")),
                              _ref(_rows(q_out, T, hq, D, some.dtype, "q_out")),
                              _ref(_rows(k_out, T, hk, D, some.dtype, "k_out")), _p(err), _s(stream)),
          "pw_qk_norm_rope")


class KvCache:
    """Paged KV cache (pw_kv_create) over tensors k, v [n_pages, n_kv_heads, page_tokens, head_dim] of any strides
    with contiguous head rows (a [pages, tokens, heads, dim] cache is passed as its transpose(1, 2))."""

    def __init__(self, k, v, n_heads: int):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be [pages, kv heads, page tokens, head_dim] tensors of one layout")
        self.k, self.v = k, v
        n_pages, self.n_kv_heads, self.page_tokens, self.head_dim = k.shape
        self.n_heads, self.dtype = n_heads, k.dtype
        self.err = torch.zeros(1, dtype=torch.int32, device=k.device)
        desc = KvDesc(Heads(_dtype(k), n_heads, self.n_kv_heads, self.head_dim), self.page_tokens, n_pages,
                      k.stride(0), k.stride(1), k.stride(2))
        self.handle = C.c_void_p()
        check(lib.pw_kv_create(C.byref(desc), k.data_ptr(), v.data_ptr(), self.err.data_ptr(), C.byref(self.handle)),
              "pw_kv_create")

    def __del__(self):
        self.close()

    def close(self):
        if getattr(self, "handle", None):
            lib.pw_kv_destroy(self.handle)
            self.handle = None

    def check_device(self, stream=None) -> int:
        """Read and clear the error word (synchronises): 0 or PW_ERR_DEVICE_CHECK (7)."""
        return lib.pw_kv_check_device(self.handle, _s(stream))

    def append(self, k, v, slots, rotary: Rotary = None, positions=None, q=None, q_out=None, stream=None):
        """Append keys (normed and rotated when rotary is given) and values [T, Hkv, D] at int32 slots [T], and norm
        and rotate the queries q [T, Hq, D] into q_out in the same launch (pw_kv_append)."""
        T, D, dt = k.shape[0], self.head_dim, self.dtype
        if rotary is not None:
            rotary._check(dt, D)
        check(lib.pw_kv_append(self.handle, None if rotary is None else rotary._ref,
                               _vec(positions, (T,), torch.int32, "positions"), _vec(slots, (T,), torch.int32, "slots"),
                               T, C.byref(_rows(k, T, self.n_kv_heads, D, dt, "k")),
                               C.byref(_rows(v, T, self.n_kv_heads, D, dt, "v")),
                               _ref(_rows(q, T, self.n_heads, D, dt, "q")),
                               _ref(_rows(q_out, T, self.n_heads, D, dt, "q_out")), _s(stream)), "pw_kv_append")

    def attend_workspace_size(self, batch: int, q_len: int = 1, n_groups: int = 0) -> int:
        n = C.c_size_t(0)
        check(lib.pw_kv_attend_workspace_size(self.handle, batch, q_len, n_groups, C.byref(n)),
              "pw_kv_attend_workspace_size")
        return n.value

    def attend(self, q, table, lens, out, ws, q_len: int = 1, scale: float = None, prefix_table=None,
               prefix_lens=None, group_offsets=None, lse=None, stream=None):
        """Attention of q [B * q_len, Hq, D] over each sequence's own pages table int32 [B, pages] (lens int32 [B])
        behind its group's shared prefix (prefix_table int32 [groups, pages], prefix_lens int32 [groups],
        group_offsets int32 [groups + 1]; one group over the whole batch needs no offsets), into out and, when given,
        lse fp32 [B * q_len, Hq] (pw_kv_attend).  ws: uint8 scratch of attend_workspace_size bytes."""
        B, D, dt = table.shape[0], self.head_dim, self.dtype
        N, H = B * q_len, self.n_heads
        groups = 0 if prefix_lens is None else prefix_lens.shape[0]
        if groups and prefix_table is None:
            raise ValueError("prefix_lens needs prefix_table")
        desc = AttendDesc(_rows(q, N, H, D, dt, "q"), _rows(out, N, H, D, dt, "out"),
                          _vec(lse, (N, H), torch.float32, "lse"), B, q_len, D ** -0.5 if scale is None else scale,
                          _vec(table, (B, table.shape[1]), torch.int32, "table"), table.shape[1],
                          _vec(lens, (B,), torch.int32, "lens"), groups,
                          None if not groups else _vec(group_offsets, (groups + 1,), torch.int32, "group_offsets"),
                          None if not groups else _vec(prefix_table, (groups, prefix_table.shape[1]), torch.int32,
                                                       "prefix_table"),
                          prefix_table.shape[1] if groups else 0,
                          None if not groups else _vec(prefix_lens, (groups,), torch.int32, "prefix_lens"))
        check(lib.pw_kv_attend(self.handle, C.byref(desc), _p(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                               _s(stream)), "pw_kv_attend")


def verify_draft(target_p, draft_p, tokens, n_draft, u, noise, out, accepted, err=None, stream=None):
    """Verify drafted tokens int32 [B, K] (n_draft int32 [B] of them each) with target probabilities fp32 [B, K+1, V],
    draft probabilities fp32 [B, K, V], uniforms u [B, K] and exponential noise [B, V]: accepted int32 [B] tokens are
    kept, out int32 [B, K+1] holds them, the next token and -1s (pw_verify_draft)."""
    B, K1, V = target_p.shape
    K, f, i = K1 - 1, torch.float32, torch.int32
    check(lib.pw_verify_draft(_vec(target_p, (B, K1, V), f, "target_p"), _vec(draft_p, (B, K, V), f, "draft_p"),
                              _vec(tokens, (B, K), i, "tokens"), _vec(n_draft, (B,), i, "n_draft"),
                              _vec(u, (B, K), f, "u"), _vec(noise, (B, V), f, "noise"), B, K, V,
                              _vec(out, (B, K1), i, "out"), _vec(accepted, (B,), i, "accepted"), _p(err), _s(stream)),
          "pw_verify_draft")
