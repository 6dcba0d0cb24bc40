"""Thin Python binding of the operators around a paged cache (argument
marshalling only, as in binding.py): norms and rotation of queries and keys
with their backward, append, read-back and one-query decode, for caches held
in 16 bits and in 4.  The definitions are those of include/gbattn.h.

All tensors of a call lie on one device.  The call is enqueued there, on
`stream` or on that device's current stream, whichever device is current.
"""
from __future__ import annotations

import ctypes
import math

import torch

from .binding import GBATTN_BF16, GBATTN_F16, GBATTN_OK, GbattnError, load_library

_DTYPES = {torch.float16: GBATTN_F16, torch.bfloat16: GBATTN_BF16}
_FACTOR_DTYPES = (torch.float8_e4m3fn, torch.uint8)
_Strides = ctypes.c_longlong * 3


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of position * base^(-2 i / rot_dim) for positions
    0 .. rows - 1, as the operators take them: fp32 [rows, rot_dim], a row's
    cosines first.  The angles are formed in 64 bits."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    a = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _on(fn, name, args, device, stream):
    """fn(*args, stream) with `device` current; raises the library's error."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    ptr = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, ptr)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, ptr)
    if rc != GBATTN_OK:
        raise GbattnError(rc, name)


def _rows(t, name, shape, dtype, device):
    """Checks a [B, heads, S, d] tensor whose rows are contiguous; its strides
    for the C ABI (None where it is contiguous)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {'[B, heads, S, d]' if shape is None else tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device} (there is no CPU path), got {t.device}")
    if t.is_contiguous():
        return None
    sb, sh, ss, sd = t.stride()
    if sd != 1 or (sb | sh | ss) % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name} needs contiguous rows of d elements that start on 16-byte boundaries, "
                         f"got strides {t.stride()}")
    return _Strides(sb, sh, ss)


def _plain(t, name, shape, dtypes, device):
    """Checks a contiguous tensor; its address, or None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {device}")
    return t.data_ptr()


_F32, _I32 = (torch.float32,), (torch.int32,)


def _first(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}; expected float16 or bfloat16")
    if t.dim() != 4:
        raise ValueError(f"{name} must have 4 dims, got shape {tuple(t.shape)}")
    return t.device, t.dtype


def _rope(rope, device):
    if rope is None:
        return None, 0, 0
    if not isinstance(rope, torch.Tensor) or rope.dim() != 2:
        raise ValueError("rope must be a tensor [rows, rot_dim] (see rope_table)")
    return _plain(rope, "rope", rope.shape, _F32, device), rope.shape[0], rope.shape[1]


def _norm_rope_args(q, k, q_weight, k_weight, rope, positions):
    device, dtype = _first(q, "q")
    B, H, S, d = q.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a tensor [B, Hkv, S, d]")
    Hkv = k.shape[1]
    qs = _rows(q, "q", q.shape, dtype, device)
    ks = _rows(k, "k", (B, Hkv, S, d), dtype, device)
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together: both, or neither (rotation alone)")
    if q_weight is None and rope is None:
        raise ValueError("nothing to do: neither norm weights nor a rotation table")
    table, rows, rot = _rope(rope, device)
    if rope is not None and positions is None and rows < S:
        raise ValueError(f"rope has {rows} rows for {S} tokens")
    ptrs = (_plain(q_weight, "q_weight", (d,), _F32, device), _plain(k_weight, "k_weight", (d,), _F32, device), table,
            _plain(positions, "positions", (B, S), _I32, device))
    return device, dtype, (B, H, Hkv, S, d), qs, ks, ptrs, rows, rot


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head with the position rotation, through
    the C ABI `attn_qk_norm_rope`.

    q [B,H,S,d], k [B,Hkv,S,d] fp16 or bf16 with contiguous rows (views of a
    projection output need no copy); q_weight, k_weight fp32 [d], or both None
    (rotation alone); rope fp32 [rows, rot_dim] from rope_table, or None (norm
    alone); positions int32 [B,S], or None (0 .. S-1).  Returns contiguous
    (q_out, k_out), which may be given as q and k themselves."""
    device, dtype, (B, H, Hkv, S, d), qs, ks, ptrs, rows, rot = _norm_rope_args(q, k, q_weight, k_weight, rope,
                                                                                positions)
    if q_out is None:
        q_out = torch.empty((B, H, S, d), dtype=dtype, device=device)
    if k_out is None:
        k_out = torch.empty((B, Hkv, S, d), dtype=dtype, device=device)
    outs = (_plain(q_out, "q_out", (B, H, S, d), (dtype,), device),
            _plain(k_out, "k_out", (B, Hkv, S, d), (dtype,), device))
    _on(load_library().attn_qk_norm_rope, "attn_qk_norm_rope",
        (q.data_ptr(), k.data_ptr(), *ptrs, *outs, B, H, Hkv, S, d, qs, ks, float(eps), rows, rot,
         int(bool(interleaved)), _DTYPES[dtype]), device, stream)
    return q_out, k_out


def attn_qk_norm_rope_bwd_workspace_bytes(d: int) -> int:
    return int(load_library().attn_qk_norm_rope_bwd_workspace_bytes(d))


def attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope=None, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, workspace=None, dq=None, dk=None,
                          dq_weight=None, dk_weight=None, stream=None):
    """Gradients of attn_qk_norm_rope through the C ABI `attn_qk_norm_rope_bwd`.

    dq_out, dk_out: the (contiguous) gradients of its outputs; the other inputs
    as it got them.  dq and dk may be given at any strides that q and k may
    have, for instance as views of the projection output's gradient.  Returns
    (dq, dk, dq_weight, dk_weight), the last two fp32 [d], or None without
    weights."""
    device, dtype, (B, H, Hkv, S, d), qs, ks, ptrs, rows, rot = _norm_rope_args(q, k, q_weight, k_weight, rope,
                                                                                positions)
    grads = (_plain(dq_out, "dq_out", (B, H, S, d), (dtype,), device),
             _plain(dk_out, "dk_out", (B, Hkv, S, d), (dtype,), device))
    if None in grads:
        raise TypeError("dq_out and dk_out must be tensors")
    lib = load_library()
    if dq is None:
        dq = torch.empty((B, H, S, d), dtype=dtype, device=device)
    if dk is None:
        dk = torch.empty((B, Hkv, S, d), dtype=dtype, device=device)
    dqs = _rows(dq, "dq", (B, H, S, d), dtype, device)
    dks = _rows(dk, "dk", (B, Hkv, S, d), dtype, device)
    ws_bytes = 0
    if q_weight is not None:
        if dq_weight is None:
            dq_weight = torch.empty(d, dtype=torch.float32, device=device)
        if dk_weight is None:
            dk_weight = torch.empty(d, dtype=torch.float32, device=device)
        if workspace is None:
            workspace = torch.empty(max(lib.attn_qk_norm_rope_bwd_workspace_bytes(d), 16), dtype=torch.uint8,
                                    device=device)
        ws_bytes = _workspace(workspace, device)
    _on(lib.attn_qk_norm_rope_bwd, "attn_qk_norm_rope_bwd",
        (*grads, q.data_ptr(), k.data_ptr(), *ptrs, dq.data_ptr(), dk.data_ptr(),
         _plain(dq_weight, "dq_weight", (d,), _F32, device), _plain(dk_weight, "dk_weight", (d,), _F32, device),
         B, H, Hkv, S, d, qs, ks, dqs, dks, float(eps), rows, rot, int(bool(interleaved)),
         workspace.data_ptr() if ws_bytes else None, ws_bytes, _DTYPES[dtype]), device, stream)
    return (dq, dk, dq_weight, dk_weight) if q_weight is not None else (dq, dk, None, None)


def _workspace(t, device):
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t.numel() * t.element_size()


def _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, device):
    """Checks a 16-bit cache and its tables: the pointers and the sizes."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.shape[1] != Hkv or k_cache.shape[3] != d:
        raise ValueError(f"k_cache must be a tensor [n_pages, {Hkv}, page_size, {d}]")
    n_pages, _, page, _ = k_cache.shape
    ptrs = (_plain(k_cache, "k_cache", k_cache.shape, (dtype,), device),
            _plain(v_cache, "v_cache", k_cache.shape, (dtype,), device))
    return _tables(ptrs, page_table, seqlens, B, device), (page, n_pages, page_table.shape[1])


def _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale, page_table, seqlens, B, Hkv, d, device):
    if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4 or k_codes.shape[1] != Hkv or \
            k_codes.shape[3] * 2 != d:
        raise ValueError(f"k_codes must be a tensor [n_pages, {Hkv}, page_size, {d // 2}]")
    n_pages, _, page, _ = k_codes.shape
    factors = (n_pages, Hkv, page, d // 16)
    ptrs = (_plain(k_codes, "k_codes", k_codes.shape, (torch.uint8,), device),
            _plain(k_factors, "k_factors", factors, _FACTOR_DTYPES, device),
            _plain(v_codes, "v_codes", k_codes.shape, (torch.uint8,), device),
            _plain(v_factors, "v_factors", factors, _FACTOR_DTYPES, device))
    if None in ptrs:
        raise TypeError("codes and factors must be tensors")
    ptrs += (_plain(k_descale, "k_descale", (Hkv,), _F32, device), _plain(v_descale, "v_descale", (Hkv,), _F32, device))
    return _tables(ptrs, page_table, seqlens, B, device), (page, n_pages, page_table.shape[1])


def _tables(ptrs, page_table, seqlens, B, device):
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a tensor [B, max_pages]")
    return ptrs + (_plain(page_table, "page_table", (B, page_table.shape[1]), _I32, device),
                   _plain(seqlens, "seqlens", (B,), _I32, device))


def _append(name, k, v, cache, new_lens, rope, interleaved, q, q_out, stream):
    device, dtype = _first(k, "k")
    B, Hkv, S, d = k.shape
    ks = _rows(k, "k", k.shape, dtype, device)
    vs = _rows(v, "v", k.shape, dtype, device)
    H, qs, q_ptr, out_ptr = Hkv, None, None, None
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 4:
            raise ValueError("q must be a tensor [B, H, S, d]")
        H = q.shape[1]
        qs = _rows(q, "q", (B, H, S, d), dtype, device)
        if q_out is None:
            q_out = torch.empty((B, H, S, d), dtype=dtype, device=device)
        q_ptr, out_ptr = q.data_ptr(), _plain(q_out, "q_out", (B, H, S, d), (dtype,), device)
    elif q_out is not None:
        raise ValueError("q_out without q")
    table, rows, rot = _rope(rope, device)
    ptrs, sizes = cache(B, Hkv, d, dtype, device)
    _on(getattr(load_library(), name), name,
        (k.data_ptr(), v.data_ptr(), *ptrs, _plain(new_lens, "new_lens", (B,), _I32, device), table, q_ptr, out_ptr,
         B, H, Hkv, S, d, *sizes, qs, ks, vs, rows, rot, int(bool(interleaved)), _DTYPES[dtype]), device, stream)
    return q_out


def attn_cache_append(k, v, k_cache, v_cache, page_table, seqlens, new_lens=None, rope=None,
                      interleaved: bool = False, q=None, q_out=None, stream=None):
    """Writes new keys and values into a 16-bit paged cache through the C ABI
    `attn_cache_append`, the keys (and q, if given) rotated on the way.

    k, v [B,Hkv,S,d] and q [B,H,S,d] (contiguous rows, any strides);
    k_cache, v_cache [n_pages,Hkv,page_size,d]; page_table int32 [B,max_pages];
    seqlens int32 [B], the new tokens included; new_lens int32 [B] (None: S);
    rope from rope_table, or None.  Returns the rotated queries (None without q)."""
    return _append("attn_cache_append", k, v,
                   lambda B, Hkv, d, dtype, dev: _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, dev),
                   new_lens, rope, interleaved, q, q_out, stream)


def attn_cache_append_fp4(k, v, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, new_lens=None,
                          k_descale=None, v_descale=None, rope=None, interleaved: bool = False, q=None, q_out=None,
                          stream=None):
    """attn_cache_append into a 4-bit paged cache (C ABI `attn_cache_append_fp4`):
    k_codes, v_codes uint8 [n_pages,Hkv,page_size,d/2]; k_factors, v_factors
    float8_e4m3fn (or uint8) [n_pages,Hkv,page_size,d/16]; k_descale, v_descale
    fp32 [Hkv] or None."""
    return _append("attn_cache_append_fp4", k, v,
                   lambda B, Hkv, d, dtype, dev: _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale,
                                                            v_descale, page_table, seqlens, B, Hkv, d, dev),
                   new_lens, rope, interleaved, q, q_out, stream)


def _gather(name, ptrs, sizes, B, Hkv, S, d, dtype, device, k_out, v_out, stream):
    if k_out is None:
        k_out = torch.empty((B, Hkv, S, d), dtype=dtype, device=device)
    if v_out is None:
        v_out = torch.empty((B, Hkv, S, d), dtype=dtype, device=device)
    outs = (_plain(k_out, "k_out", (B, Hkv, S, d), (dtype,), device),
            _plain(v_out, "v_out", (B, Hkv, S, d), (dtype,), device))
    _on(getattr(load_library(), name), name, (*ptrs, *outs, B, Hkv, S, d, *sizes, _DTYPES[dtype]), device, stream)
    return k_out, v_out


def attn_cache_gather(k_cache, v_cache, page_table, seqlens, S: int, k_out=None, v_out=None, stream=None):
    """The first S tokens of every sequence of a 16-bit paged cache as contiguous
    (k, v) [B,Hkv,S,d], zeros behind a sequence (C ABI `attn_cache_gather`)."""
    device, dtype = _first(k_cache, "k_cache")
    B, Hkv, d = _batch(seqlens), k_cache.shape[1], k_cache.shape[3]
    ptrs, sizes = _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, device)
    return _gather("attn_cache_gather", ptrs, sizes, B, Hkv, int(S), d, dtype, device, k_out, v_out, stream)


def attn_cache_gather_fp4(k_codes, k_factors, v_codes, v_factors, page_table, seqlens, S: int, k_descale=None,
                          v_descale=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """attn_cache_gather from a 4-bit paged cache, as fp16 or bf16 (C ABI
    `attn_cache_gather_fp4`)."""
    if not isinstance(k_codes, torch.Tensor) or not k_codes.is_cuda or k_codes.dim() != 4:
        raise ValueError("k_codes must be a CUDA tensor [n_pages, Hkv, page_size, d / 2] (there is no CPU path)")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; expected float16 or bfloat16")
    device = k_codes.device
    B, Hkv, d = _batch(seqlens), k_codes.shape[1], k_codes.shape[3] * 2
    ptrs, sizes = _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale, page_table, seqlens, B,
                             Hkv, d, device)
    return _gather("attn_cache_gather_fp4", ptrs, sizes, B, Hkv, int(S), d, dtype, device, k_out, v_out, stream)


def _batch(seqlens):
    if not isinstance(seqlens, torch.Tensor) or seqlens.dim() != 1:
        raise ValueError("seqlens must be an int32 tensor [B]")
    return seqlens.shape[0]


def attn_decode_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int) -> int:
    return int(load_library().attn_decode_paged_workspace_bytes(B, Hq, Hkv, d))


def _decode(name, q, Hkv, cache, scale, workspace, out, lse, return_lse, stream):
    device, dtype = _first(q, "q")
    B, H, one, d = q.shape
    if one != 1:
        raise ValueError("decode takes exactly one query per sequence: q [B,Hq,1,d]")
    q_ptr = _plain(q, "q", q.shape, (dtype,), device)
    ptrs, sizes = cache(B, d, dtype, device)
    lib = load_library()
    if workspace is None:
        workspace = torch.empty(max(lib.attn_decode_paged_workspace_bytes(B, H, Hkv, d), 16), dtype=torch.uint8,
                                device=device)
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=device)
    _on(getattr(lib, name), name,
        (q_ptr, *ptrs, _plain(out, "out", q.shape, (dtype,), device), _plain(lse, "lse", (B, H), _F32, device), B, H,
         Hkv, d, *sizes, 1.0 / math.sqrt(d) if scale is None else float(scale), workspace.data_ptr(),
         _workspace(workspace, device), _DTYPES[dtype]), device, stream)
    return out, lse


def attn_decode_paged(q, k_cache, v_cache, page_table, seqlens, scale: float | None = None, workspace=None, out=None,
                      lse=None, return_lse: bool = True, stream=None):
    """One-query decode over a 16-bit paged cache through the C ABI
    `attn_decode_paged`.

    q [B,Hq,1,d]; k_cache, v_cache [n_pages,Hkv,page_size,d]; page_table int32
    [B,max_pages]; seqlens int32 [B] (0: o = 0, lse = -inf).  workspace:
    optional buffer of attn_decode_paged_workspace_bytes(B, Hq, Hkv, d) bytes
    (allocated here if omitted).  Returns (o [B,Hq,1,d], lse [B,Hq] or None)."""
    Hkv = _kv_heads(k_cache, "k_cache")
    return _decode("attn_decode_paged", q, Hkv,
                   lambda B, d, dtype, dev: _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, dev),
                   scale, workspace, out, lse, return_lse, stream)


def attn_decode_paged_fp4(q, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, k_descale=None,
                          v_descale=None, scale: float | None = None, workspace=None, out=None, lse=None,
                          return_lse: bool = True, stream=None):
    """attn_decode_paged over a 4-bit paged cache (C ABI `attn_decode_paged_fp4`)."""
    Hkv = _kv_heads(k_codes, "k_codes")
    return _decode("attn_decode_paged_fp4", q, Hkv,
                   lambda B, d, dtype, dev: _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale,
                                                       page_table, seqlens, B, Hkv, d, dev),
                   scale, workspace, out, lse, return_lse, stream)


def _kv_heads(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a tensor of 4 dims [n_pages, Hkv, page_size, ..]")
    return t.shape[1]
