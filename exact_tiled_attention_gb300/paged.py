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
_F32, _I32, _U8, _E4M3 = torch.float32, torch.int32, torch.uint8, torch.float8_e4m3fn
_Strides = ctypes.c_longlong * 3
_get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of position * base^(-2 i / rot_dim) for positions
    0 .. rows - 1, as the operators take them: fp32 [rows, rot_dim], a row's
    cosines first.  The angles are formed in 64 bits."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    a = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


# A token's worth of work is a few microseconds on the device, so the checks are
# written for few interpreter steps: one compound condition for each tensor, and
# the reason worked out (_refuse) only where it fails.


def _call(name, args, device, stream):
    """The library's function `name` with `device` current; raises its error."""
    index = device.index
    if stream is None:
        stream = _raw_stream(index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    fn = getattr(_library(), name)
    if index == _get_device():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != GBATTN_OK:
        raise GbattnError(rc, name)


def _refuse(t, name, shape, dtype, device, rows=False):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device} (there is no CPU path)")
    if rows:
        raise ValueError(f"{name} needs contiguous rows of d elements that start on 16-byte boundaries, "
                         f"got strides {t.stride()}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(t, name, shape, dtype, device):
    """The address of a contiguous tensor."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, device)


def _opt(t, name, shape, dtype, device):
    return None if t is None else _ptr(t, name, shape, dtype, device)


def _rows(t, name, shape, dtype, device):
    """Address and strides (None: contiguous) of a [B, heads, S, d] tensor whose
    rows are contiguous."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device:
            if t.is_contiguous():
                return t.data_ptr(), None
            sb, sh, ss, sd = t.stride()
            if sd == 1 and not (sb | sh | ss) & 7:
                return t.data_ptr(), _Strides(sb, sh, ss)
    except AttributeError:
        pass
    _refuse(t, name, shape, dtype, device, rows=True)


def _first(t, name):
    """Device, type, the library's code for it and shape of the tensor that the
    others have to agree with."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} of {name}; expected float16 or bfloat16")
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{name} must have 4 dims, got shape {tuple(shape)}")
    return t.device, t.dtype, code, shape


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} dims")
    return t.shape


def _rope(rope, device):
    """Address, rows and width of the rotation's table."""
    if rope is None:
        return None, 0, 0
    shape = _dims(rope, "rope", 2)
    return _ptr(rope, "rope", shape, _F32, device), shape[0], shape[1]


def _norm_rope_args(q, k, q_weight, k_weight, rope, positions):
    device, dtype, code, shape = _first(q, "q")
    B, H, S, d = shape
    Hkv = _dims(k, "k", 4)[1]
    q_ptr, qs = _rows(q, "q", shape, dtype, device)
    k_ptr, ks = _rows(k, "k", (B, Hkv, S, d), dtype, device)
    table, rows, rot = _rope(rope, device)
    if q_weight is None or k_weight is None:
        if q_weight is not k_weight:
            raise ValueError("q_weight and k_weight go together: both, or neither (rotation alone)")
        if rope is None:
            raise ValueError("nothing to do: neither norm weights nor a rotation table")
        weights = None, None
    else:
        weights = _ptr(q_weight, "q_weight", (d,), _F32, device), _ptr(k_weight, "k_weight", (d,), _F32, device)
    if positions is None and table is not None and rows < S:
        raise ValueError(f"rope has {rows} rows for {S} tokens")
    ptrs = (q_ptr, k_ptr, *weights, table, _opt(positions, "positions", (B, S), _I32, device))
    return device, dtype, code, (B, H, Hkv, S, d), qs, ks, ptrs, rows, rot


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head with the position rotation, through
    the C ABI `attn_qk_norm_rope`.

    q [B,H,S,d], k [B,Hkv,S,d] fp16 or bf16 with contiguous rows (views of a
    projection output need no copy); q_weight, k_weight fp32 [d], or both None
    (rotation alone); rope fp32 [rows, rot_dim] from rope_table, or None (norm
    alone); positions int32 [B,S], or None (0 .. S-1).  Returns contiguous
    (q_out, k_out), which may be given as q and k themselves."""
    device, dtype, code, (B, H, Hkv, S, d), qs, ks, ptrs, rows, rot = _norm_rope_args(q, k, q_weight, k_weight, rope,
                                                                                      positions)
    if q_out is None:
        q_out = torch.empty((B, H, S, d), dtype=dtype, device=device)
        qo = q_out.data_ptr()
    else:
        qo = _ptr(q_out, "q_out", (B, H, S, d), dtype, device)
    if k_out is None:
        k_out = torch.empty((B, Hkv, S, d), dtype=dtype, device=device)
        ko = k_out.data_ptr()
    else:
        ko = _ptr(k_out, "k_out", (B, Hkv, S, d), dtype, device)
    _call("attn_qk_norm_rope", (*ptrs, qo, ko, B, H, Hkv, S, d, qs, ks, eps, rows, rot, 1 if interleaved else 0, code),
          device, stream)
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
    device, dtype, code, (B, H, Hkv, S, d), qs, ks, ptrs, rows, rot = _norm_rope_args(q, k, q_weight, k_weight, rope,
                                                                                      positions)
    q_shape, k_shape = (B, H, S, d), (B, Hkv, S, d)
    dqo = _ptr(dq_out, "dq_out", q_shape, dtype, device)
    dko = _ptr(dk_out, "dk_out", k_shape, dtype, device)
    if dq is None:
        dq = torch.empty(q_shape, dtype=dtype, device=device)
        dq_ptr, dqs = dq.data_ptr(), None
    else:
        dq_ptr, dqs = _rows(dq, "dq", q_shape, dtype, device)
    if dk is None:
        dk = torch.empty(k_shape, dtype=dtype, device=device)
        dk_ptr, dks = dk.data_ptr(), None
    else:
        dk_ptr, dks = _rows(dk, "dk", k_shape, dtype, device)
    if q_weight is None:
        dq_weight = dk_weight = None
        wgrads, ws, ws_bytes = (None, None), None, 0
    else:
        if dq_weight is None:
            dq_weight = torch.empty(d, dtype=_F32, device=device)
        if dk_weight is None:
            dk_weight = torch.empty(d, dtype=_F32, device=device)
        wgrads = (_ptr(dq_weight, "dq_weight", (d,), _F32, device), _ptr(dk_weight, "dk_weight", (d,), _F32, device))
        if workspace is None:
            workspace = torch.empty(max(_library().attn_qk_norm_rope_bwd_workspace_bytes(d), 16), dtype=_U8,
                                    device=device)
        ws, ws_bytes = _workspace(workspace, device)
    _call("attn_qk_norm_rope_bwd",
          (dqo, dko, *ptrs, dq_ptr, dk_ptr, *wgrads, B, H, Hkv, S, d, qs, ks, dqs, dks, eps, rows, rot,
           1 if interleaved else 0, ws, ws_bytes, code), device, stream)
    return dq, dk, dq_weight, dk_weight


def _workspace(t, device):
    """Address and bytes of a workspace."""
    if not isinstance(t, torch.Tensor) or t.device != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, device):
    """Addresses of a 16-bit cache and its tables; page size, pages, pages a sequence."""
    shape = _dims(k_cache, "k_cache", 4)
    n_pages, heads, page, width = shape
    if heads != Hkv or width != d:
        raise ValueError(f"k_cache must be a tensor [n_pages, {Hkv}, page_size, {d}], got {tuple(shape)}")
    max_pages = _dims(page_table, "page_table", 2)[1]
    return ((_ptr(k_cache, "k_cache", shape, dtype, device), _ptr(v_cache, "v_cache", shape, dtype, device),
             _ptr(page_table, "page_table", (B, max_pages), _I32, device), _ptr(seqlens, "seqlens", (B,), _I32, device)),
            (page, n_pages, max_pages))


def _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale, page_table, seqlens, B, Hkv, d, device):
    """The same of a 4-bit cache."""
    shape = _dims(k_codes, "k_codes", 4)
    n_pages, heads, page, width = shape
    if heads != Hkv or 2 * width != d:
        raise ValueError(f"k_codes must be a tensor [n_pages, {Hkv}, page_size, {d // 2}], got {tuple(shape)}")
    max_pages = _dims(page_table, "page_table", 2)[1]
    factors = (n_pages, Hkv, page, d // 16)
    as_bytes = _U8 if getattr(k_factors, "dtype", None) is _U8 else _E4M3
    return ((_ptr(k_codes, "k_codes", shape, _U8, device), _ptr(k_factors, "k_factors", factors, as_bytes, device),
             _ptr(v_codes, "v_codes", shape, _U8, device), _ptr(v_factors, "v_factors", factors, as_bytes, device),
             _opt(k_descale, "k_descale", (Hkv,), _F32, device), _opt(v_descale, "v_descale", (Hkv,), _F32, device),
             _ptr(page_table, "page_table", (B, max_pages), _I32, device), _ptr(seqlens, "seqlens", (B,), _I32, device)),
            (page, n_pages, max_pages))


def _append(name, first, k_ptr, ks, v, cache, new_lens, rope, interleaved, q, q_out, stream):
    device, dtype, code, shape = first
    B, Hkv, S, d = shape
    v_ptr, vs = _rows(v, "v", shape, dtype, device)
    if q is None:
        if q_out is not None:
            raise ValueError("q_out without q")
        H, q_ptr, qs, out_ptr = Hkv, None, None, None
    else:
        H = _dims(q, "q", 4)[1]
        q_shape = (B, H, S, d)
        q_ptr, qs = _rows(q, "q", q_shape, dtype, device)
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=dtype, device=device)
            out_ptr = q_out.data_ptr()
        else:
            out_ptr = _ptr(q_out, "q_out", q_shape, dtype, device)
    table, rows, rot = _rope(rope, device)
    ptrs, sizes = cache
    _call(name, (k_ptr, v_ptr, *ptrs, _opt(new_lens, "new_lens", (B,), _I32, device), table, q_ptr, out_ptr,
                 B, H, Hkv, S, d, *sizes, qs, ks, vs, rows, rot, 1 if interleaved else 0, code), device, stream)
    return q_out


def attn_cache_append(k, v, k_cache, v_cache, page_table, seqlens, new_lens=None, rope=None,
                      interleaved: bool = False, q=None, q_out=None, stream=None):
    """Writes new keys and values into a 16-bit paged cache through the C ABI
    `attn_cache_append`, the keys (and q, if given) rotated on the way.

    k, v [B,Hkv,S,d] and q [B,H,S,d] (contiguous rows, any strides);
    k_cache, v_cache [n_pages,Hkv,page_size,d]; page_table int32 [B,max_pages];
    seqlens int32 [B], the new tokens included; new_lens int32 [B] (None: S);
    rope from rope_table, or None.  Returns the rotated queries (None without q)."""
    first = device, dtype, _, (B, Hkv, _, d) = _first(k, "k")
    k_ptr, ks = _rows(k, "k", first[3], dtype, device)
    cache = _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, device)
    return _append("attn_cache_append", first, k_ptr, ks, v, cache, new_lens, rope, interleaved, q, q_out, stream)


def attn_cache_append_fp4(k, v, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, new_lens=None,
                          k_descale=None, v_descale=None, rope=None, interleaved: bool = False, q=None, q_out=None,
                          stream=None):
    """attn_cache_append into a 4-bit paged cache (C ABI `attn_cache_append_fp4`):
    k_codes, v_codes uint8 [n_pages,Hkv,page_size,d/2]; k_factors, v_factors
    float8_e4m3fn (or both uint8) [n_pages,Hkv,page_size,d/16]; k_descale,
    v_descale fp32 [Hkv] or None."""
    first = device, dtype, _, (B, Hkv, _, d) = _first(k, "k")
    k_ptr, ks = _rows(k, "k", first[3], dtype, device)
    cache = _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale, page_table, seqlens, B, Hkv, d,
                       device)
    return _append("attn_cache_append_fp4", first, k_ptr, ks, v, cache, new_lens, rope, interleaved, q, q_out, stream)


def _gather(name, cache, B, Hkv, S, d, dtype, device, k_out, v_out, stream):
    shape = (B, Hkv, S, d)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=device)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=device)
    ptrs, sizes = cache
    _call(name, (*ptrs, _ptr(k_out, "k_out", shape, dtype, device), _ptr(v_out, "v_out", shape, dtype, device), B, Hkv,
                 S, d, *sizes, _DTYPES[dtype]), device, stream)
    return k_out, v_out


def attn_cache_gather(k_cache, v_cache, page_table, seqlens, S: int, k_out=None, v_out=None, stream=None):
    """The first S tokens of every sequence of a 16-bit paged cache as contiguous
    (k, v) [B,Hkv,S,d], zeros behind a sequence (C ABI `attn_cache_gather`)."""
    device, dtype, _, (_, Hkv, _, d) = _first(k_cache, "k_cache")
    B = _dims(seqlens, "seqlens", 1)[0]
    cache = _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, device)
    return _gather("attn_cache_gather", cache, B, Hkv, int(S), d, dtype, device, k_out, v_out, stream)


def attn_cache_gather_fp4(k_codes, k_factors, v_codes, v_factors, page_table, seqlens, S: int, k_descale=None,
                          v_descale=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """attn_cache_gather from a 4-bit paged cache, as fp16 or bf16 (C ABI
    `attn_cache_gather_fp4`)."""
    _, Hkv, _, half = _dims(k_codes, "k_codes", 4)
    if not k_codes.is_cuda:
        raise ValueError("k_codes must be a CUDA tensor (there is no CPU path)")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}; expected float16 or bfloat16")
    device, B = k_codes.device, _dims(seqlens, "seqlens", 1)[0]
    cache = _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale, page_table, seqlens, B, Hkv,
                       2 * half, device)
    return _gather("attn_cache_gather_fp4", cache, B, Hkv, int(S), 2 * half, dtype, device, k_out, v_out, stream)


def attn_decode_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_len: int = 2 ** 31 - 1) -> int:
    """Bytes of the paged decodes' workspace; smaller where max_len, the tokens
    that max_pages pages hold, is short."""
    return int(load_library().attn_decode_paged_workspace_bytes(B, Hq, Hkv, d, max_len))


def _decode(name, first, q, cache, Hkv, scale, workspace, out, lse, return_lse, stream):
    device, dtype, code, shape = first
    B, H, one, d = shape
    if one != 1:
        raise ValueError("decode takes exactly one query per sequence: q [B,Hq,1,d]")
    ptrs, sizes = cache
    if workspace is None:
        need = _library().attn_decode_paged_workspace_bytes(B, H, Hkv, d, sizes[0] * sizes[2])
        workspace = torch.empty(max(need, 16), dtype=_U8, device=device)
        ws, ws_bytes = workspace.data_ptr(), need
    else:
        ws, ws_bytes = _workspace(workspace, device)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        o_ptr = out.data_ptr()
    else:
        o_ptr = _ptr(out, "out", shape, dtype, device)
    if lse is None:
        l_ptr = None
        if return_lse:
            lse = torch.empty((B, H), dtype=_F32, device=device)
            l_ptr = lse.data_ptr()
    else:
        l_ptr = _ptr(lse, "lse", (B, H), _F32, device)
    _call(name, (_ptr(q, "q", shape, dtype, device), *ptrs, o_ptr, l_ptr, B, H, Hkv, d, *sizes,
                 1.0 / math.sqrt(d) if scale is None else scale, ws, ws_bytes, code), device, stream)
    return out, lse


def attn_decode_paged(q, k_cache, v_cache, page_table, seqlens, scale: float | None = None, workspace=None, out=None,
                      lse=None, return_lse: bool = True, stream=None):
    """One-query decode over a 16-bit paged cache through the C ABI
    `attn_decode_paged`.

    q [B,Hq,1,d]; k_cache, v_cache [n_pages,Hkv,page_size,d]; page_table int32
    [B,max_pages]; seqlens int32 [B] (0: o = 0, lse = -inf).  workspace:
    optional buffer of attn_decode_paged_workspace_bytes(B, Hq, Hkv, d) bytes
    (allocated here if omitted).  Returns (o [B,Hq,1,d], lse [B,Hq] or None)."""
    first = device, dtype, _, (B, _, _, d) = _first(q, "q")
    Hkv = _dims(k_cache, "k_cache", 4)[1]
    cache = _cache(k_cache, v_cache, page_table, seqlens, B, Hkv, d, dtype, device)
    return _decode("attn_decode_paged", first, q, cache, Hkv, scale, workspace, out, lse, return_lse, stream)


def attn_decode_paged_fp4(q, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, k_descale=None,
                          v_descale=None, scale: float | None = None, workspace=None, out=None, lse=None,
                          return_lse: bool = True, stream=None):
    """attn_decode_paged over a 4-bit paged cache (C ABI `attn_decode_paged_fp4`)."""
    first = device, _, _, (B, _, _, d) = _first(q, "q")
    Hkv = _dims(k_codes, "k_codes", 4)[1]
    cache = _cache_fp4(k_codes, k_factors, v_codes, v_factors, k_descale, v_descale, page_table, seqlens, B, Hkv, d,
                       device)
    return _decode("attn_decode_paged_fp4", first, q, cache, Hkv, scale, workspace, out, lse, return_lse, stream)
