"""Python binding of the operators around a paged cache: norms and rotation of
queries and keys with their backward, append, read-back, one-query decode and
the attention of chunks of new tokens, for caches held in 16 bits and in 4.  The
definitions are those of include/gbattn.h.

As in binding.py, only arguments are marshalled here: checks of tensor metadata
(TypeError, ValueError), outputs from PyTorch's allocator, the C ABI call
(GbattnError).  That is compiled (csrc/paged_binding.cpp), because it would
otherwise take several times what a token's worth of these operators takes on
the device.  There is no fallback.

All tensors of a call lie on one device.  The call is enqueued there, on
`stream` or on that device's current stream, whichever device is current.
"""
from __future__ import annotations

import importlib.util
import os
import threading

import torch

from .binding import GbattnError, load_library

_native = None
_lock = threading.Lock()


def _load():
    """The compiled half, loaded on first use; raises if there is none for this
    Python and this PyTorch."""
    global _native
    with _lock:
        if _native is None:
            from ._build import ext_path

            load_library()
            path = ext_path()
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m exact_tiled_attention_gb300._build` (no fallback exists)")
            spec = importlib.util.spec_from_file_location(__package__ + "._paged", path)
            native = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(native)
            native.set_error(GbattnError)
            _native = native
    return _native


def rope_table(rows: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of position * base^(-2 i / rot_dim) for positions
    0 .. rows - 1, as the operators take them: fp32 [rows, rot_dim], a row's
    cosines first.  The angles are formed in 64 bits."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, device=device, dtype=torch.float64) / rot_dim)
    a = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def rope_pair_axes(sections, cycle: bool = False) -> tuple:
    """The axis of each pair of a rotation by positions of several axes, from the
    number of pairs that follow each axis: the first axis's, the next one's and so
    on, or (cycle) the axes in turn, each until its pairs are used up."""
    if not 1 <= len(sections) <= 4 or any(n < 0 for n in sections):
        raise ValueError("sections must be 1 to 4 numbers of pairs")
    if not cycle:
        return tuple(a for a, n in enumerate(sections) for _ in range(n))
    return tuple(a for i in range(max(sections)) for a, n in enumerate(sections) if i < n)


def attn_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps: float = 1e-6,
                      interleaved: bool = False, q_out=None, k_out=None, stream=None, axes=None):
    """RMS norm of every query and key head with the position rotation, through
    the C ABI `attn_qk_norm_rope`, or `attn_qk_norm_rope_axes` with axes.

    q [B,H,S,d], k [B,Hkv,S,d] fp16 or bf16 with contiguous rows (views of a
    projection output need no copy); q_weight, k_weight fp32 [d], or both None
    (rotation alone); rope fp32 [rows, rot_dim] from rope_table, or None (norm
    alone); positions int32 [B,S], or None (0 .. S-1).  With axes, the axis of
    each of the rot_dim / 2 pairs (rope_pair_axes makes them), positions is int32
    [n_axes,B,S] and a pair turns by its own axis's position.  Returns contiguous
    (q_out, k_out), which may be given as q and k themselves."""
    return (_native or _load()).attn_qk_norm_rope(q, k, q_weight, k_weight, rope, positions, eps, interleaved, q_out,
                                                  k_out, stream, axes)


def attn_qk_norm_rope_bwd_workspace_bytes(d: int) -> int:
    return int(load_library().attn_qk_norm_rope_bwd_workspace_bytes(d))


def attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope=None, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, workspace=None, dq=None, dk=None,
                          dq_weight=None, dk_weight=None, stream=None, axes=None):
    """Gradients of attn_qk_norm_rope through the C ABI `attn_qk_norm_rope_bwd`, or
    `attn_qk_norm_rope_axes_bwd` with axes.

    dq_out, dk_out: the (contiguous) gradients of its outputs; the other inputs
    as it got them.  dq and dk may be given at any strides that q and k may
    have, for instance as views of the projection output's gradient.  Returns
    (dq, dk, dq_weight, dk_weight), the last two fp32 [d], or None without
    weights."""
    return (_native or _load()).attn_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, rope, positions, eps,
                                                      interleaved, workspace, dq, dk, dq_weight, dk_weight, stream,
                                                      axes)


def attn_cache_append(k, v, k_cache, v_cache, page_table, seqlens, new_lens=None, rope=None,
                      interleaved: bool = False, q=None, q_out=None, stream=None, positions=None, axes=None):
    """Writes new keys and values into a 16-bit paged cache through the C ABI
    `attn_cache_append`, or `attn_cache_append_axes` with positions, the keys (and
    q, if given) rotated on the way.

    k, v [B,Hkv,S,d] and q [B,H,S,d] (contiguous rows, any strides);
    k_cache, v_cache [n_pages,Hkv,page_size,d]; page_table int32 [B,max_pages];
    seqlens int32 [B], the new tokens included; new_lens int32 [B] (None: S);
    rope from rope_table, or None; positions of the rotation, where they are not
    the tokens' places in their sequences: int32 [B,S], or [n_axes,B,S] with axes
    (as for attn_qk_norm_rope).  Returns the rotated queries (None without q);
    q_out may be q itself where that is contiguous."""
    return (_native or _load()).attn_cache_append(k, v, k_cache, v_cache, page_table, seqlens, new_lens, rope,
                                                  interleaved, q, q_out, stream, positions, axes)


def attn_cache_append_fp4(k, v, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, new_lens=None,
                          k_descale=None, v_descale=None, rope=None, interleaved: bool = False, q=None, q_out=None,
                          stream=None, positions=None, axes=None):
    """attn_cache_append into a 4-bit paged cache (C ABI `attn_cache_append_fp4`,
    `attn_cache_append_axes_fp4`):
    k_codes, v_codes uint8 [n_pages,Hkv,page_size,d/2]; k_factors, v_factors
    float8_e4m3fn (or both uint8) [n_pages,Hkv,page_size,d/16]; k_descale,
    v_descale fp32 [Hkv] or None."""
    return (_native or _load()).attn_cache_append_fp4(k, v, k_codes, k_factors, v_codes, v_factors, page_table,
                                                      seqlens, new_lens, k_descale, v_descale, rope, interleaved, q,
                                                      q_out, stream, positions, axes)


def attn_cache_gather(k_cache, v_cache, page_table, seqlens, S: int, k_out=None, v_out=None, stream=None):
    """The first S tokens of every sequence of a 16-bit paged cache as contiguous
    (k, v) [B,Hkv,S,d], zeros behind a sequence (C ABI `attn_cache_gather`).
    attn_fwd takes them where all sequences have S tokens: to it the zero rows
    behind a shorter one are keys."""
    return (_native or _load()).attn_cache_gather(k_cache, v_cache, page_table, seqlens, S, k_out, v_out, stream)


def attn_cache_gather_fp4(k_codes, k_factors, v_codes, v_factors, page_table, seqlens, S: int, k_descale=None,
                          v_descale=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """attn_cache_gather from a 4-bit paged cache, as fp16 or bf16 (C ABI
    `attn_cache_gather_fp4`)."""
    return (_native or _load()).attn_cache_gather_fp4(k_codes, k_factors, v_codes, v_factors, page_table, seqlens, S,
                                                      k_descale, v_descale, dtype, k_out, v_out, stream)


def attn_fwd_paged_workspace_bytes(B: int, H: int, Hkv: int, S: int, d: int, max_len: int = 2 ** 31 - 1) -> int:
    """Bytes of the paged forwards' workspace; smaller where max_len, the tokens
    that max_pages pages hold, is short."""
    return int(load_library().attn_fwd_paged_workspace_bytes(B, H, Hkv, S, d, max_len))


def attn_fwd_paged(q, k_cache, v_cache, page_table, seqlens, new_lens=None, scale: float | None = None,
                   causal: bool = True, workspace=None, out=None, lse=None, return_lse: bool = True, stream=None):
    """Attention of a chunk of new tokens over a 16-bit paged cache that holds
    them already, through the C ABI `attn_fwd_paged`.

    q [B,H,S,d] contiguous; k_cache, v_cache [n_pages,Hkv,page_size,d];
    page_table int32 [B,max_pages]; seqlens int32 [B], the new tokens included;
    new_lens int32 [B] (None: S): row i of q is the token at position
    seqlens - new_lens + i; the rows from new_lens on are padding (o = 0,
    lse = -inf).  causal: a token sees the keys up to its own, or else all of its
    sequence's.  workspace: optional buffer of attn_fwd_paged_workspace_bytes(B,
    H, Hkv, S, d) bytes (allocated here if omitted).  out and lse share memory with
    no input, the workspace or each other.  Returns (o [B,H,S,d], lse [B,H,S] or
    None)."""
    return (_native or _load()).attn_fwd_paged(q, k_cache, v_cache, page_table, seqlens, new_lens, scale, causal,
                                               workspace, out, lse, return_lse, stream)


def attn_fwd_paged_fp4(q, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, new_lens=None, k_descale=None,
                       v_descale=None, scale: float | None = None, causal: bool = True, workspace=None, out=None,
                       lse=None, return_lse: bool = True, stream=None):
    """attn_fwd_paged over a 4-bit paged cache (C ABI `attn_fwd_paged_fp4`)."""
    return (_native or _load()).attn_fwd_paged_fp4(q, k_codes, k_factors, v_codes, v_factors, page_table, seqlens,
                                                   new_lens, k_descale, v_descale, scale, causal, workspace, out, lse,
                                                   return_lse, stream)


def attn_decode_paged_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_len: int = 2 ** 31 - 1) -> int:
    """Bytes of the paged decodes' workspace; smaller where max_len, the tokens
    that max_pages pages hold, is short."""
    return int(load_library().attn_decode_paged_workspace_bytes(B, Hq, Hkv, d, max_len))


def attn_decode_paged(q, k_cache, v_cache, page_table, seqlens, scale: float | None = None, workspace=None, out=None,
                      lse=None, return_lse: bool = True, stream=None):
    """One-query decode over a 16-bit paged cache through the C ABI
    `attn_decode_paged`.

    q [B,Hq,1,d]; k_cache, v_cache [n_pages,Hkv,page_size,d]; page_table int32
    [B,max_pages]; seqlens int32 [B] (0: o = 0, lse = -inf).  workspace:
    optional buffer of attn_decode_paged_workspace_bytes(B, Hq, Hkv, d) bytes
    (allocated here if omitted).  Returns (o [B,Hq,1,d], lse [B,Hq] or None)."""
    return (_native or _load()).attn_decode_paged(q, k_cache, v_cache, page_table, seqlens, scale, workspace, out,
                                                  lse, return_lse, stream)


def attn_decode_paged_fp4(q, k_codes, k_factors, v_codes, v_factors, page_table, seqlens, k_descale=None,
                          v_descale=None, scale: float | None = None, workspace=None, out=None, lse=None,
                          return_lse: bool = True, stream=None):
    """attn_decode_paged over a 4-bit paged cache (C ABI `attn_decode_paged_fp4`)."""
    return (_native or _load()).attn_decode_paged_fp4(q, k_codes, k_factors, v_codes, v_factors, page_table, seqlens,
                                                      k_descale, v_descale, scale, workspace, out, lse, return_lse,
                                                      stream)
