"""The chunk's attention over a paged cache and the rotation by several axes
without a GPU: every refusal of the C ABI, workspace sizes, the pairs' axes, and the
plain form that the GPU tests compare with."""
import ctypes

import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300 import _build, binding
from tests import chunk_util as cu
from tests import paged_util as pu
from tests.test_paged_abi import APPEND, CACHE, FAKE, NORM, NORM_BWD, _call, _strides


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load_library()


FORWARD = dict(CACHE, q=FAKE, new=FAKE, o=FAKE, lse=None, B=2, H=4, Hkv=2, S=3, d=128, scale=0.1, causal=1, ws=FAKE,
               wsb=1 << 30, dtype=0, stream=None)


@pytest.mark.parametrize("fp4", [False, True])
def test_forward_refusals(lib, fp4):
    pool = "kc kf vc vf kd vd table lens " if fp4 else "kc vc table lens "
    order = "q " + pool + "new o lse B H Hkv S d page n width scale causal ws wsb dtype stream"
    fn = lib.attn_fwd_paged_fp4 if fp4 else lib.attn_fwd_paged

    def call(**kw):
        return _call(fn, FORWARD, order, kw)

    for field in ("B", "H", "Hkv", "S", "n", "width"):
        assert call(**{field: 0}) == -1, field
        assert call(**{field: -1}) == -1, field
    assert call(H=5) == -2 and call(H=16386) == -1
    assert call(B=1 << 15, S=1 << 16) == -1
    assert call(width=1 << 27) == -1 and call(n=1 << 30, page=64) == -1
    assert call(n=1 << 30, Hkv=2) == -1  # a page and head is one coordinate
    assert call(d=96) == -3 and call(d=256) == -3
    assert call(dtype=5) == -4
    for scale in (float("nan"), float("inf"), float("-inf")):
        assert call(scale=scale) == -1
    for page in (0, 8, 24, 48, 2048):
        assert call(page=page) == -11, page
    for field in ["q", "o", "ws", "kc", "vc", "table", "lens"] + (["kf", "vf"] if fp4 else []):
        assert call(**{field: None}) == -5, field
        assert call(**{field: FAKE + 2}) == -5, field
    assert call(new=FAKE + 2) == -5 and call(lse=FAKE + 2) == -5
    need = lib.attn_fwd_paged_workspace_bytes(2, 4, 2, 3, 128, 32)
    assert call(wsb=need - 1) == -6
    if not torch.cuda.is_available():
        assert call(wsb=need) == -10 and call(new=None) == -10 and call(scale=-0.5) == -10


def test_forward_workspace(lib):
    """States of one or two tiles of 128 rows, whichever takes more, for the most CTAs that can have work."""
    size = lib.attn_fwd_paged_workspace_bytes
    one, two = 2 * 128 * 130 * 4, 2 * 256 * 130 * 4
    assert size(1, 32, 8, 16, 128, 1000) == 64 * one + 8 * 8      # 8 units of 8 tiles
    assert size(1, 32, 8, 32, 128, 1 << 20) == 160 * one + 8 * 8  # 128 rows: one tile
    assert size(1, 32, 8, 33, 128, 1 << 20) == 160 * two + 8 * 8
    assert size(4, 32, 8, 2048, 128, 16384) == 160 * two + 4 * 8 * 32 * 8
    # two blocks of 65 heads, a token a tile: 4 units of one tile (more than 2 of two), whichever are taken
    assert size(1, 130, 1, 2, 64, 64) == 4 * (2 * 128 * 66 * 4) + 4 * 8
    assert size(1, 5, 2, 4, 64, 64) == 0 and size(1, 4, 2, 0, 64, 64) == 0 and size(1, 4, 2, 4, 64, 0) == 0


AXES = ctypes.create_string_buffer(bytes([0, 1, 2, 2] * 16), 64)
AXES_CALLS = {
    "attn_qk_norm_rope_axes":
        (NORM, "q k qw kw rope pos axes qo ko B H Hkv S d n_axes qs ks eps rows rot inter dtype stream"),
    "attn_qk_norm_rope_axes_bwd":
        (NORM_BWD, "dqo dko q k qw kw rope pos axes dq dk dqw dkw B H Hkv S d n_axes qs ks dqs dks eps rows rot inter "
                   "ws wsb dtype stream"),
    "attn_cache_append_axes":
        (APPEND, "k v kc vc table lens new rope pos axes q qo B H Hkv S d n_axes page n width qs ks vs rows rot inter "
                 "dtype stream"),
    "attn_cache_append_axes_fp4":
        (APPEND, "k v kc kf vc vf kd vd table lens new rope pos axes q qo B H Hkv S d n_axes page n width qs ks vs "
                 "rows rot inter dtype stream"),
}


@pytest.mark.parametrize("name", sorted(AXES_CALLS))
def test_axes_refusals(lib, name):
    base, order = AXES_CALLS[name]
    defaults = dict(base, pos=FAKE, axes=AXES, n_axes=3)

    def call(**kw):
        return _call(getattr(lib, name), defaults, order, kw)

    assert call(n_axes=0) == -1 and call(n_axes=5) == -1 and call(n_axes=-1) == -1
    assert call(n_axes=2) == -1  # an entry of the pairs' axes is 2
    assert call(pos=None) == -5 and call(pos=FAKE + 2) == -5 and call(axes=None) == -5
    assert call(rope=None) == -5
    assert call(rot=0, rope=None, rows=0) == -5  # no rotation
    assert call(rot=24) == -11
    # the refusals of the forms without axes
    assert call(H=5) == -2 and call(d=96) == -3 and call(dtype=5) == -4 and call(S=0) == -1
    assert call(qs=_strides(8, 16, 4)) == -5
    if not torch.cuda.is_available():
        assert call() == -10 and call(n_axes=4) == -10


def test_pair_axes():
    assert gb.rope_pair_axes((2, 1, 3)) == (0, 0, 1, 2, 2, 2)
    assert gb.rope_pair_axes((2, 1, 3), cycle=True) == (0, 1, 2, 0, 2, 2)
    assert gb.rope_pair_axes([3]) == (0, 0, 0)
    for bad in ((), (1, 2, 3, 4, 5), (1, -1)):
        with pytest.raises(ValueError):
            gb.rope_pair_axes(bad)


def test_plain_form_against_single_queries():
    """The chunk's plain form is paged_util's decode, query by query."""
    g = torch.Generator().manual_seed(1)
    H, Hkv, n, m, d = 4, 2, 37, 9, 16
    q, k, v = torch.randn(H, m, d, generator=g), torch.randn(Hkv, n, d, generator=g), torch.randn(Hkv, n, d, generator=g)
    for causal in (True, False):
        lim = cu.limits(n, m, causal)
        o, lse, _, _ = cu.attention(q, k, v, lim, 0.25, 0.0)
        for i in range(m):
            seen = n - m + i + 1 if causal else n
            ro, rl, _, _ = pu.attention(q[:, i], k[:, :seen], v[:, :seen], 0.25, 0.0)
            assert torch.allclose(o[:, i], ro, atol=1e-12) and torch.allclose(lse[:, i], rl, atol=1e-12)
    assert cu.limits(3, 5, True).tolist() == [-1, -1, 0, 1, 2] and cu.limits(3, 5, False).tolist() == [-1, -1, 2, 2, 2]


@pytest.mark.parametrize("fp4", [False, True])
def test_forward_refuses_scales_that_log2_e_takes_out_of_fp32(lib, fp4):
    pool = "kc kf vc vf kd vd table lens " if fp4 else "kc vc table lens "
    order = "q " + pool + "new o lse B H Hkv S d page n width scale causal ws wsb dtype stream"
    fn = lib.attn_fwd_paged_fp4 if fp4 else lib.attn_fwd_paged
    for scale in (2.4e38, -2.4e38, 3e38):
        assert _call(fn, FORWARD, order, dict(scale=scale)) == -1, scale
    if not torch.cuda.is_available():
        for scale in (2.29e38, -2.29e38, 1e-45, 0.0):
            assert _call(fn, FORWARD, order, dict(scale=scale)) == -10, scale
