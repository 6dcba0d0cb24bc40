"""The operators around a paged cache without a GPU: every refusal of the C ABI
and of the Python wrappers, the workspace sizes, the rotation table, and the
plain forms that the GPU tests compare with (their gradients against
differences, their 4-bit rounding against every midpoint)."""
import ctypes

import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300 import _build, binding
from tests import paged_util as pu

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation rejects first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return binding.load_library()


def _call(fn, defaults, order, kw):
    a = dict(defaults, **kw)
    assert set(kw) <= set(defaults)
    return fn(*[a[n] for n in order.split()])


NORM = dict(q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, rope=FAKE, pos=FAKE, qo=FAKE, ko=FAKE, B=2, H=4, Hkv=2, S=8, d=64,
            qs=None, ks=None, eps=1e-6, rows=8, rot=64, inter=0, dtype=1, stream=None)
NORM_ORDER = "q k qw kw rope pos qo ko B H Hkv S d qs ks eps rows rot inter dtype stream"


def _strides(*s):
    return (ctypes.c_longlong * 3)(*s)


def _norm(lib, **kw):
    return _call(lib.attn_qk_norm_rope, NORM, NORM_ORDER, kw)


def test_norm_rope_refusals(lib):
    for name in ("B", "H", "Hkv", "S"):
        assert _norm(lib, **{name: 0}) == -1
    assert _norm(lib, H=16386) == -1
    assert _norm(lib, B=1 << 15, S=(1 << 15) + 1, rows=1 << 16) == -1  # more tokens than 2^30
    assert _norm(lib, H=5) == -2
    for d in (0, 32, 96, 256):
        assert _norm(lib, d=d) == -3
    assert _norm(lib, dtype=2) == -4
    for name in ("q", "k", "qo", "ko", "rope"):
        assert _norm(lib, **{name: None}) == -5
        assert _norm(lib, **{name: FAKE + 8}) == -5
    assert _norm(lib, qw=None) == -5 and _norm(lib, kw=None) == -5  # one weight without the other
    assert _norm(lib, qw=None, kw=None, rot=0, rope=None) == -5     # nothing to do
    assert _norm(lib, qw=FAKE + 4) == -5
    assert _norm(lib, pos=FAKE + 2) == -5
    assert _norm(lib, qs=_strides(512, 64, 60)) == -5
    assert _norm(lib, ks=_strides(514, 64, 64)) == -5
    for rot in (-16, 8, 24, 80):
        assert _norm(lib, rot=rot) == -11
    assert _norm(lib, rows=0) == -1
    assert _norm(lib, pos=None, rows=7) == -1  # token 7 has no row
    if not torch.cuda.is_available():
        assert _norm(lib) == -10
        assert _norm(lib, qw=None, kw=None) == -10
        assert _norm(lib, rot=0, rope=None, rows=0, pos=None) == -10
        assert _norm(lib, qs=_strides(512, 64, 128)) == -10


NORM_BWD = dict(NORM, dqo=FAKE, dko=FAKE, dq=FAKE, dk=FAKE, dqw=FAKE, dkw=FAKE, dqs=None, dks=None, ws=FAKE,
                wsb=1 << 20)
NORM_BWD_ORDER = ("dqo dko q k qw kw rope pos dq dk dqw dkw B H Hkv S d qs ks dqs dks eps rows rot inter ws wsb dtype "
                  "stream")


def _norm_bwd(lib, **kw):
    return _call(lib.attn_qk_norm_rope_bwd, NORM_BWD, NORM_BWD_ORDER, kw)


def test_norm_rope_bwd_refusals(lib):
    need = lib.attn_qk_norm_rope_bwd_workspace_bytes(64)
    assert need == 2 * 1024 * 64 * 4 and lib.attn_qk_norm_rope_bwd_workspace_bytes(80) == 0
    assert _norm_bwd(lib, S=0) == -1 and _norm_bwd(lib, H=3) == -2 and _norm_bwd(lib, d=100) == -3
    assert _norm_bwd(lib, dtype=-1) == -4
    for name in ("dqo", "dko", "q", "k", "dq", "dk", "dqw", "dkw", "ws"):
        assert _norm_bwd(lib, **{name: None}) == -5, name
    for name in ("dqo", "dko", "dq", "dk", "ws"):
        assert _norm_bwd(lib, **{name: FAKE + 8}) == -5, name
    assert _norm_bwd(lib, dqs=_strides(4, 8, 8)) == -5
    assert _norm_bwd(lib, wsb=need - 1) == -6
    assert _norm_bwd(lib, rot=72) == -11
    if not torch.cuda.is_available():
        assert _norm_bwd(lib, wsb=need) == -10
        assert _norm_bwd(lib, qw=None, kw=None, dqw=None, dkw=None, ws=None, wsb=0) == -10


CACHE = dict(kc=FAKE, kf=FAKE, vc=FAKE, vf=FAKE, kd=None, vd=None, table=FAKE, lens=FAKE, page=16, n=4, width=2)
APPEND = dict(CACHE, k=FAKE, v=FAKE, new=None, rope=FAKE, q=FAKE, qo=FAKE, B=2, H=4, Hkv=2, S=3, d=128, qs=None,
              ks=None, vs=None, rows=40, rot=128, inter=0, dtype=0, stream=None)
GATHER = dict(CACHE, ko=FAKE, vo=FAKE, B=2, Hkv=2, S=20, d=128, dtype=0, stream=None)
DECODE = dict(CACHE, q=FAKE, o=FAKE, lse=None, B=2, Hq=4, Hkv=2, d=128, scale=0.1, ws=FAKE, wsb=1 << 26, dtype=0,
              stream=None)
TAIL = {
    "attn_cache_append": "new rope q qo B H Hkv S d page n width qs ks vs rows rot inter dtype stream",
    "attn_cache_gather": "ko vo B Hkv S d page n width dtype stream",
    "attn_decode_paged": "o lse B Hq Hkv d page n width scale ws wsb dtype stream",
}
HEAD = {"attn_cache_append": "k v ", "attn_cache_gather": "", "attn_decode_paged": "q "}
DEFAULTS = {"attn_cache_append": APPEND, "attn_cache_gather": GATHER, "attn_decode_paged": DECODE}


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("name", sorted(TAIL))
def test_cache_refusals(lib, name, fp4):
    pool = "kc kf vc vf kd vd table lens " if fp4 else "kc vc table lens "
    fn = getattr(lib, name + ("_fp4" if fp4 else ""))

    def call(**kw):
        return _call(fn, DEFAULTS[name], HEAD[name] + pool + TAIL[name], kw)

    for field in ("B", "Hkv", "n", "width") + (("S",) if "S" in DEFAULTS[name] else ()):
        assert call(**{field: 0}) == -1, field
    assert call(width=1 << 27, page=16) == -1  # more slots than an int counts
    assert call(n=1 << 30, page=64) == -1      # more blocks of 16 slots
    assert call(d=96) == -3 and call(d=256) == -3
    assert call(dtype=5) == -4
    for page in (0, 8, 24, 48, 2048):
        assert call(page=page) == -11, page
    required = {"kc", "vc", "table", "lens"} | ({"kf", "vf"} if fp4 else set())
    required |= {"attn_cache_append": {"k", "v"}, "attn_cache_gather": {"ko", "vo"},
                 "attn_decode_paged": {"q", "o", "ws"}}[name]
    for field in required:
        assert call(**{field: None}) == -5, field
        assert call(**{field: FAKE + 2}) == -5, field
    if fp4:
        assert call(kd=FAKE + 1) == -5
    if name == "attn_cache_append":
        assert call(H=5) == -2 and call(H=16386) == -1 and call(B=1 << 15, S=1 << 16) == -1
        assert call(q=None) == -5 and call(qo=None) == -5  # one without the other
        assert call(rope=None) == -5 and call(rows=0) == -1 and call(rot=20) == -11
        assert call(new=FAKE + 1) == -5
        for s in ("qs", "ks", "vs"):
            assert call(**{s: _strides(8, 16, 4)}) == -5
    if name == "attn_cache_gather":
        assert call(B=1 << 15, Hkv=2) == -1 and call(S=(1 << 30) + 1) == -1
    if name == "attn_decode_paged":
        assert call(Hq=5) == -2 and call(B=65536) == -1
        need = lib.attn_decode_paged_workspace_bytes(2, 4, 2, 128, 32)
        assert call(wsb=need - 1) == -6
        assert call(lse=FAKE + 2) == -5
    if not torch.cuda.is_available():
        assert call() == -10
        if name == "attn_cache_append":
            assert call(q=None, qo=None, rope=None, rot=0, rows=0) == -10


def test_decode_workspace(lib):
    """States for the most CTAs that can have work, whatever the lengths are."""
    size = lib.attn_decode_paged_workspace_bytes
    one = size(1, 32, 8, 128, 1 << 20)
    assert one == 1024 * 2 * 4 * 130 * 4 + 8 * 8
    assert size(64, 32, 8, 128, (1 << 31) - 1) == one + 63 * 64
    assert size(1, 32, 1, 64, 1 << 20) == 1024 * 2 * 16 * 66 * 4 + 2 * 8
    assert size(1, 32, 8, 128, 1000) == 8 * 16 * 2 * 4 * 130 * 4 + 8 * 8
    assert size(1, 5, 2, 64, 64) == 0 and size(1, 4, 2, 64, 0) == 0


def test_status_words(lib):
    assert b"page" in lib.gbattn_error_string(-11) and b"outside" in lib.gbattn_error_string(-12)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the wrappers' checks before any device is needed")
def test_wrappers_refuse_cpu_tensors_and_wrong_arguments():
    q, k = torch.zeros(1, 2, 3, 64, dtype=torch.float16), torch.zeros(1, 1, 3, 64, dtype=torch.float16)
    pool = torch.zeros(2, 1, 16, 64, dtype=torch.float16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    rope = gb.rope_table(4, 64, device="cpu")
    with pytest.raises(ValueError, match="no CPU path"):
        gb.attn_qk_norm_rope(q, k, rope=rope)
    with pytest.raises(ValueError, match="no CPU path"):
        gb.attn_cache_append(k, k, pool, pool, table, lens)
    with pytest.raises(ValueError, match="no CPU path"):
        gb.attn_decode_paged(q[:, :, :1], pool, pool, table, lens)
    with pytest.raises(ValueError, match="no CPU path"):
        gb.attn_cache_gather(pool, pool, table, lens, 3)
    with pytest.raises(TypeError):
        gb.attn_decode_paged([1.0], pool, pool, table, lens)
    with pytest.raises(ValueError):
        gb.attn_decode_paged(q, pool[0], pool, table, lens)


def test_rope_table():
    t = gb.rope_table(40000, 64, base=1e6, device="cpu")
    a = torch.tensor(39999.0, dtype=torch.float64) * 1e6 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert torch.equal(t[39999, :32], a.cos().float()) and torch.equal(t[39999, 32:], a.sin().float())
    assert torch.equal(t[0], torch.cat([torch.ones(32), torch.zeros(32)]))
    for bad in (0, 3, -2):
        with pytest.raises(ValueError):
            gb.rope_table(4, bad, device="cpu")


@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (32, False), (32, True), (64, True)])
def test_plain_gradients_against_differences(rot, interleaved):
    """The formula of the backward against central differences of the forward in
    64 bits: the error of a difference is h^2 / 6 of the third derivative, a few
    hundred for these sizes, plus 2^-53 |f| / h."""
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(2, 5, 64, generator=g, dtype=torch.float64), torch.rand(64, generator=g, dtype=torch.float64) + 0.5
    dy = torch.randn(2, 5, 64, generator=g, dtype=torch.float64)
    table = gb.rope_table(9, rot, device="cpu") if rot else None
    pos = torch.tensor([8, 0, 3, 3, 1])

    def f(x, w):
        return (pu.norm_rope(x, w, table, pos, 1e-6, interleaved)[0] * dy).sum()

    dx, dw, _, _ = pu.norm_rope_bwd(dy, x, w, table, pos, 1e-6, interleaved)
    h = 1e-5
    for _ in range(8):
        e, ew = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64)
        slope = (f(x + h * e, w + h * ew) - f(x - h * e, w - h * ew)) / (2 * h)
        assert abs(slope - (dx * e).sum() - (dw * ew).sum()) <= 1e-6


def test_plain_four_bit_rounding():
    """Every midpoint of the eight magnitudes goes to the even code, and every
    value next to one to its own side."""
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    x = torch.zeros(16)
    for i in range(7):
        mid = (mags[i] + mags[i + 1]) / 2
        even = i if i % 2 == 0 else i + 1
        for v, code in ((mid, even), (mid * (1 - 2 ** -23), i), (mid * (1 + 2 ** -22), i + 1)):
            for sign in (1.0, -1.0):
                x[0], x[1] = 6.0, sign * v  # factor 1
                codes, f = pu.quantise(x, 1.0)
                assert f.float().item() == 1.0
                assert codes[0].item() == 7 | ((code + (8 if sign < 0 else 0)) << 4)
    assert pu.quantise(torch.zeros(16), 1.0)[1].float().item() == 0.0
    assert pu.quantise(torch.full((16,), 1e9), 1.0)[1].float().item() == 448.0
