"""Edges of the operators around a paged cache on the GPU: what stands behind a
partial rotation, reports of two kinds at once, and values that 4 bits cannot hold."""
import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300.binding import GBATTN_EDEVICE_TIMEOUT, GBATTN_EINDEX
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _bits(t):
    return t.view({2: torch.int16, 1: torch.uint8}[t.element_size()])


def _same(a, b):
    """Equal bit for bit, but for which NaN a NaN is."""
    nan = torch.isnan(a)
    return torch.equal(nan, torch.isnan(b)) and torch.equal(_bits(a)[~nan], _bits(b)[~nan])


def _tail(x, rot):
    """x [..., d] with infinities, NaN and zeros of both signs behind element rot;
    every other row keeps its values, and every planted one a finite neighbour."""
    x = x.clone()
    for i, v in enumerate((INF, -INF, NAN, -0.0, 0.0)):
        x[..., i % 2::2, rot + 3 * i % 16] = v
    return x


PARTIAL = [(d, dtype, rot, interleaved)
           for d, dtype, rots in ((64, torch.float16, (16, 32, 48)), (128, torch.bfloat16, (16, 64, 96, 112)))
           for rot in rots for interleaved in (False, True)]


@pytest.mark.parametrize("d,dtype,rot,interleaved", PARTIAL)
def test_elements_behind_the_rotation_pass_as_they_are(d, dtype, rot, interleaved):
    """The rotation alone and its backward keep them bit for bit, and the rotated
    ones are those of rows without the infinities and NaN."""
    g = torch.Generator().manual_seed(61)
    q, k = (torch.randn(2, h, 7, d, generator=g).to(dtype) for h in (6, 2))
    rope = gb.rope_table(7, rot)
    args = dict(rope=rope, interleaved=interleaved)
    planted = [_tail(x, rot).cuda() for x in (q, k)]
    clean = [x.clone() for x in planted]
    for x in clean:
        x[..., rot:] = 1.0
    for fn in (lambda a: gb.attn_qk_norm_rope(*a, **args), lambda a: gb.attn_qk_norm_rope_bwd(*a, *a, **args)[:2]):
        for got, ref, x in zip(fn(planted), fn(clean), planted):
            assert _same(got[..., rot:], x[..., rot:])
            assert torch.equal(_bits(got[..., :rot]), _bits(ref[..., :rot]))
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("d,dtype,rot,interleaved", PARTIAL)
def test_norm_behind_the_rotation_is_the_norm_alone(d, dtype, rot, interleaved):
    """With weights, elements behind the rotation are those of the norm without a
    rotation bit for bit, zeros of both signs among them."""
    g = torch.Generator().manual_seed(62)
    q, k = (torch.randn(2, h, 7, d, generator=g).to(dtype) for h in (6, 2))
    for x in (q, k):
        x[..., ::2, rot + 1], x[..., 1::2, rot + 2] = -0.0, 0.0
    w = [1 + 0.1 * torch.randn(d, generator=g).cuda() for _ in "qk"]
    w[0][d - 1] = -w[0][d - 1]
    x = [q.cuda(), k.cuda()]
    alone = gb.attn_qk_norm_rope(*x, *w)
    turned = gb.attn_qk_norm_rope(*x, *w, rope=gb.rope_table(7, rot), interleaved=interleaved)
    for a, b in zip(alone, turned):
        assert torch.equal(_bits(a[..., rot:]), _bits(b[..., rot:]))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("d,dtype,rot,interleaved", PARTIAL)
def test_append_behind_the_rotation(bits, d, dtype, rot, interleaved):
    """Stored keys and rotated queries: 16 bits as given, 4 bits the codes of what
    was given (NaN apart: it has a test of its own)."""
    g = torch.Generator().manual_seed(63)
    S, Hkv = 9, 2
    q, k, v = (_tail(torch.randn(1, h, S, d, generator=g).to(dtype), rot) for h in (4, Hkv, Hkv))
    if bits == 4:
        k, v = (torch.where(torch.isnan(x), 1.0, x) for x in (k, v))
    rope = gb.rope_table(S, rot, device="cpu")
    k32, _ = pu.turn(k[0].float(), rope, torch.arange(S), interleaved)
    args = dict(rope=rope.cuda(), interleaved=interleaved, q=q.cuda())
    at = _i32([[1]]), _i32([S])
    if bits == 16:
        pool = [torch.zeros(2, Hkv, 16, d, dtype=dtype, device="cuda") for _ in "kv"]
        out = gb.attn_cache_append(k.cuda(), v.cuda(), *pool, *at, **args)
        for got, ref in zip(pool, (k32.to(dtype), v[0])):
            assert _same(got[1, :, :S].cpu(), ref)
    else:
        pool = [torch.zeros(2, Hkv, 16, n, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 16) * 2]
        out = gb.attn_cache_append_fp4(k.cuda(), v.cuda(), *pool, *at, **args)
        for i, ref in enumerate((k32, v[0].float())):
            codes, factors = pu.quantise(ref, 1.0)
            assert torch.equal(pool[2 * i][1, :, :S].cpu(), codes)
            assert torch.equal(pool[2 * i + 1][1, :, :S].cpu(), factors.view(torch.uint8))
    assert _same(out[..., rot:].cpu(), q[..., rot:]) and torch.isfinite(out[..., :rot]).all()
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("first", ["index", "timeout"])
def test_an_index_report_does_not_hide_a_timeout(first):
    """A position outside the table and a wait that gives up, in either order: both
    are reported, the timeout first, and then the word reads clear."""
    gb.gbattn_device_status()
    q, k = (torch.randn(1, h, 3, 64, device="cuda").half() for h in (2, 1))
    rope = gb.rope_table(3, 64)
    pos = _i32([[0, 1, 7]])
    if first == "index":
        gb.attn_qk_norm_rope(q, k, rope=rope, positions=pos)
    gb.gbattn_selftest_bounded_wait(False)
    if first == "timeout":
        gb.attn_qk_norm_rope(q, k, rope=rope, positions=pos)
    assert gb.gbattn_device_status() == GBATTN_EDEVICE_TIMEOUT
    assert gb.gbattn_device_status() == GBATTN_EINDEX
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_four_bits_of_nan(d, dtype):
    """NaN counts as the largest value, as infinity does: its group's factor is 448
    and its own code 6, whatever else the group holds and whichever lane has it; it
    reads back as 2688 descale and not as a number like its neighbours'."""
    n = d // 16
    k = torch.zeros(1, 1, 4 * 16, d, dtype=dtype)
    for i in range(16):
        for j, other in enumerate((0.0, -1.0, 60000.0, -INF)):
            group = k[0, 0, 4 * i + j].view(n, 16)[(i + j) % n]
            group[:] = other
            group[i] = -NAN if j % 2 else NAN
    descale = torch.full((1,), 0.25)
    codes = [torch.zeros(4, 1, 16, d // 2, dtype=torch.uint8, device="cuda") for _ in "kv"]
    factors = [torch.full((4, 1, 16, n), 9, dtype=torch.uint8, device="cuda") for _ in "kv"]
    table, lens = _i32([[2, 0, 3, 1]]), _i32([64])
    args = dict(k_descale=descale.cuda(), v_descale=descale.cuda())
    gb.attn_cache_append_fp4(k.cuda(), k.cuda(), codes[0], factors[0], codes[1], factors[1], table, lens, **args)
    # the formula with an infinity in each NaN's place
    ref_codes, ref_factors = pu.quantise(torch.where(torch.isnan(k[0, 0]), INF, k[0, 0].float()), 0.25)
    for c, f in zip(codes, factors):
        assert torch.equal(c[table[0].long()].flatten(0, 2).cpu(), ref_codes)
        assert torch.equal(f[table[0].long()].flatten(0, 2).cpu(), ref_factors.view(torch.uint8))
    got, _ = gb.attn_cache_gather_fp4(codes[0], factors[0], codes[1], factors[1], table, lens, 64, dtype=dtype, **args)
    nan = torch.isnan(k[0, 0])
    assert (got[0, 0].cpu()[nan] == 672.0).all() and torch.isfinite(got).all()
    groups = nan.view(64, n, 16).any(-1)
    assert (got[0, 0].cpu().view(64, n, 16)[~groups] == 0).all()


def test_four_bits_of_groups_that_round_to_nothing():
    """Groups below half of the smallest factor's reach get factor 0, and codes of 0
    with their elements' signs; they read back as zeros."""
    k = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
    k[0, 0, 1], k[0, 0, 2] = -1e-30, torch.where(torch.arange(64) % 3 == 0, -1e-6, 1e-6).bfloat16()
    k[0, 0, 3, ::2] = -0.0
    codes = [torch.full((1, 1, 16, 32), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    factors = [torch.full((1, 1, 16, 4), 9, dtype=torch.uint8, device="cuda") for _ in "kv"]
    gb.attn_cache_append_fp4(k.cuda(), k.cuda(), codes[0], factors[0], codes[1], factors[1], _i32([[0]]), _i32([4]))
    sign = torch.signbit(k[0, 0]).to(torch.uint8) * 8
    for c, f in zip(codes, factors):
        assert (f[0, 0, :4] == 0).all()
        assert torch.equal(c[0, 0, :4].cpu(), sign[:, ::2] | (sign[:, 1::2] << 4))
    got = gb.attn_cache_gather_fp4(codes[0], factors[0], codes[1], factors[1], _i32([[0]]), _i32([4]), 4)
    assert all((x == 0).all() for x in got)
