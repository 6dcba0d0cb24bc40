"""Attention of a chunk of new tokens over a paged cache on the GPU, against its
plain form in 64 bits (bounds in chunk_util)."""
import math

import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300.binding import GBATTN_EINDEX
from tests import chunk_util as cu
from tests import paged_util as pu
from tests.test_paged_gpu import Pool, _i32, _same_bits

pytestmark = pytest.mark.gpu


beyond = 0  # columns that _forward adds to a page table


@pytest.fixture(params=["narrow", "wide"])
def table_width(request, monkeypatch):
    """What a page table could hold decides how the work is divided and which kernels
    take it: tables as the test makes them, and the same ones with room for far more."""
    if request.param == "wide":
        monkeypatch.setitem(globals(), "beyond", 20000)


def _forward(pool, q, table, lens, news, **kw):
    if beyond:
        table = torch.nn.functional.pad(table, (0, beyond), value=1 << 30)
    fn = gb.attn_fwd_paged if pool.bits == 16 else gb.attn_fwd_paged_fp4
    return fn(q, *pool.gpu, table.cuda(), _i32(lens), new_lens=None if news is None else _i32(news), **pool.kw, **kw)


def _make(bits, dtype, Hkv, d, page, lens, seed, spare=2, nan=False):
    g = torch.Generator().manual_seed(seed)
    width = max(1, (max(lens) + page - 1) // page) + 1
    n_pages = sum((n + page - 1) // page for n in lens) + spare
    pool = Pool(bits, n_pages, Hkv, page, d, dtype, g, nan=nan)
    return pool, pu.page_table(lens, page, n_pages, width, g, beyond=1 << 30), g


def _ok(pool, q, table, lens, news, o, lse, causal, scale):
    half_p = pu.u(torch.float16) if pool.bits == 4 else pu.u(pool.dtype)
    cu.check(o, lse, q, lambda b, n: (pool.values(0, table[b], n), pool.values(1, table[b], n)), lens, news, causal,
             scale, half_p, 2.0 ** -24 if pool.bits == 4 else 0.0,
             pool.bits == 4 or pool.dtype is torch.float16, pu.u(q.dtype))


CHUNKS = [
    # dtype, H, Hkv, d, page, S, lens, new (None: S each)
    (torch.bfloat16, 1, 1, 128, 16, 1, [1], None),
    (torch.bfloat16, 8, 2, 128, 64, 16, [16, 77, 300], None),
    (torch.float16, 6, 2, 64, 16, 33, [33, 40, 0, 700, 15], [33, 1, 0, 32, 15]),
    (torch.bfloat16, 9, 1, 128, 32, 5, [127, 128, 129, 5], [5, 4, 5, 2]),
    (torch.float16, 16, 1, 128, 128, 40, [1000, 0, 999, 41], [40, 0, 0, 39]),
    (torch.bfloat16, 4, 4, 64, 256, 300, [300, 513, 1000], [300, 257, 128]),
    (torch.bfloat16, 32, 8, 128, 64, 70, [200, 2000], None),
    (torch.float16, 5, 5, 128, 1024, 129, [129, 1153], None),
    (torch.bfloat16, 130, 1, 64, 16, 3, [100, 3], None),
    (torch.bfloat16, 7, 1, 64, 64, 260, [260, 300, 261], [260, 19, 200]),
    (torch.float16, 2, 1, 128, 16, 20, [5, 12, 20], None),  # rows before the sequence's start are padding
    (torch.bfloat16, 2, 2, 64, 16, 4, [0, 0], None),
    (torch.bfloat16, 4, 2, 128, 64, 3, [20000], None),
    # more units of one row tile than SMs, of two not: a CTA for each
    (torch.bfloat16, 8, 8, 128, 64, 200, [200, 300, 129, 0, 500, 257, 256, 131, 420, 100], [200, 200, 1, 0, 130, 200, 128, 131, 199, 100]),
    (torch.float16, 16, 8, 64, 16, 100, [100, 300, 65, 0, 500, 257, 256, 131, 420, 64], [100, 100, 1, 0, 65, 100, 64, 99, 100, 64]),
    # few units of one row tile, of one or several CTAs each; rows before the sequence's start
    (torch.bfloat16, 7, 1, 128, 32, 130, [100, 700, 130], None),
    (torch.float16, 12, 4, 64, 128, 300, [300, 1200], None),
]


# More key tiles than CTAs, so that each CTA works through several units, whole
# and split ones, in both block sizes.
LONG = [
    # dtype, H, Hkv, d, page, S
    (torch.bfloat16, 8, 4, 128, 64, 3),
    (torch.float16, 4, 2, 64, 16, 9),
    (torch.bfloat16, 8, 4, 128, 128, 90),
    (torch.float16, 8, 4, 64, 32, 100),
]


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cfg", CHUNKS)
def test_chunk(cfg, causal, bits):
    dtype, H, Hkv, d, page, S, lens, news = cfg
    pool, table, g = _make(bits, dtype, Hkv, d, page, lens, 31)
    q = torch.randn(len(lens), H, S, d, generator=g).to(dtype).cuda()
    scale = 1 / math.sqrt(d)
    o, lse = _forward(pool, q, table, lens, news, causal=causal)
    assert gb.gbattn_device_status() == 0
    _ok(pool, q, table, lens, news or [S] * len(lens), o, lse, causal, scale)
    again = _forward(pool, q, table, lens, news, causal=causal)
    assert _same_bits(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cfg", LONG)
def test_runs_of_several_units(cfg, bits):
    dtype, H, Hkv, d, page, S = cfg
    g = torch.Generator().manual_seed(32)
    lens = torch.randint(100, 1500, (36,), generator=g).tolist()
    lens[7], lens[20], lens[21] = 0, 3, 6000
    news = [min(n, int(m)) for n, m in zip(lens, torch.randint(0, S + 1, (36,), generator=g))]
    pool, table, g = _make(bits, dtype, Hkv, d, page, lens, 33)
    q = torch.randn(len(lens), H, S, d, generator=g).to(dtype).cuda()
    o, lse = _forward(pool, q, table, lens, news)
    assert gb.gbattn_device_status() == 0
    _ok(pool, q, table, lens, news, o, lse, True, 1 / math.sqrt(d))
    for _ in range(5):
        again = _forward(pool, q, table, lens, news)
        assert gb.gbattn_device_status() == 0
        assert _same_bits(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("bits", [16, 4])
def test_units_of_one_row_tile_in_runs(bits):
    """More units of one row tile than clusters take, and so many key tiles that they are
    cut into runs: 104 units of 33 to 36 tiles."""
    lens, S, d = [4500], 400, 64
    pool, table, g = _make(bits, torch.bfloat16, 8, d, 64, lens, 42)
    q = torch.randn(1, 32, S, d, generator=g).bfloat16().cuda()
    o, lse = _forward(pool, q, table, lens, None)
    assert gb.gbattn_device_status() == 0
    _ok(pool, q, table, lens, [S], o, lse, True, 1 / math.sqrt(d))
    again = _forward(pool, q, table, lens, None)
    assert _same_bits(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [1, 30, 90])
@pytest.mark.parametrize("bits", [16, 4])
def test_slots_behind_the_length_and_unused_pages_hold_nan(bits, S):
    lens, page, H, Hkv, d = [1, 333, 130, 700], 64, 8, 2, 128
    news = [1, min(S, 333), S, S]
    pool, table, g = _make(bits, torch.bfloat16, Hkv, d, page, lens, 34, spare=9)
    q = torch.randn(4, H, S, d, generator=g).bfloat16().cuda()
    o, lse = _forward(pool, q, table, lens, news)
    dirty, _, _ = _make(bits, torch.bfloat16, Hkv, d, page, lens, 34, spare=9, nan=True)
    for t, src in zip(dirty.gpu, pool.gpu):
        t, src = (x.view(torch.uint8) if x.element_size() == 1 else x for x in (t, src))
        for b, n in enumerate(lens):
            for i in range((n + page - 1) // page):
                rows = min(page, n - i * page)
                t[table[b, i], :, :rows] = src[table[b, i], :, :rows]
    dirty.kw = pool.kw
    for causal in (True, False):
        o, lse = _forward(pool, q, table, lens, news, causal=causal)
        o2, lse2 = _forward(dirty, q, table, lens, news, causal=causal)
        assert torch.isfinite(o2).all() and _same_bits(o, o2) and torch.equal(lse, lse2)


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("dtype,H,Hkv,d,S,L", [
    (torch.bfloat16, 4, 2, 128, 9, 150), (torch.float16, 8, 1, 64, 20, 500), (torch.bfloat16, 2, 2, 128, 200, 350),
    (torch.float16, 4, 1, 64, 100, 130), (torch.bfloat16, 2, 1, 128, 300, 300), (torch.bfloat16, 1, 1, 64, 256, 1000)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite(dtype, H, Hkv, d, S, L, value):
    """A NaN or an infinity in a token's v reaches the tokens that see it, in its
    element, and nothing else; in its k, the tokens that see it alone."""
    page = 16
    pool, table, g = _make(16, dtype, Hkv, d, page, [L, L], 35)
    q = torch.randn(2, H, S, d, generator=g).to(dtype).cuda()
    clean = _forward(pool, q, table, [L, L], None)
    at = [L - S + t for t in sorted({0, 1, S // 2, S - 1})] + [L - S - 1] * (L > S)
    # a token and an element each, the same element twice
    el = [(7 * i) % d for i in range(len(at))]
    el[-1] = el[0]
    for p, e in zip(at, el):
        pool.gpu[1][table[0, p // page], :, p % page, e] = value
    o, lse = _forward(pool, q, table, [L, L], None)
    assert gb.gbattn_device_status() == 0
    bad = torch.zeros(S, d, dtype=torch.bool, device="cuda")
    for p, e in zip(at, el):
        bad[max(0, p - (L - S)):, e] = True
    assert torch.equal(torch.isnan(o[0]) | torch.isinf(o[0]), bad.expand(H, S, d))
    assert _same_bits(torch.where(bad, 0.0, o[0].float()).to(dtype), torch.where(bad, 0.0, clean[0][0].float()).to(dtype))
    assert _same_bits(o[1], clean[0][1]) and torch.equal(lse, clean[1])
    if math.isnan(value):
        t0 = S // 2
        pool.gpu[0][table[1, (L - S + t0) // page], :, (L - S + t0) % page, 3] = value
        o, lse = _forward(pool, q, table, [L, L], None)
        assert torch.isnan(o[1, :, t0:]).all() and torch.isnan(lse[1, :, t0:]).all()
        assert _same_bits(o[1, :, :t0].contiguous(), clean[0][1, :, :t0].contiguous())
        assert torch.equal(lse[1, :, :t0], clean[1][1, :, :t0])


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("dtype,H,Hkv,d,S,L", [
    (torch.bfloat16, 8, 2, 64, 3, 700), (torch.float16, 4, 2, 64, 12, 900), (torch.bfloat16, 4, 2, 128, 9, 900),
    (torch.float16, 2, 2, 128, 200, 700), (torch.bfloat16, 1, 1, 64, 256, 1000), (torch.float16, 40, 8, 128, 300, 9000)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_give_nan(dtype, H, Hkv, d, S, L, value):
    """However the work is divided: a value in the first, a middle and the last tile
    before the chunk and in the chunk, with a weight that counts or (a key against the
    queries, at a scale that makes it so) one that is 0 in fp32."""
    page = 64
    pool, table, g = _make(16, dtype, Hkv, d, page, [L, L], 46)
    pool.gpu[0][table[1, 1], :, 3] = -4.0
    q = (0.5 + torch.rand(2, H, S, d, generator=g)).to(dtype).cuda()
    clean = _forward(pool, q, table, [L, L], None, scale=1.0)
    at = [(0, 2), (0, L // 2), (0, L - S - 1), (0, L - S), (0, L - S // 2 - 1), (1, page + 3)]
    bad = torch.zeros(2, 1, S, d, dtype=torch.bool)
    for i, (b, p) in enumerate(at):
        pool.gpu[1][table[b, p // page], :, p % page, 9 * i + 1] = value
        bad[b, :, max(0, p - (L - S)):, 9 * i + 1] = True
    bad = bad.cuda()
    o, lse = _forward(pool, q, table, [L, L], None, scale=1.0)
    assert gb.gbattn_device_status() == 0
    assert torch.equal(torch.isnan(o), bad.expand_as(o)) and torch.isfinite(lse).all()
    assert _same_bits(o.masked_fill(bad, 0.0), clean[0].masked_fill(bad, 0.0)) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("d", [64, 128])
def test_notes_of_many_short_segments(d):
    """Units of two row tiles of which the second is empty in all but a few: many
    segments for each CTA, where only one of the row tiles' warps meets the keys.  A NaN
    in v of one token of each sequence, another element each, and in every slot behind
    it."""
    page, Hkv, S, B = 64, 4, 200, 300
    g = torch.Generator().manual_seed(43)
    news = [int(m) for m in torch.randint(1, 129, (B,), generator=g)]
    for b in range(0, B, 7):
        news[b] = 129 + b % 72  # the second row tile has rows
    lens = [m + int(n) for m, n in zip(news, torch.randint(0, 120, (B,), generator=g))]
    pool, table, g = _make(16, torch.bfloat16, Hkv, d, page, lens, 44)
    q = torch.randn(B, Hkv, S, d, generator=g).bfloat16().cuda()
    clean = _forward(pool, q, table, lens, news)
    assert gb.gbattn_device_status() == 0
    bad = torch.zeros(B, 1, S, d, dtype=torch.bool)
    for b, (n, m) in enumerate(zip(lens, news)):
        last = int(table[b, (n - 1) // page])
        pool.gpu[1][last, :, (n - 1) % page + 1:] = float("nan")
        t, e = (5 * b) % m, (11 * b) % d
        pool.gpu[1][int(table[b, (n - m + t) // page]), :, (n - m + t) % page, e] = float("nan")
        bad[b, 0, t:m, e] = True
    bad = bad.cuda()
    for _ in range(20):
        o, lse = _forward(pool, q, table, lens, news)
        assert gb.gbattn_device_status() == 0 and torch.equal(lse, clean[1])
        assert torch.equal(torch.isnan(o), bad.expand_as(o))
        assert _same_bits(o.masked_fill(bad, 0.0), clean[0].masked_fill(bad, 0.0))


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [1, 20, 70])
@pytest.mark.parametrize("bits", [16, 4])
def test_pages_that_do_not_exist(bits, S):
    """A page outside the pool is left out, and reported; a sequence without any
    counts no key."""
    lens, page, H, Hkv, d = [300, 80], 16, 4, 2, 64
    pool, table, g = _make(bits, torch.float16, Hkv, d, page, lens, 36)
    n_pages = pool.gpu[0].shape[0]
    q = torch.randn(2, H, S, d, generator=g).half().cuda()
    gb.gbattn_device_status()
    for bad in (-1, n_pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2], t[0, 18] = bad, bad  # slots 32 .. 47 and 288 .. 299, the last ones
        o, lse = _forward(pool, q, t, lens, None, causal=False)
        assert gb.gbattn_device_status() == GBATTN_EINDEX and gb.gbattn_device_status() == 0
        keep = [i for i in range(300) if i // page not in (2, 18)]
        k, v = (pool.values(i, table[0], 300)[:, keep] for i in range(2))
        half_p = pu.u(torch.float16)
        ro, rl, to, tl = cu.attention(q[0].cpu(), k, v, torch.full((S,), len(keep) - 1), 0.125, half_p, 2.0 ** -24, True)
        assert ((o[0].double().cpu() - ro).abs() <= to + half_p * (ro.abs() + to) + 2.0 ** -25).all()
        assert ((lse[0].double().cpu() - rl).abs() <= tl).all()
        t[1] = bad
        o, lse = _forward(pool, q, t, lens, None)
        assert gb.gbattn_device_status() == GBATTN_EINDEX
        assert (o[1] == 0).all() and torch.isneginf(lse[1]).all() and torch.isfinite(o[0]).all()
    gb.gbattn_device_status()


@pytest.mark.parametrize("bits", [16, 4])
def test_lengths_outside_their_ranges(bits):
    """Lengths are clamped into the page table, numbers of new tokens into 0 .. S."""
    page, H, Hkv, d, S = 16, 4, 2, 128, 5
    pool, table, g = _make(bits, torch.bfloat16, Hkv, d, page, [64, 64, 64, 64], 37)
    table = table[:, :4].contiguous()
    q = torch.randn(4, H, S, d, generator=g).bfloat16().cuda()
    o, lse = _forward(pool, q, table, [1 << 30, -5, 64, -(2 ** 31)], [5, 5, 100, 5], causal=False)
    ref, rl = _forward(pool, q, table, [64, 0, 64, 0], [5, 0, 5, 0], causal=False)
    assert gb.gbattn_device_status() == 0 and _same_bits(o, ref) and torch.equal(lse, rl)
    o, _ = _forward(pool, q, table, [64, 64, 2, 2 ** 31 - 1], [-1, -(2 ** 31), 2 ** 31 - 1, 2 ** 31 - 1])
    ref, _ = _forward(pool, q, table, [64, 64, 2, 64], [0, 0, 5, 0])
    assert gb.gbattn_device_status() == 0 and _same_bits(o[:3], ref[:3])
    assert torch.isfinite(o).all() and (o[2, :, :3] == 0).all()


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [2, 40, 130])
@pytest.mark.parametrize("bits", [16, 4])
def test_scales_scores_and_given_arguments(bits, S):
    """Scores that grow along the keys by more than the lazy reference allows, up to a
    softmax that is one key's; scales of every sign; out, lse and workspace given."""
    lens, page, H, Hkv, d = [400, 329], 32, 4, 1, 128
    pool, table, g = _make(bits, torch.float16, Hkv, d, page, lens, 38)
    q = (torch.randn(2, H, S, d, generator=g) * torch.tensor([0.01, 1.0, 30.0, 300.0])[:, None, None]).half().cuda()
    ws = torch.empty(gb.attn_fwd_paged_workspace_bytes(2, H, Hkv, S, d), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, H, S, device="cuda")
    for scale in (0.7, -0.3, 0.0):
        ws.fill_(255)
        o, l2 = _forward(pool, q, table, lens, None, scale=scale, out=out, lse=lse, workspace=ws)
        assert o is out and l2 is lse and gb.gbattn_device_status() == 0
        _ok(pool, q if scale >= 0 else -q, table, lens, [S, S], o, lse, True, abs(scale))
    o, none = _forward(pool, q, table, lens, None, return_lse=False)
    assert none is None


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [2, 100])
def test_wide_queries_over_four_bits(S):
    """bf16 queries far outside fp16's range, whose products the row's scale keeps exact."""
    pool, table, g = _make(4, torch.bfloat16, 1, 64, 64, [200], 39)
    q = torch.randn(1, 3, S, 64, generator=g)
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q = q.bfloat16().cuda()
    for scale in (1e-30, 1e30):
        qs = q[:, [0, 2] if scale < 1 else [1, 2]].contiguous()
        o, lse = _forward(pool, qs, table, [200], None, scale=scale)
        _ok(pool, qs, table, [200], [S], o, lse, True, scale)


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [2, 100])
@pytest.mark.parametrize("scale", [2.0 ** -127, 2.0 ** -140])
def test_scales_below_the_normal_numbers(scale, S):
    """Scores of up to 2^127 before their scale."""
    pool, table, g = _make(16, torch.bfloat16, 2, 64, 64, [300], 47)
    pool.t[0] = pool.t[0] * 2.0 ** 60
    pool.gpu[0] = pool.t[0].cuda()
    q = (torch.randn(1, 4, S, 64, generator=g) * 2.0 ** 61).bfloat16().cuda()
    o, lse = _forward(pool, q, table, [300], None, scale=scale)
    assert gb.gbattn_device_status() == 0
    _ok(pool, q, table, [300], [S], o, lse, True, scale)


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [2, 100])
@pytest.mark.parametrize("scale,descale,size", [(-100, -30, 124), (118, 10, -126), (-146, 20, 126), (2, 100, -105)])
def test_scale_times_descale_outside_fp32(scale, descale, size, S):
    """Powers of two whose product with the size of the queries is an ordinary scale,
    while the scale times the descale (or the scale itself) is no normal number."""
    pool, table, g = _make(4, torch.bfloat16, 2, 64, 64, [300], 48)
    pool.descale[0] = pool.descale[0] * 2.0 ** descale
    pool.kw["k_descale"] = pool.descale[0].cuda()
    q = (torch.rand(1, 4, S, 64, generator=g) - 0.5).bfloat16() * 2.0 ** size
    assert (q.float().abs().amax(-1) > 2.0 ** (size - 2)).all()
    q = q.cuda()
    o, lse = _forward(pool, q, table, [300], None, scale=2.0 ** scale)
    assert gb.gbattn_device_status() == 0
    _ok(pool, q, table, [300], [S], o, lse, True, 2.0 ** scale)


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("S", [2, 100])
def test_a_scale_of_zero_with_wide_factors(S):
    """Every score is 0, whatever the descale and the queries are."""
    pool, table, g = _make(4, torch.bfloat16, 2, 64, 64, [300], 53)
    pool.descale[0] = pool.descale[0] * 2.0 ** 100
    pool.kw["k_descale"] = pool.descale[0].cuda()
    q = torch.randn(1, 4, S, 64, generator=g).bfloat16() * 2.0 ** 100
    for scale in (0.0, -0.0):
        o, lse = _forward(pool, q.cuda(), table, [300], None, scale=scale)
        assert gb.gbattn_device_status() == 0
        # the keys' magnitude does not matter to the bound: at a scale of 0 it is 0
        _ok(pool, q, table, [300], [S], o, lse, True, 0.0)


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, in both units of work."""
    page, Hkv, d = 1024, 2, 128
    n_pages = 8400  # 2.2e9 elements, 4.4e9 bytes
    kc, vc = (torch.empty(n_pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    g = torch.Generator().manual_seed(42)
    table = torch.tensor([[n_pages - 1, -1], [n_pages - 2, n_pages - 3]], dtype=torch.int32)
    lens = [140, 1140]
    new = torch.randn(2, 3, 2, Hkv, page, d, generator=g).bfloat16()[0].cuda()
    kc[n_pages - 3:], vc[n_pages - 3:] = new[:, 0], new[:, 1]
    for S in (40, 140):
        q = torch.randn(2, Hkv, S, d, generator=g).bfloat16().cuda()
        o, lse = gb.attn_fwd_paged(q, kc, vc, table.cuda(), _i32(lens))
        assert gb.gbattn_device_status() == 0
        kv = gb.attn_cache_gather(kc, vc, table.cuda(), _i32(lens), 1140)
        cu.check(o, lse, q, lambda b, n: tuple(t[b, :, :n].cpu() for t in kv), lens, [S, S], True, 1 / math.sqrt(d),
                 pu.u(torch.bfloat16), half_o=pu.u(torch.bfloat16))
    codes = [torch.zeros(2 * n_pages, Hkv, page, n, dtype=torch.uint8, device="cuda") for _ in "kv" for n in (64, 8)]
    table = 2 * table.clamp(min=0) + 1
    gb.attn_cache_append_fp4(kv[0], kv[1], *codes, table.cuda(), _i32([1140, 1140]), new_lens=_i32([0, 1140]))
    q = torch.randn(2, Hkv, 40, d, generator=g).bfloat16().cuda()
    o, lse = gb.attn_fwd_paged_fp4(q, *codes, table.cuda(), _i32([0, 1140]))
    assert gb.gbattn_device_status() == 0
    back = gb.attn_cache_gather_fp4(*codes, table.cuda(), _i32([0, 1140]), 1140, dtype=torch.float16)  # exact
    cu.check(o, lse, q, lambda b, n: tuple(t[b, :, :n].cpu() for t in back), [0, 1140], [40, 40], True,
             1 / math.sqrt(d), pu.u(torch.float16), 2.0 ** -24, True, pu.u(torch.bfloat16))


@pytest.mark.parametrize("S", [1, 200])
@pytest.mark.parametrize("bits", [16, 4])
def test_longest_cache(bits, S):
    """As many tokens as a page table may hold, where the pages that are looked up ahead
    would be past what 32 bits count.  All but the last two pages are one page; the
    queries follow a key of the last but one, beside which the other pages' weights are
    as good as 0."""
    dtype, d, page = torch.bfloat16, 64, 1024
    g = torch.Generator().manual_seed(41)
    pool = Pool(bits, 3, 1, page, d, dtype, g)
    n_pages, rest = (2 ** 31 - 257) // page, 700
    table = torch.zeros(1, n_pages, dtype=torch.int32)
    table[0, -2:] = torch.tensor([1, 2])
    tail = torch.tensor([1, 2], dtype=torch.int32)
    n = page + rest
    k, v = pool.values(0, tail, n), pool.values(1, tail, n)
    q = (8 * k[:, 5].float()).to(dtype)[None, :, None].expand(1, 1, S, d).contiguous()
    scale = 1 / math.sqrt(d)
    first = pool.values(0, torch.zeros(1, dtype=torch.int32), page)[0].double() @ q[0, 0, 0].double() * scale
    own = float(k[0, 5].double() @ q[0, 0, 0].double()) * scale
    assert torch.logsumexp(first, 0) + math.log(n_pages) < own - 20
    o, lse = _forward(pool, q.cuda(), table, [(n_pages - 1) * page + rest], None, scale=scale)
    assert gb.gbattn_device_status() == 0
    half_p = pu.u(torch.float16) if bits == 4 else pu.u(dtype)
    cu.check(o, lse, q, lambda b, _: (k, v), [n], [S], True, scale, half_p, 2.0 ** -24 if bits == 4 else 0.0, bits == 4,
             pu.u(dtype))


@pytest.mark.parametrize("S,lens,causal", [(3, [700], True), (3, [2500, 100], True), (300, [2500, 301], True),
                                           (3, [2500, 0], False)])
@pytest.mark.parametrize("bits", [16, 4])
def test_units_by_the_longest_tables_key_tiles_pass_32_bits(bits, S, lens, causal):
    """Units times the key tiles that the table has room for pass 2^31, so the list of
    tiles is divided in 64 bits: whole units and runs, one and two row tiles, against the
    same call with a table that is divided in 32."""
    dtype, heads, d, page = torch.bfloat16, 130, 64, 1024
    pool, table, g = _make(bits, dtype, heads, d, page, lens, 50)
    q = torch.randn(len(lens), heads, S, d, generator=g).to(dtype).cuda()
    widths = [128, (2 ** 31 - 257) // page]
    assert len(lens) * heads * (widths[1] * page // 128) > 2 ** 31
    outs = [_forward(pool, q, torch.nn.functional.pad(table, (0, w - table.shape[1]), value=1 << 30), lens, None,
                     causal=causal) for w in widths]
    assert gb.gbattn_device_status() == 0
    assert _same_bits(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    _ok(pool, q, table, lens, [S] * len(lens), *outs[1], causal, 1 / math.sqrt(d))


@pytest.mark.parametrize("bits", [16, 4])
def test_more_sequences_than_a_grid_dimension_holds(bits):
    """70000 sequences of 0 to 16 tokens, a page each (some share one), against the
    definition for all of them at once."""
    B, H, S, d, page, dtype = 70000, 2, 2, 64, 16, torch.float16
    g = torch.Generator().manual_seed(52)
    pool = Pool(bits, 300, 1, page, d, dtype, g)
    lens = torch.randint(0, page + 1, (B,), generator=g)
    table = torch.randint(0, 300, (B, 1), generator=g, dtype=torch.int32)
    q = torch.randn(B, H, S, d, generator=g).to(dtype).cuda()
    o, lse = _forward(pool, q, table, lens.tolist(), None)
    assert gb.gbattn_device_status() == 0
    every = torch.arange(300, dtype=torch.int32)
    k, v = (pool.values(i, every, 300 * page).double().view(300, page, d).cuda()[table[:, 0].cuda().long()] for i in range(2))
    lens, scale = lens.cuda(), 1 / math.sqrt(d)
    seen = torch.arange(page, device="cuda") <= (lens[:, None] - S + torch.arange(S, device="cuda"))[..., None]  # [B, S, page]
    raw = torch.einsum("bhsd,bpd->bhsp", q.double(), k)
    mag = torch.einsum("bhsd,bpd->bhsp", q.double().abs(), k.abs()).amax(-1, keepdim=True) * scale
    s = (raw * scale).masked_fill(~seen[:, None], -math.inf)
    real = seen.any(-1)[:, None].expand(B, H, S)
    rl = torch.logsumexp(s, -1)
    p = torch.exp(s - rl.masked_fill(~real, 0.0)[..., None])
    ro = torch.einsum("bhsp,bpd->bhsd", p, v)
    # chunk_util's bound, with fp16 weights (over 4 bits too)
    half = pu.u(torch.float16)
    e = 2 * d * pu.U32 * mag + mag * 4 * pu.U32 + 2.0 ** -20
    tol = (half + 2 * e) * torch.einsum("bhsp,bpd->bhsd", p, v.abs()) + 2.0 ** -25 * torch.einsum(
        "bsp,bpd->bsd", seen.double(), v.abs())[:, None]
    tol = tol + half * (ro.abs() + tol) + 2.0 ** -25
    assert ((o.double() - ro).abs() <= tol).all()
    assert ((lse.double() - rl).abs() <= e[..., 0] + rl.abs() * 4 * pu.U32 + 2.0 ** -20)[real].all()
    assert (o[~real] == 0).all() and torch.isneginf(lse[~real]).all() and not real.all()


@pytest.mark.parametrize("S", [3, 90])
@pytest.mark.parametrize("bits", [16, 4])
def test_streams_graphs_and_two_calls_at_once(bits, S):
    """A captured step (append, attention) replayed with other lengths, behind fills
    and copies, and two calls on two streams with a workspace each."""
    page, H, Hkv, d, B = 16, 8, 2, 128, 4
    pool, table, g = _make(bits, torch.bfloat16, Hkv, d, page, [300] * B, 40)
    q, other = (torch.randn(B, H, S, d, generator=g).bfloat16().cuda() for _ in range(2))
    k, v = (torch.randn(B, Hkv, S, d, generator=g).bfloat16().cuda() for _ in "kv")
    rope, td = gb.rope_table(400, d), table.cuda()
    lens, new = _i32([S] * B), _i32([S] * B)
    fn = gb.attn_fwd_paged if bits == 16 else gb.attn_fwd_paged_fp4

    def step():
        qr = pool.append(k, v, td, lens, rope=rope, q=q, new_lens=new)
        out = fn(qr, *pool.gpu, td, lens, new_lens=new, **pool.kw)
        qr.fill_(float("nan"))
        return [t.clone() for t in out]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for a, b in (([S] * B, [S] * B), ([300, 117, 0, 290], [S, 1, 0, S - 1]), ([100, 128, 129, 300], [S, S, 2, 0])):
        lens.copy_(_i32(a))
        new.copy_(_i32(b))
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
        assert all(torch.equal(x, y) for x, y in zip(first, step()))
    refs = [fn(x, *pool.gpu, td, lens, **pool.kw) for x in (q, other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty(gb.attn_fwd_paged_workspace_bytes(B, H, Hkv, S, d), dtype=torch.uint8, device="cuda")
          for _ in streams]
    for _ in range(5):
        outs = [fn(x, *pool.gpu, td, lens, **pool.kw, workspace=w, stream=s) for x, w, s in zip((q, other), ws, streams)]
        torch.cuda.synchronize()
        for a, b in zip(outs, refs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # what a call on another stream allocates is that stream's
    need = gb.attn_fwd_paged_workspace_bytes(B, H, Hkv, S, d, table.shape[1] * page)
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(streams[0]):
        for _ in range(8):
            busy @ busy
    o, lse = fn(q, *pool.gpu, td, lens, **pool.kw, stream=streams[0])
    fills = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (need, need, q.numel() * 2, B * H * S * 4)]
    torch.cuda.synchronize()
    assert torch.equal(o, refs[0][0]) and torch.equal(lse, refs[0][1]) and all((f == 255).all() for f in fills)
    assert gb.gbattn_device_status() == 0


def test_agrees_with_the_contiguous_forward_and_the_decode():
    """The same attention through attn_fwd over the gathered cache, and through the
    decode for its last token: all within their bounds of one definition, so within
    the parity tests' bounds of each other."""
    from tests.parity_util import LSE_MAX_ABS, O_MAX_ABS

    lens, page, H, Hkv, d, S = [500] * 3, 32, 8, 2, 128, 200
    pool, table, g = _make(16, torch.bfloat16, Hkv, d, page, lens, 41)
    q = torch.randn(3, H, S, d, generator=g).bfloat16().cuda()
    kv = pool.gather(table.cuda(), _i32(lens), 500)
    for causal in (True, False):
        o, lse = _forward(pool, q, table, lens, None, causal=causal)
        o1, l1 = gb.attn_fwd(q, *kv, causal=causal)
        assert (o.float() - o1.float()).abs().max() <= O_MAX_ABS and (lse - l1).abs().max() <= LSE_MAX_ABS
    last = q[:, :, -1:].contiguous()
    o2, l2 = pool.decode(last, table.cuda(), _i32(lens))
    assert (o[:, :, -1:].float() - o2.float()).abs().max() <= O_MAX_ABS
    assert (lse[:, :, -1] - l2).abs().max() <= LSE_MAX_ABS


def test_wrapper_refusals():
    g = torch.Generator().manual_seed(45)
    pool, pool4 = Pool(16, 3, 2, 16, 64, torch.float16, g), Pool(4, 3, 2, 16, 64, torch.float16, g)
    table, lens = _i32([[0, 1]]), _i32([20])
    q = torch.zeros(1, 4, 5, 64, dtype=torch.float16, device="cuda")
    bad = [
        lambda: gb.attn_fwd_paged(q.bfloat16(), *pool.gpu, table, lens),
        lambda: gb.attn_fwd_paged(q.transpose(1, 2), *pool.gpu, table, lens),
        lambda: gb.attn_fwd_paged(q[:, :3].contiguous(), *pool.gpu, table, lens),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table.long(), lens),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, new_lens=_i32([5, 5])),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, new_lens=lens.long()),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table.cpu(), lens),
        lambda: gb.attn_fwd_paged(q, pool.gpu[0], pool.gpu[1][:2], table, lens),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, scale=float("nan")),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, scale=float("inf")),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, lse=torch.zeros(1, 4, device="cuda")),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, out=q.float()),
        lambda: gb.attn_fwd_paged(q, *pool.gpu, table, lens, workspace=torch.empty(16, device="cuda")),
        lambda: gb.attn_fwd_paged(q[:, :, :0], *pool.gpu, table, lens),
        lambda: gb.attn_fwd_paged_fp4(q, *pool4.gpu[:3], None, table, lens),
        lambda: gb.attn_fwd_paged_fp4(q, pool4.gpu[0], pool4.gpu[1][..., :2], *pool4.gpu[2:], table, lens),
        lambda: gb.attn_fwd_paged_fp4(q, *pool4.gpu, table, lens, v_descale=torch.ones(3, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, gb.GbattnError)):
            f()
            pytest.fail(f"call {i} was not refused")
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("bits", [16, 4])
def test_outputs_that_share_memory_are_refused(bits):
    g = torch.Generator().manual_seed(49)
    B, H, Hkv, S, d, page = 2, 4, 2, 5, 64, 16
    # everything from one block of memory, so that neighbours can be had
    block = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    used = 0

    def place(t):
        nonlocal used
        at, used = used, used + (t.numel() * t.element_size() + 255) // 256 * 256
        view = block[at:at + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        view.copy_(t)
        return view

    pool = Pool(bits, 3, Hkv, page, d, torch.float16, g)
    pool.gpu = [place(t.view(torch.uint8)).view(t.dtype) if t.element_size() == 1 else place(t) for t in pool.gpu]
    pool.kw = {n: place(t) for n, t in pool.kw.items()}
    table, lens, news = place(_i32([[0, 1], [2, 0]])), place(_i32([20, 10])), place(_i32([5, 3]))
    q = place(torch.randn(B, H, S, d, generator=g).half().cuda())
    ws = place(torch.zeros(gb.attn_fwd_paged_workspace_bytes(B, H, Hkv, S, d, 32), dtype=torch.uint8, device="cuda"))
    out, lse = place(torch.zeros_like(q)), place(torch.zeros(B, H, S, device="cuda"))
    fn = gb.attn_fwd_paged if bits == 16 else gb.attn_fwd_paged_fp4

    def call(**kw):
        kw = dict(dict(new_lens=news, workspace=ws, out=out, lse=lse), **pool.kw, **kw)
        return fn(q, *pool.gpu, table, lens, **kw)

    ref = fn(q, *pool.gpu, table, lens, new_lens=news, **pool.kw)
    o, l2 = call()
    assert o is out and l2 is lse and torch.equal(o, ref[0]) and torch.equal(l2, ref[1])
    inputs = [q, *pool.gpu, *pool.kw.values(), table, lens, news, ws]
    for like, name in ((out, "out"), (lse, "lse")):
        size = like.numel() * like.element_size()
        for other in [*inputs, lse if name == "out" else out]:
            first = other.data_ptr() - block.data_ptr()
            last = first + other.numel() * other.element_size()
            for at in {first, max(0, first - size + 16), (last - 1) // 16 * 16}:
                bad = block[at:at + size].view(like.dtype).view(like.shape)
                with pytest.raises(ValueError, match="is written"):  # (its end may lie in a third tensor)
                    call(**{name: bad})
    # side by side is no overlap
    both = place(torch.zeros(2, *q.shape, dtype=q.dtype, device="cuda"))
    both[0].copy_(q)
    o, _ = fn(both[0], *pool.gpu, table, lens, new_lens=news, out=both[1], **pool.kw)
    assert torch.equal(o, ref[0]) and torch.equal(both[0], q)
    assert gb.gbattn_device_status() == 0


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
def test_text_and_images_served_in_chunks(bits):
    """As a program runs them: two sequences of different lengths take chunks of text
    and images (norms and rotation by three axes, append, attention of the chunk), then
    one token each by append and decode; each step against the definition applied to
    what the step before it gave."""
    g = torch.Generator().manual_seed(51)
    B, H, Hkv, d, page, dtype = 2, 4, 2, 64, 16, torch.bfloat16
    pool = Pool(bits, 30, Hkv, page, d, dtype, g)
    table = pu.page_table([200, 200], page, 30, 13, g)
    rope, axes = gb.rope_table(256, d), gb.rope_pair_axes((8, 12, 12))
    w = [1 + 0.1 * torch.randn(d, generator=g) for _ in "qk"]
    wd = [x.cuda() for x in w]
    done, scale = [0, 0], 1 / math.sqrt(d)
    for S, news in ((50, [50, 31]), (70, [12, 70]), (3, [3, 3]), (1, [1, 1])):
        x = torch.randn(B, S, H + 2 * Hkv, d, generator=g).to(dtype).cuda().transpose(1, 2)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        pos = torch.randint(0, 256, (3, B, S), generator=g, dtype=torch.int32)
        qn, kn = gb.attn_qk_norm_rope(q, k, *wd, rope=rope, positions=pos.cuda(), axes=axes)
        done = [a + b for a, b in zip(done, news)]
        pool.append(kn, v, table.cuda(), _i32(done), new_lens=_i32(news))
        pool.pull()
        if S > 1:
            o, lse = _forward(pool, qn, table, done, news)
        else:
            o, lse = pool.decode(qn, table.cuda(), _i32(done))
            lse = lse[..., None]
        assert gb.gbattn_device_status() == 0
        for b, (n, m) in enumerate(zip(done, news)):
            half = rope.shape[1] // 2
            at = torch.stack([pos[a, b] for a in axes], -1).long()
            own = torch.cat([rope.cpu()[at, torch.arange(half)], rope.cpu()[at, half + torch.arange(half)]], -1)
            for i, (raw, got) in enumerate(((q, qn), (k, kn))):
                ref, mag = pu.norm_rope(raw[b].double().cpu(), w[i].double(), own, torch.arange(S), 1e-6, False)
                assert ((got[b].double().cpu() - ref).abs() <= pu.u(dtype) * ref.abs() + 20 * pu.U32 * mag).all()
            if bits == 16:
                assert torch.equal(pool.values(0, table[b], n)[:, n - m:], kn[b, :, :m].float().cpu())
        if S > 1:
            _ok(pool, qn, table, done, news, o, lse, True, scale)
        else:
            half_p = pu.u(torch.float16) if bits == 4 else pu.u(dtype) ** 2
            cu.check(o, lse, qn, lambda b, n: (pool.values(0, table[b], n), pool.values(1, table[b], n)), done, news,
                     True, scale, half_p, 2.0 ** -24 if bits == 4 else 0.0, bits == 4, pu.u(dtype))
