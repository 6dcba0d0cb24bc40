"""The paged cache on the GPU: append, read-back and one-query decode, held in 16
bits and in 4, against their plain forms in 64 bits (bounds in paged_util; what
the 4-bit cache holds is compared bit for bit), and a run of all of them as a
program makes it."""
import math

import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300.binding import GBATTN_EINDEX
from tests import paged_util as pu

pytestmark = pytest.mark.gpu


class Pool:
    """A cache of `bits` bits filled with random bit patterns that stand for
    finite values (and, where `nan`, NaN in every slot)."""

    def __init__(self, bits, n_pages, Hkv, page, d, dtype, gen, nan=False):
        self.bits, self.page, self.d, self.Hkv, self.dtype = bits, page, d, Hkv, dtype
        shape = (n_pages, Hkv, page)
        if bits == 16:
            self.t = [torch.randn(*shape, d, generator=gen).to(dtype) for _ in "kv"]
            if nan:
                self.t = [torch.full_like(t, float("nan")) for t in self.t]
            self.descale = None
        else:
            self.t = []
            for _ in "kv":
                self.t.append(torch.randint(0, 256, (*shape, d // 2), generator=gen, dtype=torch.uint8))
                f = torch.rand(*shape, d // 16, generator=gen).to(torch.float8_e4m3fn)
                if nan:
                    f = torch.full((*shape, d // 16), 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn)
                self.t.append(f)
            self.descale = [0.5 + torch.rand(Hkv, generator=gen) for _ in "kv"]
        self.gpu = [t.cuda() for t in self.t]
        self.kw = {} if bits == 16 else dict(k_descale=self.descale[0].cuda(), v_descale=self.descale[1].cuda())

    def values(self, which, table_row, n):
        """Rows 0 .. n - 1 of a sequence as the fp32 values they stand for, [Hkv, n, d]."""
        if self.bits == 16:
            return pu.sequence(self.t[which], table_row, self.page, n).float()
        codes = pu.sequence(self.t[2 * which], table_row, self.page, n)
        f = pu.sequence(self.t[2 * which + 1].view(torch.uint8), table_row, self.page, n).view(torch.float8_e4m3fn)
        return pu.dequantise(codes, f, self.descale[which][:, None])

    def pull(self):
        self.t = [t.cpu() for t in self.gpu]

    def append(self, k, v, table, lens, **kw):
        fn = gb.attn_cache_append if self.bits == 16 else gb.attn_cache_append_fp4
        return fn(k, v, *self.gpu, table, lens, **self.kw, **kw)

    def gather(self, table, lens, S, **kw):
        if self.bits == 16:
            return gb.attn_cache_gather(*self.gpu, table, lens, S, **kw)
        return gb.attn_cache_gather_fp4(*self.gpu, table, lens, S, dtype=self.dtype, **self.kw, **kw)

    beyond = 0  # columns that decode() adds to a page table

    def decode(self, q, table, lens, **kw):
        if self.beyond:
            table = torch.nn.functional.pad(table, (0, self.beyond), value=1 << 30)
        fn = gb.attn_decode_paged if self.bits == 16 else gb.attn_decode_paged_fp4
        return fn(q, *self.gpu, table, lens, **self.kw, **kw)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same_bits(a, b):
    view = {2: torch.int16, 1: torch.uint8}[a.element_size()]
    return torch.equal(a.view(view), b.view(view))


def _decode_ok(pool, q, table, lens, o, lse, scale, what=""):
    o, lse = o.double().cpu(), lse.double().cpu()
    half_p = pu.u(torch.float16) if pool.bits == 4 else pu.u(pool.dtype) ** 2
    fp16_p = pool.bits == 4 or pool.dtype is torch.float16
    for b, n in enumerate(lens):
        k, v = pool.values(0, table[b], n), pool.values(1, table[b], n)
        # 4 bits: q is scaled into fp16, off by up to 2^-24 of its row's largest
        ro, rl, to, tl = pu.attention(q[b, :, 0].cpu(), k, v, scale, half_p, 2.0 ** -24 if pool.bits == 4 else 0.0,
                                      fp16_p)
        tol = to + pu.u(q.dtype) * (ro.abs() + to) + 2.0 ** -25
        assert torch.isfinite(o[b]).all(), f"{what} sequence {b}"
        bad = (o[b, :, 0] - ro).abs() - tol
        assert (bad <= 0).all(), f"{what} sequence {b} (length {n}): {bad.max():.3e} over the bound"
        if n == 0:
            assert torch.isneginf(lse[b]).all() and (o[b] == 0).all()
        else:
            assert ((lse[b] - rl).abs() <= tl).all(), f"{what} sequence {b}: lse"


@pytest.fixture(params=["narrow", "wide"])
def table_width(request, monkeypatch):
    """What a page table could hold decides how the work is divided: tables as the
    test makes them, and the same ones with room for far more."""
    if request.param == "wide":
        monkeypatch.setattr(Pool, "beyond", 20000)


DECODE = [
    # bits, dtype, Hq, Hkv, d, page, lens
    (16, torch.bfloat16, 1, 1, 128, 16, [1]),
    (16, torch.bfloat16, 8, 2, 128, 64, [1, 77, 300]),
    (16, torch.float16, 6, 2, 64, 16, [15, 16, 17, 0, 31, 32, 33]),
    (16, torch.bfloat16, 9, 1, 128, 32, [63, 64, 65, 127, 128, 129]),
    (16, torch.float16, 16, 1, 128, 128, [1000, 0, 999]),
    (16, torch.bfloat16, 34, 2, 64, 16, [130, 500]),
    (16, torch.bfloat16, 32, 1, 128, 1024, [5, 1025]),
    (16, torch.float16, 5, 5, 128, 256, [2049, 64, 65, 1000]),
    (16, torch.bfloat16, 4, 2, 128, 64, [20000]),
    (16, torch.bfloat16, 2, 1, 64, 16, [0, 0, 0]),
    (4, torch.bfloat16, 1, 1, 128, 16, [1]),
    (4, torch.bfloat16, 8, 2, 128, 64, [1, 77, 300]),
    (4, torch.float16, 6, 2, 64, 16, [15, 16, 17, 0, 31, 32, 33]),
    (4, torch.bfloat16, 9, 1, 128, 32, [63, 64, 65, 127, 128, 129]),
    (4, torch.float16, 16, 1, 128, 128, [1000, 0, 999]),
    (4, torch.bfloat16, 34, 2, 64, 16, [130, 500]),
    (4, torch.float16, 32, 1, 64, 1024, [5, 1025]),
    (4, torch.float16, 5, 5, 128, 256, [2049, 64, 65, 1000]),
    (4, torch.bfloat16, 4, 2, 128, 64, [20000]),
    (4, torch.bfloat16, 2, 1, 64, 16, [0, 0, 0]),
]


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("cfg", DECODE)
def test_decode(cfg):
    bits, dtype, Hq, Hkv, d, page, lens = cfg
    g = torch.Generator().manual_seed(21)
    width = max(1, (max(lens) + page - 1) // page) + 1
    n_pages = sum((n + page - 1) // page for n in lens) + 2
    pool = Pool(bits, n_pages, Hkv, page, d, dtype, g)
    table = pu.page_table(lens, page, n_pages, width, g, beyond=1 << 30)
    q = torch.randn(len(lens), Hq, 1, d, generator=g).to(dtype).cuda()
    o, lse = pool.decode(q, table.cuda(), _i32(lens))
    assert gb.gbattn_device_status() == 0
    _decode_ok(pool, q, table, lens, o, lse, 1 / math.sqrt(d))
    o2, lse2 = pool.decode(q, table.cuda(), _i32(lens))
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # repeats bitwise


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
def test_decode_many_short_sequences(bits):
    """More sequences than a block has threads, idle ones among them, lengths on
    both sides of a unit: every CTA's run holds several segments."""
    g = torch.Generator().manual_seed(22)
    lens = [(0, 1, 64, 65, 130, 17)[i % 6] for i in range(301)]
    page, Hq, Hkv, d = 16, 4, 2, 64
    n_pages = sum((n + page - 1) // page for n in lens)
    pool = Pool(bits, n_pages, Hkv, page, d, torch.float16, g)
    table = pu.page_table(lens, page, n_pages, 9, g)
    q = torch.randn(len(lens), Hq, 1, d, generator=g).half().cuda()
    o, lse = pool.decode(q, table.cuda(), _i32(lens))
    _decode_ok(pool, q, table, lens, o, lse, 0.125)
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("B,Hq,Hkv,d", [(2, 8, 4, 64), (15, 8, 4, 128), (20, 39, 3, 64), (43, 5, 5, 64), (30, 12, 12, 128)])
@pytest.mark.parametrize("bits", [16, 4])
def test_decode_small_batches(bits, B, Hq, Hkv, d):
    """From few sequences to about as many as there are places for blocks, and an
    idle one."""
    g = torch.Generator().manual_seed(28)
    page = 32
    lens = torch.randint(1, 600, (B,), generator=g).tolist()
    lens[0], lens[-1] = 600, 0
    n_pages = sum((n + page - 1) // page for n in lens)
    pool = Pool(bits, n_pages, Hkv, page, d, torch.bfloat16, g)
    table = pu.page_table(lens, page, n_pages, 19, g)
    q = torch.randn(B, Hq, 1, d, generator=g).bfloat16().cuda()
    o, lse = pool.decode(q, table.cuda(), _i32(lens))
    _decode_ok(pool, q, table, lens, o, lse, 1 / math.sqrt(d))
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bits", [16, 4])
def test_decode_one_long_sequence_among_many(bits, d):
    """More rows than the merge takes a CTA each for, one of them split over a
    large part of the grid."""
    g = torch.Generator().manual_seed(27)
    lens = [(1, 0, 40)[i % 3] for i in range(330)]
    lens[17] = 30011
    page, Hq, Hkv = 64, 4, 1
    n_pages = sum((n + page - 1) // page for n in lens)
    pool = Pool(bits, n_pages, Hkv, page, d, torch.bfloat16, g)
    table = pu.page_table(lens, page, n_pages, 470, g)
    q = torch.randn(len(lens), Hq, 1, d, generator=g).bfloat16().cuda()
    o, lse = pool.decode(q, table.cuda(), _i32(lens))
    _decode_ok(pool, q, table, lens, o, lse, 1 / math.sqrt(d))
    assert gb.gbattn_device_status() == 0


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
def test_decode_rows_behind_the_length_are_not_used(bits):
    """Slots behind each length, unused pages and factors hold NaN."""
    g = torch.Generator().manual_seed(23)
    lens, page, Hq, Hkv, d = [1, 333, 50, 700], 64, 8, 2, 128
    n_pages = 30
    pool = Pool(bits, n_pages, Hkv, page, d, torch.bfloat16, g)
    table = pu.page_table(lens, page, n_pages, 12, g)
    q = torch.randn(4, Hq, 1, d, generator=g).bfloat16().cuda()
    o, lse = pool.decode(q, table.cuda(), _i32(lens))
    dirty = Pool(bits, n_pages, Hkv, page, d, torch.bfloat16, g, nan=True)
    for t, src in zip(dirty.gpu, pool.gpu):
        t, src = (x.view(torch.uint8) if x.element_size() == 1 else x for x in (t, src))
        for b, n in enumerate(lens):
            for i in range((n + page - 1) // page):
                rows = min(page, n - i * page)
                t[table[b, i], :, :rows] = src[table[b, i], :, :rows]
    dirty.kw = pool.kw
    o2, lse2 = dirty.decode(q, table.cuda(), _i32(lens))
    assert torch.isfinite(o2).all() and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
def test_decode_large_scores_and_given_arguments(bits):
    """Scores that grow along the keys by more than the lazy reference allows,
    up to a softmax that is one key's; a given scale (also a negative one), out,
    lse and workspace."""
    g = torch.Generator().manual_seed(24)
    lens, page, Hq, Hkv, d = [400, 129], 32, 4, 1, 128
    pool = Pool(bits, 20, Hkv, page, d, torch.float16, g)
    table = pu.page_table(lens, page, 20, 13, g)
    q = (torch.randn(2, Hq, 1, d, generator=g) * torch.tensor([0.01, 1.0, 30.0, 300.0])[:, None, None]).half().cuda()
    ws = torch.empty(gb.attn_decode_paged_workspace_bytes(2, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, Hq, device="cuda")
    for scale in (0.7, -0.3, 0.0):
        o, l2 = pool.decode(q, table.cuda(), _i32(lens), scale=scale, out=out, lse=lse, workspace=ws)
        assert o is out and l2 is lse
        # the plain form takes |scale| for its bounds and the sign with q
        _decode_ok(pool, q if scale >= 0 else -q, table, lens, o, lse, abs(scale))
    o, none = pool.decode(q, table.cuda(), _i32(lens), return_lse=False)
    assert none is None


# (B, Hq, Hkv, L): a warp that holds the last key alone; a part of a split sequence
# that does, folded by a CTA a row; many rows, folded by a warp each
LAST_KEY = [(2, 4, 2, {16: 17, 4: 33}), (1, 4, 1, {16: 193, 4: 385}), (160, 8, 1, {16: 2048, 4: 2048})]


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("where", ["key", "value"])
@pytest.mark.parametrize("case", LAST_KEY)
@pytest.mark.parametrize("bits", [16, 4])
def test_nan_in_a_row_that_counts(bits, case, where):
    """NaN in the last key of every sequence but one: all of o and lse of its heads
    are NaN; in the last value: its elements of o, whose weight is far below the
    smallest fp32 number here (the keys of the second half point against q)."""
    g = torch.Generator().manual_seed(77)
    B, Hq, Hkv, L, d = *case[:3], case[3][bits], 64
    n = (L + 15) // 16
    pool = Pool(bits, B * n, Hkv, 16, d, torch.bfloat16, g)
    table = torch.arange(B * n, dtype=torch.int32).view(B, n)
    sign = torch.where(torch.arange(n * 16) < L // 2, 1.0, -1.0).view(n, 1, 16, 1)
    q = torch.full((B, Hq, 1, d), 1.0, dtype=torch.bfloat16)
    page, slot = table[1:, -1].long() if B > 1 else table[:, -1].long(), (L - 1) % 16
    if bits == 16:
        pool.t[0] = (sign * torch.ones(B, n, Hkv, 16, d)).flatten(0, 1).to(torch.bfloat16)
        pool.t[0 if where == "key" else 1][page, :, slot, 5] = float("nan")
    else:
        code = torch.where(sign > 0, 0x22, 0xAA).to(torch.uint8)  # 1 and -1
        pool.t[0] = code.expand(B, n, Hkv, 16, d // 2).flatten(0, 1).contiguous()
        pool.t[1] = torch.ones_like(pool.t[1].float()).to(torch.float8_e4m3fn)
        pool.t[1 if where == "key" else 3].view(torch.uint8)[page, :, slot, 0] = 0x7F  # elements 0 .. 15
    pool.gpu = [t.cuda() for t in pool.t]
    o, lse = pool.decode(q.cuda(), table.cuda(), _i32([L] * B), scale=4.0)
    o, lse = o.cpu()[:, :, 0], lse.cpu()
    touched = slice(1, None) if B > 1 else slice(None)
    if B > 1:
        assert torch.isfinite(o[0]).all() and torch.isfinite(lse[0]).all()
    if where == "key":
        assert torch.isnan(o[touched]).all() and torch.isnan(lse[touched]).all()
    else:
        bad = torch.zeros(d, dtype=torch.bool)
        bad[slice(5, 6) if bits == 16 else slice(0, 16)] = True
        assert torch.isnan(o[touched][..., bad]).all() and torch.isfinite(o[touched][..., ~bad]).all()
        assert torch.isfinite(lse[touched]).all()


@pytest.mark.usefixtures("table_width")
def test_decode_wide_queries_over_four_bits():
    """bf16 queries far outside fp16's range, whose products the row's scale keeps exact."""
    g = torch.Generator().manual_seed(25)
    pool = Pool(4, 5, 1, 64, 64, torch.bfloat16, g)
    table = pu.page_table([200], 64, 5, 4, g)
    q = torch.randn(1, 3, 1, 64, generator=g)
    q[0, 0] *= 1e30
    q[0, 1] *= 1e-30
    q[0, 2] = 0
    q = q.bfloat16().cuda()
    for scale in (1e-30, 1e30):
        pick = [0, 2] if scale < 1 else [1, 2]
        qs = q[:, pick]
        o, lse = pool.decode(qs.contiguous(), table.cuda(), _i32([200]), scale=scale)
        _decode_ok(pool, qs, table, [200], o, lse, scale)


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_that_do_not_exist(bits):
    """A page outside the pool is left out of the attention, read back as zeros
    and not written; the status word says so."""
    g = torch.Generator().manual_seed(26)
    lens, page, Hq, Hkv, d = [100, 40], 16, 4, 2, 64
    pool = Pool(bits, 12, Hkv, page, d, torch.float16, g)
    table = pu.page_table(lens, page, 12, 7, g)
    q = torch.randn(2, Hq, 1, d, generator=g).half().cuda()
    gb.gbattn_device_status()
    for bad in (-1, 12, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        o, lse = pool.decode(q, t.cuda(), _i32(lens))
        assert gb.gbattn_device_status() == GBATTN_EINDEX and gb.gbattn_device_status() == 0
        keep = [i for i in range(100) if i // page != 2]
        k, v = (pool.values(i, table[0], 100)[:, keep] for i in range(2))
        ro, rl, to, tl = pu.attention(q[0, :, 0].cpu(), k, v, 0.125, pu.u(torch.float16), 2.0 ** -24, True)
        assert ((o[0, :, 0].double().cpu() - ro).abs() <= to + pu.u(torch.float16) * (ro.abs() + to) + 2.0 ** -25).all()
        assert ((lse[0].double().cpu() - rl).abs() <= tl).all()
        kk, vv = pool.gather(t.cuda(), _i32(lens), 100)
        assert gb.gbattn_device_status() == GBATTN_EINDEX
        whole = pool.gather(table.cuda(), _i32(lens), 100)
        assert gb.gbattn_device_status() == 0
        for got, ref in zip((kk, vv), whole):
            assert (got[0, :, 32:48] == 0).all()
            ref[0, :, 32:48] = 0
            assert torch.equal(got, ref)
        before = [x.clone() for x in pool.gpu]
        new = torch.randn(2, Hkv, 1, d, generator=g).half().cuda()
        t = table.clone()
        t[0, 6] = bad
        pool.append(new, new, t.cuda(), _i32([97, 0]))
        assert gb.gbattn_device_status() == GBATTN_EINDEX
        pool.append(new, new, table.cuda(), _i32([113, -3]))  # slot 112: behind the last page of the table
        assert gb.gbattn_device_status() == GBATTN_EINDEX
        assert all(_same_bits(a, b) for a, b in zip(before, pool.gpu))
    # lengths outside the table are clamped into it
    o, lse = pool.decode(q, pu.page_table([112, 0], page, 12, 7, g).cuda(), _i32([1 << 30, -5]))
    assert gb.gbattn_device_status() == 0
    assert torch.isfinite(o).all() and (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    k, _ = pool.gather(pu.page_table([112, 0], page, 12, 7, g).cuda(), _i32([1 << 30, -5]), 130)
    assert gb.gbattn_device_status() == 0
    assert (k[0, :, :112] != 0).any() and (k[0, :, 112:] == 0).all() and (k[1] == 0).all()


APPEND = [
    # bits, dtype, B, S, H (0: no q), Hkv, d, page, rot, interleaved
    (16, torch.bfloat16, 3, 1, 8, 2, 128, 64, 128, False),
    (16, torch.float16, 2, 37, 6, 3, 64, 16, 32, True),
    (16, torch.bfloat16, 2, 70, 0, 1, 128, 32, 96, False),
    (16, torch.float16, 5, 9, 4, 4, 64, 1024, 0, False),
    (16, torch.bfloat16, 2, 200, 16, 8, 128, 64, 128, False),
    (4, torch.bfloat16, 3, 1, 8, 2, 128, 64, 128, False),
    (4, torch.float16, 2, 37, 6, 3, 64, 16, 32, True),
    (4, torch.bfloat16, 2, 70, 0, 1, 128, 32, 96, False),
    (4, torch.float16, 5, 9, 4, 4, 64, 1024, 0, False),
    (4, torch.bfloat16, 2, 200, 16, 8, 128, 64, 128, False),
]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("cfg", APPEND)
def test_append(cfg, ragged):
    """What is stored, and that every other slot keeps its bits."""
    bits, dtype, B, S, H, Hkv, d, page, rot, interleaved = cfg
    g = torch.Generator().manual_seed(31)
    new = [min(S, (0, 1, S, S - 1, 2)[i % 5]) for i in range(B)] if ragged else [S] * B
    lens = [n + (0, 13, 64, 5, 200)[i % 5] for i, n in enumerate(new)]
    width = max((n + page - 1) // page for n in lens) + 1
    n_pages = sum((n + page - 1) // page for n in lens) + 2
    pool = Pool(bits, n_pages, Hkv, page, d, dtype, g)
    table = pu.page_table(lens, page, n_pages, width, g)
    x = torch.randn(B, S, H + 2 * Hkv, d, generator=g).to(dtype)
    x[:, :, :, :16] *= 30  # groups of different sizes
    x[:, -1, :, 16:32] = 0
    x = x.cuda().transpose(1, 2)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    rope = gb.rope_table(max(lens) + 1, rot, device="cpu") if rot else None
    out = pool.append(k, v, table.cuda(), _i32(lens), new_lens=_i32(new) if ragged else None,
                      rope=None if rope is None else rope.cuda(), interleaved=interleaved, q=q if H else None)
    assert gb.gbattn_device_status() == 0
    before = [t.clone() for t in pool.t]
    pool.pull()
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n - m, n)
        kb, vb, qb = (t[b, :, :m].cpu() for t in (k, v, q))
        if H:
            ob = out[b].double().cpu()
            ref, mag = (qb.double(), qb.double().abs()) if rope is None else pu.turn(qb.double(), rope, pos, interleaved)
            tol = pu.u(dtype) * ref.abs() + 3 * pu.U32 * mag + 2.0 ** -25
            assert ((ob[:, :m] - ref).abs() <= tol).all() and (ob[:, m:] == 0).all()
        else:
            assert out is None
        pages, rows = table[b][pos // page].long(), pos % page
        # the same products and sum in fp32, rounded one by one
        k32 = kb.float() if rope is None else pu.turn(kb.float(), rope, pos, interleaved)[0]
        if bits == 16:
            for i, ref in enumerate((k32.to(dtype), vb)):
                assert torch.equal(pool.t[i][pages, :, rows], ref.transpose(0, 1))
                before[i][pages, :, rows] = pool.t[i][pages, :, rows]
        else:
            for i, ref in enumerate((k32, vb.float())):
                codes, f = pu.quantise(ref, pool.descale[i][:, None])
                assert torch.equal(pool.t[2 * i][pages, :, rows], codes.transpose(0, 1))
                f, got = f.view(torch.uint8), pool.t[2 * i + 1].view(torch.uint8)
                assert torch.equal(got[pages, :, rows], f.transpose(0, 1))
                before[2 * i][pages, :, rows] = pool.t[2 * i][pages, :, rows]
                before[2 * i + 1].view(torch.uint8)[pages, :, rows] = got[pages, :, rows]
    assert all(_same_bits(a, b) for a, b in zip(before, pool.t))


@pytest.mark.parametrize("rot,interleaved", [(128, False), (48, False), (48, True), (0, False)])
@pytest.mark.parametrize("bits", [16, 4])
def test_append_rotates_queries_in_place(bits, rot, interleaved):
    g = torch.Generator().manual_seed(32)
    B, S, H, Hkv, d = 2, 45, 12, 4, 128
    q, k, v = (torch.randn(B, h, S, d, generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    table = pu.page_table([60, 30], 16, 8, 4, g).cuda()
    rope = gb.rope_table(64, rot) if rot else None
    args = dict(new_lens=_i32([45, 20]), rope=rope, interleaved=interleaved)
    pools = [Pool(bits, 8, Hkv, 16, d, torch.bfloat16, torch.Generator().manual_seed(1)) for _ in range(2)]
    ref = pools[0].append(k, v, table, _i32([60, 30]), q=q, **args)
    for _ in range(20):
        mine = q.clone()
        out = pools[1].append(k, v, table, _i32([60, 30]), q=mine, q_out=mine, **args)
        assert out is mine and torch.equal(mine, ref)
    assert all(_same_bits(a, b) for a, b in zip(pools[0].gpu, pools[1].gpu))


def test_append_four_bits_of_extreme_values():
    """Zeros, subnormals, infinities and values beyond the largest factor; NaN is
    stored as some number and does not spread beyond its group."""
    k = torch.zeros(1, 1, 6, 64, dtype=torch.bfloat16)
    k[0, 0, 1] = 1e-30
    k[0, 0, 2] = 3e38
    k[0, 0, 3, 5], k[0, 0, 3, 6] = float("inf"), -float("inf")
    k[0, 0, 4] = torch.linspace(-7, 7, 64).bfloat16()
    k[0, 0, 5] = 1.0
    k[0, 0, 5, 20] = float("nan")
    codes = [torch.zeros(1, 1, 16, 32, dtype=torch.uint8, device="cuda") for _ in "kv"]
    factors = [torch.zeros(1, 1, 16, 4, dtype=torch.uint8, device="cuda") for _ in "kv"]
    kd = k.cuda()
    gb.attn_cache_append_fp4(kd, kd, codes[0], factors[0], codes[1], factors[1], _i32([[0]]), _i32([6]))
    rc, rf = pu.quantise(k[0, 0, :5].float(), 1.0)
    assert torch.equal(codes[0][0, 0, :5].cpu(), rc)
    assert torch.equal(factors[0][0, 0, :5].cpu(), rf.view(torch.uint8))
    got, _ = gb.attn_cache_gather_fp4(codes[0], factors[0], codes[1], factors[1], _i32([[0]]), _i32([6]), 6)
    row = got[0, 0, 5].float().cpu()
    assert torch.isfinite(row).all()
    keep = torch.ones(64, dtype=torch.bool)
    keep[16:32] = False
    # 1 in a group of ones: factor E4M3(1 / 6) = 0.171875, code 6
    assert (row[keep] == 6 * 0.171875).all()


@pytest.mark.parametrize("bits,dtype,d", [(16, torch.bfloat16, 128), (16, torch.float16, 64),
                                          (4, torch.bfloat16, 128), (4, torch.float16, 64)])
def test_gather(bits, dtype, d):
    g = torch.Generator().manual_seed(41)
    lens, page, Hkv = [1, 0, 77, 16, 129], 16, 3
    pool = Pool(bits, 20, Hkv, page, d, dtype, g)
    table = pu.page_table(lens, page, 20, 9, g)
    for S in (1, 100, 131):
        k, v = pool.gather(table.cuda(), _i32(lens), S)
        assert gb.gbattn_device_status() == 0
        for b, n in enumerate(lens):
            n = min(n, S)
            for i, got in enumerate((k, v)):
                assert torch.equal(got[b, :, :n].cpu(), pool.values(i, table[b], n).to(dtype))
                assert (got[b, :, n:] == 0).all()


def test_offsets_beyond_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: append to, decode from
    and read back its last pages."""
    page, Hkv, d = 1024, 2, 128
    n_pages = 8400  # 2.2e9 elements, 4.4e9 bytes
    kc, vc = (torch.empty(n_pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    g = torch.Generator().manual_seed(42)
    S, lens = 40, [40, 1040]
    table = torch.tensor([[n_pages - 1, -1], [n_pages - 2, n_pages - 3]], dtype=torch.int32)
    kc[n_pages - 3:].zero_()
    vc[n_pages - 3:].zero_()
    q, k, v = (torch.randn(2, Hkv, S, d, generator=g).bfloat16() for _ in range(3))
    gb.attn_cache_append(k.cuda(), v.cuda(), kc, vc, table.cuda(), _i32(lens))
    ka, va = gb.attn_cache_gather(kc, vc, table.cuda(), _i32(lens), 1040)
    assert torch.equal(ka[0, :, :40].cpu(), k[0]) and torch.equal(va[1, :, 1000:].cpu(), v[1])
    assert (ka[1, :, :1000] == 0).all() and (ka[0, :, 40:] == 0).all()
    qq = q[:, :, :1].contiguous().cuda()
    o, lse = gb.attn_decode_paged(qq, kc, vc, table.cuda(), _i32(lens))
    assert gb.gbattn_device_status() == 0
    for b, n in enumerate(lens):
        ro, rl, to, tl = pu.attention(q[b, :, 0], ka[b, :, :n].cpu(), va[b, :, :n].cpu(), 1 / math.sqrt(d),
                                      pu.u(torch.bfloat16) ** 2)
        assert ((o[b, :, 0].double().cpu() - ro).abs() <= to + pu.u(torch.bfloat16) * (ro.abs() + to)).all()
        assert ((lse[b].double().cpu() - rl).abs() <= tl).all()


def test_paged_decode_agrees_with_the_padded_one():
    """The same cache as pages and as a padded rectangle: both within their bounds
    of the same definition, so within the parity tests' bounds of each other."""
    from tests.parity_util import LSE_MAX_ABS, O_MAX_ABS

    g = torch.Generator().manual_seed(43)
    B, Hq, Hkv, L, d, page = 3, 8, 2, 640, 128, 64
    k, v = (torch.randn(B, Hkv, L, d, generator=g).bfloat16().cuda() for _ in "kv")
    q = torch.randn(B, Hq, 1, d, generator=g).bfloat16().cuda()
    lens = _i32([640, 333, 1])
    kc, vc = (t.unflatten(2, (L // page, page)).transpose(1, 2).flatten(0, 1).contiguous() for t in (k, v))
    table = torch.arange(B * L // page, dtype=torch.int32, device="cuda").view(B, -1)
    o1, l1, _ = gb.attn_decode_splitkv(q, k, v, lens)
    o2, l2 = gb.attn_decode_paged(q, kc, vc, table, lens)
    assert (o1.float() - o2.float()).abs().max() <= O_MAX_ABS
    assert (l1 - l2).abs().max() <= LSE_MAX_ABS


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
def test_streams_graphs_and_two_calls_at_once(bits):
    """A captured step replayed with other lengths, and two calls on two streams
    with a workspace each."""
    g = torch.Generator().manual_seed(44)
    page, Hq, Hkv, d, B = 16, 8, 2, 128, 4
    pool = Pool(bits, 80, Hkv, page, d, torch.bfloat16, g)
    table = pu.page_table([300] * B, page, 80, 19, g).cuda()
    q = torch.randn(B, Hq, 1, d, generator=g).bfloat16().cuda()
    k, v = (torch.randn(B, Hkv, 1, d, generator=g).bfloat16().cuda() for _ in "kv")
    rope = gb.rope_table(400, d)
    lens = _i32([1, 2, 3, 4])

    def step():
        qr = pool.append(k, v, table, lens, rope=rope, q=q)
        return pool.decode(qr, table, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = step()
    for new in ([1, 2, 3, 4], [300, 17, 0, 64], [65, 128, 129, 300]):
        lens.copy_(_i32(new))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        ref = step()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    other = torch.randn(B, Hq, 1, d, generator=g).bfloat16().cuda()
    refs = [pool.decode(x, table, lens) for x in (q, other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty(gb.attn_decode_paged_workspace_bytes(B, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
          for _ in streams]
    for _ in range(5):
        outs = [pool.decode(x, table, lens, workspace=w, stream=s) for x, w, s in zip((q, other), ws, streams)]
        torch.cuda.synchronize()
        for a, b in zip(outs, refs):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert gb.gbattn_device_status() == 0


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.usefixtures("table_width")
def test_calls_after_copies_fills_and_joins(bits):
    """The operators start early behind the previous kernel of their stream; here
    what they read and overwrite comes from copies, fills and other streams, eager
    and captured, and their results are read at once by the next kernel."""
    g = torch.Generator().manual_seed(45)
    B, S, Hq, Hkv, d, page, n = 8, 160, 8, 2, 64, 16, 40
    pool = Pool(bits, B * n, Hkv, page, d, torch.bfloat16, g)
    table = torch.arange(B * n, dtype=torch.int32, device="cuda").view(B, n)
    src = [torch.randn(B, h, S, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
    host = [x.cpu().pin_memory() for x in src]
    w = [1 + 0.1 * torch.randn(d, generator=g).cuda() for _ in "qk"]
    rope, lens = gb.rope_table(1024, d), _i32([600] * B)
    x = [torch.empty_like(t) for t in src]
    dw = [torch.empty(d, device="cuda") for _ in "qk"]
    side = torch.cuda.Stream()

    def run(join):
        for t in x:
            t.zero_()
        if join:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for t, h in zip(x, host):
                    t.copy_(h, non_blocking=True)
            torch.cuda.current_stream().wait_stream(side)
        else:
            for t, h in zip(x, src):
                t.copy_(h)
        q, k = gb.attn_qk_norm_rope(x[0], x[1], *w, rope=rope)
        grads = gb.attn_qk_norm_rope_bwd(q, k, x[0], x[1], *w, rope=rope, dq_weight=dw[0], dk_weight=dw[1])
        for t in x[:2]:
            t.fill_(float("nan"))
        q = pool.append(k, x[2], table, lens, q=q)
        k.fill_(float("nan"))
        x[2].zero_()
        kk, vv = pool.gather(table, lens, 640)
        o, lse = pool.decode(q[:, :, -1:].contiguous(), table, lens)
        return [t.clone() for t in (*grads, q, kk, vv, o, lse)]

    ref = run(False)
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in ref)
    for join in (False, True):
        for _ in range(10):
            assert all(torch.equal(a, b) for a, b in zip(run(join), ref))
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = run(join)
        for _ in range(10):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("bits", [16, 4])
def test_a_given_stream_owns_what_the_call_allocates(bits):
    """Work queued on the current stream right after a call on another one gets
    none of that call's memory: the decode's workspace and outputs are untouched
    by fills of the same sizes, while the other stream is still busy."""
    g = torch.Generator().manual_seed(46)
    page, Hq, Hkv, d, B = 64, 8, 2, 128, 3
    pool = Pool(bits, 40, Hkv, page, d, torch.bfloat16, g)
    lens = [700, 33, 512]
    table = pu.page_table(lens, page, 40, 11, g).cuda()
    q = torch.randn(B, Hq, 1, d, generator=g).bfloat16().cuda()
    sl = _i32(lens)
    ref = pool.decode(q, table, sl)
    side = torch.cuda.Stream()
    need = gb.attn_decode_paged_workspace_bytes(B, Hq, Hkv, d, 11 * page)
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            for _ in range(8):
                busy @ busy
        o, lse = pool.decode(q, table, sl, stream=stream)
        fills = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                 for n in (need, need, q.numel() * 2, B * Hq * 4) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
        assert all((f == 255).all() for f in fills)


def test_wrapper_refusals():
    g = torch.Generator().manual_seed(45)
    pool, pool4 = Pool(16, 3, 2, 16, 64, torch.float16, g), Pool(4, 3, 2, 16, 64, torch.float16, g)
    table, lens = _i32([[0, 1]]), _i32([20])
    q = torch.zeros(1, 4, 1, 64, dtype=torch.float16, device="cuda")
    k = torch.zeros(1, 2, 1, 64, dtype=torch.float16, device="cuda")
    bad = [
        lambda: gb.attn_decode_paged(q.bfloat16(), *pool.gpu, table, lens),
        lambda: gb.attn_decode_paged(q.expand(1, 4, 2, 64), *pool.gpu, table, lens),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table.long(), lens),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table, lens.float()),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table[:, :1].expand(2, 1), lens),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table.cpu(), lens),
        lambda: gb.attn_decode_paged(q, pool.gpu[0], pool.gpu[1][:2], table, lens),
        lambda: gb.attn_decode_paged(q, pool.gpu[0][..., :32], pool.gpu[1][..., :32], table, lens),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table, lens, lse=torch.zeros(4, device="cuda")),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table, lens, out=q.float()),
        lambda: gb.attn_decode_paged(q[:, :3], *pool.gpu, table, lens),
        lambda: gb.attn_decode_paged(q, *pool.gpu, table, lens, workspace=torch.empty(16, device="cuda")),
        lambda: gb.attn_decode_paged_fp4(q, *pool4.gpu[:3], None, table, lens),
        lambda: gb.attn_decode_paged_fp4(q, pool4.gpu[0], pool4.gpu[1][..., :2], *pool4.gpu[2:], table, lens),
        lambda: gb.attn_decode_paged_fp4(q, *pool4.gpu, table, lens, k_descale=torch.ones(3, device="cuda")),
        lambda: gb.attn_cache_append(k, k[:, :1], *pool.gpu, table, lens),
        lambda: gb.attn_cache_append(k, k, *pool.gpu, table, lens, q_out=q),
        lambda: gb.attn_cache_append(k, k, *pool.gpu, table, lens, q=q[:, :3]),
        lambda: gb.attn_cache_append(k, k, *pool.gpu, table, lens, rope=torch.zeros(40, 24, device="cuda")),
        lambda: gb.attn_cache_append(k, k, *pool.gpu, table, lens, new_lens=_i32([1, 1])),
        lambda: gb.attn_cache_append(k, k, pool.gpu[0][:, :, :8], pool.gpu[1][:, :, :8], table, lens),
        lambda: gb.attn_cache_gather(*pool.gpu, table, lens, 0),
        lambda: gb.attn_cache_gather_fp4(*pool4.gpu, table, lens, 4, dtype=torch.float32),
        lambda: gb.attn_cache_gather(*pool.gpu, table, _i32([[20]]), 4),
    ]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, gb.GbattnError)):
            f()
            pytest.fail(f"call {i} was not refused")
    assert gb.gbattn_device_status() == 0


@pytest.mark.usefixtures("table_width")
@pytest.mark.parametrize("bits", [16, 4])
def test_a_prompt_in_chunks_and_then_tokens(bits):
    """As a program runs them: a prompt in two chunks (norm and rotation, append,
    read-back, attn_fwd), then three tokens of decode, against the same network
    piece in 64 bits.  The bounds follow the kernels' own 16-bit intermediates:
    each step is compared with the definition applied to what the previous step
    gave, so no error is counted twice."""
    g = torch.Generator().manual_seed(50)
    B, H, Hkv, d, page, dtype = 2, 4, 2, 64, 16, torch.bfloat16
    pool = Pool(bits, 24, Hkv, page, d, dtype, g)
    table_h = pu.page_table([90] * B, page, 24, 6, g)
    table = table_h.cuda()
    rope = gb.rope_table(96, d)
    w = [1 + 0.1 * torch.randn(d, generator=g) for _ in "qk"]
    wd = [x.cuda() for x in w]
    done, scale = 0, 1 / math.sqrt(d)
    for S in (50, 29, 1, 1, 1):
        x = torch.randn(B, S, H + 2 * Hkv, d, generator=g).to(dtype).cuda().transpose(1, 2)
        q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        pos = (done + torch.arange(S, dtype=torch.int32, device="cuda")).expand(B, S).contiguous()
        qn, kn = gb.attn_qk_norm_rope(q, k, *wd, rope=rope, positions=pos)
        done += S
        lens = _i32([done] * B)
        pool.append(kn, v, table, lens)
        pool.pull()
        if S > 1:
            kk, vv = pool.gather(table, lens, done)
            o, lse = gb.attn_fwd(qn, kk, vv, causal=True)
        else:
            o, lse = pool.decode(qn, table, lens)
        assert gb.gbattn_device_status() == 0
        for b in range(B):
            for i, (raw, got) in enumerate(((q, qn), (k, kn))):
                ref, mag = pu.norm_rope(raw[b].double().cpu(), w[i].double(), rope.cpu(), pos[b].long().cpu(), 1e-6, False)
                err = (got[b].double().cpu() - ref).abs()
                assert (err <= pu.u(dtype) * ref.abs() + 20 * pu.U32 * mag).all()
            if bits == 16:
                assert torch.equal(pool.values(0, table_h[b], done)[:, -S:], kn[b].float().cpu())
            for t in range(S):  # query t of the chunk sees done - S + t + 1 tokens
                n = done - S + t + 1
                kv = [pool.values(i, table_h[b], n) for i in range(2)]
                if S > 1:  # what attn_fwd read: the values rounded to 16 bits
                    kv = [x.to(dtype).float() for x in kv]
                half_p = pu.u(dtype) if S > 1 else pu.u(torch.float16) if bits == 4 else pu.u(dtype) ** 2
                ro, rl, to, tl = pu.attention(qn[b, :, t].cpu(), *kv, scale, half_p, 2.0 ** -24, bits == 4)
                err = (o[b, :, t].double().cpu() - ro).abs()
                assert (err <= to + pu.u(dtype) * (ro.abs() + to)).all(), f"{S} tokens, query {t}: {err.max():.3e}"
                got = lse[b].view(H, -1)[:, t].double().cpu()
                assert ((got - rl).abs() <= tl).all()
