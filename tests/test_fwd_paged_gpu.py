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


def _forward(pool, q, table, lens, news, **kw):
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
