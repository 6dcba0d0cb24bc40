"""Rotation by positions of several axes on the GPU: norms and rotation with their
backward, and the appends, against the plain forms in 64 bits (bounds in
paged_util), which see a table made of each pair's own axis's angles, and bit for
bit against the rotation by one position over that same table."""
import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300.binding import GBATTN_EINDEX
from tests import paged_util as pu
from tests.test_norm_rope_gpu import EPS, _check
from tests.test_paged_gpu import Pool, _i32, _same_bits

pytestmark = pytest.mark.gpu


def _axes(kind, rot, n_axes, g):
    """The pairs' axes: sections one behind another, in turn, or at random."""
    pairs = rot // 2
    if kind == "random":
        return tuple(torch.randint(0, n_axes, (pairs,), generator=g).tolist())
    cuts = [pairs // n_axes] * n_axes
    cuts[0] += pairs - sum(cuts)
    return gb.rope_pair_axes(cuts, cycle=kind == "cycle")


def _own_table(table, pos, axes):
    """The rows that the tokens of pos [n_axes, ..., S] turn by: [..., S, rot]."""
    half = table.shape[1] // 2
    at = torch.stack([pos[a] for a in axes], -1).long()
    i = torch.arange(half)
    return torch.cat([table[at, i], table[at, half + i]], -1)


CASES = [
    # B, S, H, Hkv, d, dtype, rot, interleaved, n_axes, kind, norm
    (1, 1, 1, 1, 128, torch.bfloat16, 128, False, 3, "sections", True),
    (3, 7, 4, 2, 128, torch.bfloat16, 128, False, 3, "cycle", True),
    (2, 33, 8, 1, 64, torch.float16, 64, False, 2, "sections", False),
    (2, 5, 6, 3, 64, torch.bfloat16, 32, False, 4, "random", True),
    (1, 17, 4, 4, 128, torch.float16, 96, False, 3, "sections", False),
    (2, 9, 10, 5, 128, torch.float16, 16, True, 2, "cycle", True),
    (5, 3, 2, 1, 64, torch.float16, 64, True, 4, "sections", True),
    (2, 31, 4, 2, 64, torch.bfloat16, 48, False, 1, "sections", False),
    (1, 31, 4, 2, 128, torch.float16, 128, True, 3, "random", False),
    (2, 700, 16, 16, 128, torch.bfloat16, 128, False, 3, "sections", True),
]


def _tensors(cfg, seed=41):
    B, S, H, Hkv, d, dtype, rot, _, n_axes, kind, norm = cfg
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, H + 2 * Hkv, d, generator=g).to(dtype).cuda().transpose(1, 2)
    w = [1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)] if norm else [None, None]
    table = gb.rope_table(90, rot, device="cpu")
    pos = torch.randint(0, 90, (n_axes, B, S), generator=g, dtype=torch.int32)
    dy = [torch.randn(B, h, S, d, generator=g).to(dtype).cuda() for h in (H, Hkv)]
    wd = [None if t is None else t.cuda() for t in w]
    return x[:, :H], x[:, H:H + Hkv], w, wd, table, pos, _axes(kind, rot, n_axes, g), dy


@pytest.mark.parametrize("cfg", CASES)
def test_forward_and_backward(cfg):
    B, S, H, Hkv, d, dtype, rot, interleaved, n_axes, kind, norm = cfg
    q, k, w, wd, table, pos, axes, dy = _tensors(cfg)
    kw = dict(eps=EPS, interleaved=interleaved)
    own = dict(rope=table.cuda(), positions=pos.cuda(), axes=axes, **kw)
    outs = gb.attn_qk_norm_rope(q, k, *wd, **own)
    grads = gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, **own)
    assert gb.gbattn_device_status() == 0
    each = _own_table(table, pos, axes)
    one = dict(rope=each.flatten(0, 1).cuda(), positions=torch.arange(B * S, dtype=torch.int32).view(B, S).cuda(), **kw)
    for a, b in zip(outs + grads, gb.attn_qk_norm_rope(q, k, *wd, **one) + gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, **one)):
        assert (a is None and b is None) or torch.equal(a, b)
    for i, x in enumerate((q, k)):
        wi = None if w[i] is None else w[i].double()
        for b in range(B):
            xd, p = x[b].double().cpu(), torch.arange(S)
            y, mag = pu.norm_rope(xd, wi, each[b], p, EPS, interleaved)
            _check(outs[i][b], y, mag, dtype, 20, f"output {i} of sequence {b}")
            dx, _, mag_dx, _ = pu.norm_rope_bwd(dy[i][b].double().cpu(), xd, wi, each[b], p, EPS, interleaved)
            _check(grads[i][b], dx, mag_dx, dtype, 64, f"gradient {i} of sequence {b}")


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(interleaved):
    """As for one position: directional derivatives of the 64-bit forward against
    the kernel's gradients, each off by at most u of its magnitude."""
    cfg = (2, 6, 3, 1, 64, torch.float16, 32, interleaved, 3, "cycle", True)
    q, k, w, wd, table, pos, axes, dy = _tensors(cfg)
    grads = gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, rope=table.cuda(), positions=pos.cuda(), axes=axes, eps=EPS,
                                     interleaved=interleaved)
    each, p, g = _own_table(table, pos, axes), torch.arange(6), torch.Generator().manual_seed(6)
    for i, x in enumerate((q, k)):
        xd, wi, dyi = x.double().cpu(), w[i].double(), dy[i].double().cpu()

        def f(x, w):
            return sum((pu.norm_rope(x[b], w, each[b], p, EPS, interleaved)[0] * dyi[b]).sum() for b in range(2))

        mag = torch.stack([pu.norm_rope_bwd(dyi[b], xd[b], wi, each[b], p, EPS, interleaved)[2] for b in range(2)])
        for _ in range(3):
            e, ew = torch.randn(xd.shape, generator=g, dtype=torch.float64), torch.randn(64, generator=g, dtype=torch.float64)
            h = 1e-5
            slope = (f(xd + h * e, wi + h * ew) - f(xd - h * e, wi - h * ew)) / (2 * h)
            got = (grads[i].double().cpu() * e).sum() + (grads[2 + i].double().cpu() * ew).sum()
            assert abs(slope - got) <= pu.u(torch.float16) * (mag * e.abs()).sum() + 1e-4


APPEND = [
    # dtype, B, S, H (0: no q), Hkv, d, page, rot, interleaved, n_axes, kind (None: positions of one axis)
    (torch.bfloat16, 3, 1, 8, 2, 128, 64, 128, False, 3, "sections"),
    (torch.float16, 5, 37, 6, 3, 64, 16, 32, True, 2, "cycle"),
    (torch.bfloat16, 4, 70, 0, 1, 128, 32, 96, False, 4, "random"),
    (torch.bfloat16, 2, 200, 16, 8, 128, 64, 128, False, 3, "cycle"),
    (torch.float16, 2, 9, 4, 4, 64, 1024, 64, False, 1, None),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("cfg", APPEND)
def test_append(cfg, bits):
    """What is stored (bit for bit), the queries, and that every other slot keeps its bits."""
    dtype, B, S, H, Hkv, d, page, rot, interleaved, n_axes, kind = cfg
    g = torch.Generator().manual_seed(42)
    new = [min(S, (S, 1, 0, S - 1, 2)[i % 5]) for i in range(B)]
    lens = [n + (0, 13, 64, 5, 200)[i % 5] for i, n in enumerate(new)]
    width = max((n + page - 1) // page for n in lens) + 1
    n_pages = sum((n + page - 1) // page for n in lens) + 2
    pool = Pool(bits, n_pages, Hkv, page, d, dtype, g)
    table = pu.page_table(lens, page, n_pages, width, g)
    x = torch.randn(B, S, H + 2 * Hkv, d, generator=g).to(dtype).cuda().transpose(1, 2)
    q, k, v = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    rope = gb.rope_table(50, rot, device="cpu")
    pos = torch.randint(0, 50, (n_axes, B, S), generator=g, dtype=torch.int32)
    axes = _axes(kind, rot, n_axes, g) if kind else None
    given = pos.clone()
    for b, m in enumerate(new):
        given[:, b, m:] = -7  # positions of padding are not looked at
    out = pool.append(k, v, table.cuda(), _i32(lens), new_lens=_i32(new), rope=rope.cuda(), interleaved=interleaved,
                      q=q if H else None, positions=(given if kind else given[0]).cuda(), axes=axes)
    assert gb.gbattn_device_status() == 0
    before = [t.clone() for t in pool.t]
    pool.pull()
    each = _own_table(rope, pos, axes or (0,) * (rot // 2))
    for b, (n, m) in enumerate(zip(lens, new)):
        i, at = torch.arange(m), torch.arange(n - m, n)
        kb, vb, qb = (t[b, :, :m].cpu() for t in (k, v, q))
        if H:
            ob = out[b].double().cpu()
            ref, mag = pu.turn(qb.double(), each[b], i, interleaved)
            tol = pu.u(dtype) * ref.abs() + 3 * pu.U32 * mag + 2.0 ** -25
            assert ((ob[:, :m] - ref).abs() <= tol).all() and (ob[:, m:] == 0).all()
        pages, rows = table[b][at // page].long(), at % page
        k32 = pu.turn(kb.float(), each[b], i, interleaved)[0]
        if bits == 16:
            for j, ref in enumerate((k32.to(dtype), vb)):
                assert torch.equal(pool.t[j][pages, :, rows], ref.transpose(0, 1))
                before[j][pages, :, rows] = pool.t[j][pages, :, rows]
        else:
            for j, ref in enumerate((k32, vb.float())):
                codes, f = pu.quantise(ref, pool.descale[j][:, None])
                assert torch.equal(pool.t[2 * j][pages, :, rows], codes.transpose(0, 1))
                got = pool.t[2 * j + 1].view(torch.uint8)
                assert torch.equal(got[pages, :, rows], f.view(torch.uint8).transpose(0, 1))
                before[2 * j][pages, :, rows] = pool.t[2 * j][pages, :, rows]
                before[2 * j + 1].view(torch.uint8)[pages, :, rows] = got[pages, :, rows]
    assert all(_same_bits(a, b) for a, b in zip(before, pool.t))


def test_positions_outside_the_table_are_reported():
    q = torch.randn(2, 4, 3, 64, device="cuda", dtype=torch.float16)
    rope = gb.rope_table(8, 64)
    axes = gb.rope_pair_axes((16, 8, 8))
    pos = torch.zeros(3, 2, 3, dtype=torch.int32, device="cuda")
    good = gb.attn_qk_norm_rope(q, q, rope=rope, positions=pos + 7, axes=axes)
    assert gb.gbattn_device_status() == 0
    pos += 7
    pos[2, 1, 2] = 8
    out = gb.attn_qk_norm_rope(q, q, rope=rope, positions=pos, axes=axes)
    assert gb.gbattn_device_status() == GBATTN_EINDEX and gb.gbattn_device_status() == 0
    assert torch.equal(out[0], good[0])
    pool = Pool(16, 4, 4, 16, 64, torch.float16, torch.Generator().manual_seed(1))
    pool.append(q, q, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), _i32([3, 0]), rope=rope, positions=pos,
                axes=axes)  # the second sequence's tokens are padding
    assert gb.gbattn_device_status() == 0
    pos[0, 0, 1] = -1
    pool.append(q, q, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), _i32([3, 0]), rope=rope, positions=pos,
                axes=axes)
    assert gb.gbattn_device_status() == GBATTN_EINDEX and gb.gbattn_device_status() == 0


def test_wrapper_refusals():
    q = torch.randn(2, 4, 3, 64, device="cuda", dtype=torch.float16)
    rope = gb.rope_table(8, 64)
    pos = torch.zeros(3, 2, 3, dtype=torch.int32, device="cuda")
    axes = gb.rope_pair_axes((16, 8, 8))
    for bad in (dict(axes=axes[:-1]), dict(axes=axes + (0,)), dict(axes=(3,) * 32), dict(axes=(-1,) * 32),
                dict(positions=None), dict(positions=pos[0]), dict(positions=pos[:, :1]), dict(positions=pos.cpu()),
                dict(positions=pos[:0]), dict(positions=torch.zeros(5, 2, 3, dtype=torch.int32, device="cuda")),
                dict(rope=None)):
        with pytest.raises(ValueError):
            gb.attn_qk_norm_rope(q, q, **dict(dict(rope=rope, positions=pos, axes=axes), **bad))
    for bad in (dict(axes=5), dict(axes=(0.5,) * 32), dict(positions=pos.long())):
        with pytest.raises(TypeError):
            gb.attn_qk_norm_rope(q, q, **dict(dict(rope=rope, positions=pos, axes=axes), **bad))
    pool = Pool(16, 4, 4, 16, 64, torch.float16, torch.Generator().manual_seed(1))
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for bad in (dict(axes=axes), dict(positions=pos), dict(positions=pos[0], rope=None)):
        with pytest.raises(ValueError):
            pool.append(q, q, table, _i32([3, 3]), **dict(dict(rope=rope), **bad))
    assert gb.gbattn_device_status() == 0


def test_axes_whose_entries_run_code():
    """Entries are whatever has an index; a list that one of them empties counts as it
    was, and one that raises ends the call."""
    q = torch.randn(2, 4, 3, 64, device="cuda", dtype=torch.float16)
    kw = dict(rope=gb.rope_table(8, 64), positions=torch.randint(0, 8, (3, 2, 3), dtype=torch.int32, device="cuda"))
    axes = gb.rope_pair_axes((16, 8, 8))
    ref = gb.attn_qk_norm_rope(q, q, axes=axes, **kw)

    class Entry:
        def __init__(self, value, act):
            self.value, self.act = value, act

        def __index__(self):
            self.act()
            return self.value

    entries = []
    entries += [Entry(a, entries.clear) for a in axes]
    out = gb.attn_qk_norm_rope(q, q, axes=entries, **kw)
    assert not entries and all(torch.equal(a, b) for a, b in zip(out, ref))

    def fail():
        raise KeyError("entry")

    with pytest.raises(KeyError):
        gb.attn_qk_norm_rope(q, q, axes=[*axes[:-1], Entry(0, fail)], **kw)
    pool = Pool(16, 4, 4, 16, 64, torch.float16, torch.Generator().manual_seed(1))
    entries += [Entry(a, entries.clear) for a in axes]
    back = pool.append(q, q, torch.zeros(2, 1, dtype=torch.int32, device="cuda"), _i32([3, 0]), q=q, axes=entries, **kw)
    assert not entries and torch.equal(back[0], ref[0][0]) and gb.gbattn_device_status() == 0


def test_streams_and_graph():
    cfg = (2, 33, 8, 2, 128, torch.bfloat16, 128, False, 3, "sections", True)
    q, k, w, wd, table, pos, axes, dy = _tensors(cfg)
    kw = dict(rope=table.cuda(), positions=pos.cuda(), axes=axes, eps=EPS)
    ref = gb.attn_qk_norm_rope(q, k, *wd, **kw) + gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = gb.attn_qk_norm_rope(q, k, *wd, **kw, stream=side) + gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, **kw, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gb.attn_qk_norm_rope(q, k, *wd, **kw) + gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, **kw)
    kw["positions"].copy_((pos + 1) % 90)  # a captured graph follows the positions
    graph.replay()
    ref = gb.attn_qk_norm_rope(q, k, *wd, **kw) + gb.attn_qk_norm_rope_bwd(*dy, q, k, *wd, **kw)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
