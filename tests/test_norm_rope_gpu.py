"""attn_qk_norm_rope and its backward on the GPU against their plain forms in 64
bits (bounds in paged_util): head sizes, types, rotations, odd lengths, views of
a projection output, scattered positions, in-place outputs, gradients against
differences, streams, graph capture and repeated runs."""
import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300.binding import GBATTN_EINDEX
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _case(B, S, H, Hkv, d, dtype, rot, seed, fused=True, far=0, norm=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, S, H + 2 * Hkv, d, generator=g).to(dtype)
    qk = x.cuda().transpose(1, 2)
    q, k = qk[:, :H], qk[:, H:H + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    w = [1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)] if norm else [None, None]
    rows = far + S
    pos = torch.randint(0, rows, (B, S), generator=g, dtype=torch.int32) if far else None
    table = gb.rope_table(rows, rot, device="cpu") if rot else None
    dy = [torch.randn(B, h, S, d, generator=g).to(dtype) for h in (H, Hkv)]
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    return q, k, w, table, pos, dy, [cuda(t) for t in w], cuda(table), cuda(pos), [t.cuda() for t in dy]


def _check(got, ref, mag, dtype, ops, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    tol = pu.u(dtype) * ref.abs() + ops * pu.U32 * mag + torch.finfo(dtype).smallest_normal * pu.u(dtype)
    bad = (got - ref).abs() - tol
    assert (bad <= 0).all(), f"{what}: {bad.max():.3e} over the bound"


SHAPES = [
    # B, S, H, Hkv, d, dtype, rot, interleaved, far, norm
    (1, 1, 1, 1, 128, torch.bfloat16, 128, False, 0, True),
    (3, 7, 4, 2, 128, torch.bfloat16, 128, False, 0, True),
    (2, 33, 8, 1, 64, torch.float16, 64, False, 100, True),
    (2, 5, 6, 3, 64, torch.bfloat16, 32, False, 0, True),
    (1, 17, 4, 4, 128, torch.float16, 96, False, 0, True),
    (2, 9, 10, 5, 128, torch.float16, 16, True, 50, True),
    (5, 3, 2, 1, 64, torch.float16, 64, True, 0, True),
    (2, 65, 12, 4, 128, torch.bfloat16, 0, False, 0, True),
    (2, 31, 4, 2, 128, torch.float16, 128, False, 9, False),
    (2, 31, 4, 2, 64, torch.bfloat16, 48, False, 0, False),
    (1, 31, 4, 2, 64, torch.float16, 32, True, 0, False),
    (2, 700, 16, 16, 128, torch.bfloat16, 128, False, 0, True),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("cfg", SHAPES)
def test_forward_and_backward(cfg, fused):
    B, S, H, Hkv, d, dtype, rot, interleaved, far, norm = cfg
    q, k, w, table, pos, dy, wd, td, pd, dyd = _case(B, S, H, Hkv, d, dtype, rot, 1, fused, far, norm)
    outs = gb.attn_qk_norm_rope(q, k, *wd, rope=td, positions=pd, eps=EPS, interleaved=interleaved)
    grads = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td, positions=pd, eps=EPS, interleaved=interleaved)
    torch.cuda.synchronize()
    assert gb.gbattn_device_status() == 0
    for i, x in enumerate((q, k)):
        wi = None if w[i] is None else w[i].double()
        dw, mag_dw = 0.0, 0.0
        for b in range(B):
            p = torch.arange(S) if pos is None else pos[b].long()
            xd = x[b].double().cpu()
            y, mag = pu.norm_rope(xd, wi, table, p, EPS, interleaved)
            _check(outs[i][b], y, mag, dtype, 20, f"output {i} of sequence {b}")
            dx, dwb, mag_dx, magb = pu.norm_rope_bwd(dy[i][b].double(), xd, wi, table, p, EPS, interleaved)
            # g rounds 4 times; n, its products and the mean (16 fused adds, 4 tree steps) below 40 together.
            _check(grads[i][b], dx, mag_dx, dtype, 64, f"gradient {i} of sequence {b}")
            if norm:
                dw, mag_dw = dw + dwb, mag_dw + magb
        if norm:
            # A chain of at most B S heads adds, each term within 24 roundings.
            n = B * S * x.shape[1]
            err = (grads[2 + i].double().cpu() - dw).abs()
            assert (err <= (n + 64) * pu.U32 * mag_dw).all(), f"weight gradient {i}: {err.max():.3e}"
        else:
            assert grads[2 + i] is None


def test_gradients_against_differences():
    """Directional derivatives of the 64-bit forward (central differences, error
    below 1e-6 of the sum's scale) against the kernel's gradients, each of which
    is off by at most u relative to its magnitude: u sum |mag e| bounds both."""
    B, S, H, Hkv, d, dtype, rot = 2, 6, 3, 1, 64, torch.float16, 32
    q, k, w, table, _, dy, wd, td, _, dyd = _case(B, S, H, Hkv, d, dtype, rot, 5)
    dq, dk, dqw, dkw = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td, eps=EPS)
    p = torch.arange(S)
    g = torch.Generator().manual_seed(6)
    for i, (x, dx, dw) in enumerate(((q, dq, dqw), (k, dk, dkw))):
        xd, wi, dyi = x.double().cpu(), w[i].double(), dy[i].double()

        def f(x, w):
            return sum((pu.norm_rope(x[b], w, table, p, EPS, False)[0] * dyi[b]).sum() for b in range(B))

        mag = torch.stack([pu.norm_rope_bwd(dyi[b], xd[b], wi, table, p, EPS, False)[2] for b in range(B)])
        for _ in range(4):
            e, ew = torch.randn(xd.shape, generator=g, dtype=torch.float64), torch.randn(d, generator=g, dtype=torch.float64)
            h = 1e-5
            slope = (f(xd + h * e, wi + h * ew) - f(xd - h * e, wi - h * ew)) / (2 * h)
            got = (dx.double().cpu() * e).sum() + (dw.double().cpu() * ew).sum()
            assert abs(slope - got) <= pu.u(dtype) * (mag * e.abs()).sum() + 1e-4


def test_in_place_and_given_outputs():
    q, k, _, _, _, dy, wd, td, _, dyd = _case(2, 40, 6, 2, 128, torch.bfloat16, 96, 8, fused=False)
    ref = gb.attn_qk_norm_rope(q, k, *wd, rope=td)
    q2, k2 = q.clone(), k.clone()
    out = gb.attn_qk_norm_rope(q2, k2, *wd, rope=td, q_out=q2, k_out=k2)
    assert out[0] is q2 and torch.equal(q2, ref[0]) and torch.equal(k2, ref[1])
    # gradients straight into a projection output's gradient; its other part stays
    buf = torch.full((2, 40, 10, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    view = buf.transpose(1, 2)
    ws = torch.empty(gb.attn_qk_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    ref = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td)
    got = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td, dq=view[:, :6], dk=view[:, 6:8], workspace=ws)
    assert torch.equal(view[:, :6], ref[0]) and torch.equal(view[:, 6:8], ref[1])
    assert (view[:, 8:] == 7.0).all()
    assert torch.equal(got[2], ref[2]) and torch.equal(got[3], ref[3])  # repeats bitwise


def test_strides_of_single_rows_and_shared_ones():
    """The stride of a dimension of one says nothing: a tensor is not refused for
    it.  Inputs may repeat rows by a stride of 0; outputs whose rows share memory
    are refused."""
    q, k, _, _, _, _, wd, td, _, dyd = _case(3, 1, 4, 2, 64, torch.bfloat16, 64, 13)
    ref = gb.attn_qk_norm_rope(q, k, *wd, rope=td)
    ref_bwd = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td)
    buf = torch.empty(3, 8, 64, dtype=torch.bfloat16, device="cuda")
    odd = torch.as_strided(buf, (3, 4, 1, 64), (512, 64, 1, 1))
    odd.copy_(q)
    got = gb.attn_qk_norm_rope(odd, k, *wd, rope=td)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    got = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td, dq=torch.as_strided(buf, (3, 4, 1, 64), (512, 64, 1, 1)))
    assert torch.equal(got[0], ref_bwd[0])
    got = gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td, dk=buf[:, ::3][:, :2].unsqueeze(2))
    assert torch.equal(got[1], ref_bwd[1])
    got = gb.attn_qk_norm_rope(q[:1].expand(3, -1, -1, -1), k, *wd, rope=td)
    assert all(torch.equal(got[0][b], ref[0][0]) for b in range(3))
    for strides in ((0, 64, 64, 1), (512, 0, 64, 1), (512, 32, 64, 1), (128, 64, 64, 1)):
        with pytest.raises(ValueError, match="share memory"):
            gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td, dq=torch.as_strided(buf, (3, 4, 1, 64), strides))


def test_zero_rows_and_extreme_values():
    """A zero row's norm is eps^-1/2 and its output 0; rows of the largest fp16
    values have a finite norm; a NaN stays in its own row."""
    q, k, w, table, _, _, wd, td, _, _ = _case(1, 4, 2, 1, 64, torch.float16, 64, 9, fused=False)
    q[0, 0, 0] = 0
    q[0, 0, 1] = 65504.0
    q[0, 1, 2, 5] = float("nan")
    y, _ = gb.attn_qk_norm_rope(q, k, *wd, rope=td, eps=EPS)
    assert (y[0, 0, 0] == 0).all()
    ref, mag = pu.norm_rope(q[0, 0, 1:2].double().cpu()[None], w[0].double(), table, torch.tensor([1]), EPS, False)
    _check(y[0, 0, 1:2][None], ref, mag, torch.float16, 20, "largest values")
    assert torch.isnan(y[0, 1, 2]).all()
    y[0, 1, 2] = 0
    assert torch.isfinite(y).all()


def test_positions_outside_the_table_are_reported():
    q, k, _, _, _, _, wd, td, _, _ = _case(1, 3, 2, 1, 64, torch.bfloat16, 64, 10)
    gb.gbattn_device_status()
    pos = torch.tensor([[-1, 2, 3]], dtype=torch.int32, device="cuda")
    got = gb.attn_qk_norm_rope(q, k, *wd, rope=td, positions=pos)
    assert gb.gbattn_device_status() == GBATTN_EINDEX
    assert gb.gbattn_device_status() == 0
    clamped = torch.tensor([[0, 2, 2]], dtype=torch.int32, device="cuda")
    ref = gb.attn_qk_norm_rope(q, k, *wd, rope=td, positions=clamped)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert gb.gbattn_device_status() == 0


def test_wrapper_refusals():
    q, k, _, _, _, dy, wd, td, _, dyd = _case(1, 3, 2, 1, 64, torch.bfloat16, 64, 10)
    for kw in (dict(k=k.half()), dict(k_weight=None), dict(q_weight=wd[0].half()), dict(rope=td[:2]),
               dict(rope=td.double()), dict(positions=torch.zeros(1, 3, dtype=torch.int64, device="cuda")),
               dict(rope=None, q_weight=None, k_weight=None), dict(q=q[..., ::2]), dict(q=q.float()),
               dict(k=k[:, :, :2]), dict(q_weight=wd[0].cpu())):
        a = dict(q=q, k=k, q_weight=wd[0], k_weight=wd[1], rope=td)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            gb.attn_qk_norm_rope(**a)
    with pytest.raises(gb.GbattnError):
        gb.attn_qk_norm_rope(q, k, *wd, rope=gb.rope_table(3, 8))  # 8: no multiple of 16
    with pytest.raises((TypeError, ValueError)):
        gb.attn_qk_norm_rope_bwd(dyd[0][:, :1], dyd[1], q, k, *wd, rope=td)
    with pytest.raises(gb.GbattnError):
        gb.attn_qk_norm_rope_bwd(*dyd, q, k, *wd, rope=td,
                                 workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_streams_and_graph():
    """Captured once, replayed with other inputs; an eager call of the same
    tensors between the replays; a side stream."""
    q, k, _, _, _, _, wd, td, _, dyd = _case(2, 50, 4, 2, 128, torch.bfloat16, 128, 11, fused=False)
    q2, k2, *_ = _case(2, 50, 4, 2, 128, torch.bfloat16, 128, 12, fused=False)
    args = dict(rope=td)
    ref = [(*gb.attn_qk_norm_rope(a, b, *wd, **args), *gb.attn_qk_norm_rope_bwd(*dyd, a, b, *wd, **args))
           for a, b in ((q, k), (q2, k2))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    qs, ks = q.clone(), k.clone()
    with torch.cuda.graph(graph, stream=side):
        got = (*gb.attn_qk_norm_rope(qs, ks, *wd, **args), *gb.attn_qk_norm_rope_bwd(*dyd, qs, ks, *wd, **args))
    for i, (a, b) in enumerate(((q, k), (q2, k2), (q, k))):
        qs.copy_(a)
        ks.copy_(b)
        graph.replay()
        eager = (*gb.attn_qk_norm_rope(qs, ks, *wd, **args), *gb.attn_qk_norm_rope_bwd(*dyd, qs, ks, *wd, **args))
        torch.cuda.synchronize()
        for x, y, z in zip(got, ref[i % 2], eager):
            assert torch.equal(x, y) and torch.equal(z, y)
    torch.cuda.synchronize()
    out = gb.attn_qk_norm_rope(q, k, *wd, **args, stream=side)
    side.synchronize()
    assert torch.equal(out[0], ref[0][0])
