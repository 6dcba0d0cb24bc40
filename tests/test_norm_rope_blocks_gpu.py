"""attn_qk_norm_rope and its backward where a CTA walks on to further token blocks
(more tokens than the grid covers at once, the last block ragged): rows that the
ring requests across a block's end, angles read again for each block, and weight
gradients summed over several blocks.  All rows against the plain forms in 64
bits, which run on the GPU here."""
import pytest
import torch

import exact_tiled_attention_gb300 as gb
from tests import paged_util as pu

pytestmark = pytest.mark.gpu
EPS = 1e-6
B, H, HKV = 3, 128, 16  # 18 chunks of heads forward, 9 backward: grids of 541 and 128 CTAs over the tokens
S = {128: 3501, 64: 6507}  # blocks of 16 and of 32 tokens: 657 and 611 of them


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("rot,interleaved", [(1.0, False), (0.5, False), (0.5, True)])
@pytest.mark.parametrize("d,dtype", [(128, torch.bfloat16), (64, torch.float16)])
def test_rows_of_later_token_blocks(d, dtype, rot, interleaved, norm):
    g = torch.Generator(device="cuda").manual_seed(71)
    s, rot = S[d], int(rot * d)
    x = torch.randn(B, s, H + HKV, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    xs = x[:, :H], x[:, H:]
    dy = [torch.randn(B, h, s, d, generator=g, device="cuda").to(dtype) for h in (H, HKV)]
    w = [1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in "qk"] if norm else [None, None]
    rope = gb.rope_table(2 * s, rot)
    pos = torch.randint(0, 2 * s, (B, s), generator=g, device="cuda", dtype=torch.int32)
    args = dict(rope=rope, positions=pos, eps=EPS, interleaved=interleaved)
    outs = gb.attn_qk_norm_rope(*xs, *w, **args)
    grads = gb.attn_qk_norm_rope_bwd(*dy, *xs, *w, **args)
    assert gb.gbattn_device_status() == 0

    def check(got, ref, mag, ops, what):
        tol = pu.u(dtype) * ref.abs() + ops * pu.U32 * mag + torch.finfo(dtype).smallest_normal * pu.u(dtype)
        over = (got.double() - ref).abs() - tol
        assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound"  # a NaN fails too

    for i, y in enumerate(outs):
        wi = None if w[i] is None else w[i].double()
        dw, mag_dw = 0.0, 0.0
        for b in range(B):
            p = pos[b].long()
            for h in range(0, y.shape[1], 32):
                part = slice(h, h + 32)
                xd, dyd = xs[i][b, part].double(), dy[i][b, part].double()
                check(y[b, part], *pu.norm_rope(xd, wi, rope, p, EPS, interleaved), 20, f"output {i}, sequence {b}")
                dx, dwb, mag_dx, magb = pu.norm_rope_bwd(dyd, xd, wi, rope, p, EPS, interleaved)
                check(grads[i][b, part], dx, mag_dx, 64, f"gradient {i}, sequence {b}")
                if norm:
                    dw, mag_dw = dw + dwb, mag_dw + magb
        if norm:
            # Terms within 24 roundings.  Sums: a thread's blocks (at most 6) of 16 heads
            # one after another, 2 or 3 steps over the lanes, 4 warps, then for each
            # column 16 of the 1024 partials and 6 steps.
            err = (grads[2 + i].double() - dw).abs()
            assert (err <= (24 + 6 * 16 + 3 + 4 + 16 + 6) * pu.U32 * mag_dw).all(), f"weight gradient {i}: {err.max():.3e}"
