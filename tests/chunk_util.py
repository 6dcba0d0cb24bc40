"""Plain 64-bit form of the attention of a chunk of new tokens over a paged cache,
on the CPU, and the bound that the tests hold the kernels to.

The bound counts roundings as paged_util does for the decode: the weights are
rounded to one 16-bit term, relative error half_p (with fp16 terms also 2^-25 of
the largest, which is at least 1 before the division); a score is a sum of d exact
products, each add within 2 U32 of the running magnitude; exp2, its argument and
the rescalings are below 2^-20 of a weight together.  The sum of weights is not
rounded with them, so their errors do not cancel.  O rounds once more."""
import numpy as np
import torch

from tests.paged_util import U32


def limits(n, rows, causal):
    """Last key that each of the rows sees (-1: padding), for a sequence of n tokens
    whose last `rows` are the rows."""
    pos = torch.arange(rows) + n - rows
    return torch.where(pos < 0, -1, pos if causal else n - 1)


def attention(q, k, v, lim, scale, half_p, extra_k=0.0, fp16_p=False):
    """q [H, m, d], k and v [Hkv, n, d], lim [m].  Returns o [H, m, d], lse [H, m]
    and the bounds of their errors, that of o before its last rounding."""
    H, m, d = q.shape
    Hkv, n, _ = k.shape
    g = H // Hkv
    o = torch.zeros(H, m, d, dtype=torch.float64)
    lse = torch.full((H, m), -np.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(o), torch.zeros(H, m, dtype=torch.float64)
    if n == 0 or m == 0:
        return o, lse, tol, tol_lse
    seen = torch.arange(n) <= lim[:, None]  # [m, n]
    rows = lim >= 0
    for h in range(H):
        kk, vv = k[h // g].double(), v[h // g].double()
        # what no row sees may hold anything
        used = seen.any(0)
        kk, vv = torch.where(used[:, None], kk, 0.0), torch.where(used[:, None], vv, 0.0)
        qq = q[h].double()
        s = (qq @ kk.T * scale).masked_fill(~seen, -np.inf)
        mag = (qq.abs() @ kk.abs().T * scale).masked_fill(~seen, 0.0)
        e = 2 * d * U32 * mag.amax(-1, keepdim=True)
        if extra_k:
            e = e + extra_k * scale * qq.abs().amax(-1, keepdim=True) * kk.abs().sum(-1).amax()
        e = e + mag.amax(-1, keepdim=True) * 4 * U32 + 2.0 ** -20
        l = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(rows, l, 0.0)[:, None]).masked_fill(~seen, 0.0)
        o[h] = p @ vv
        lse[h] = l
        tol[h] = (half_p + 2 * e) * (p @ vv.abs())
        if fp16_p:
            tol[h] += 2.0 ** -25 * (seen.double() @ vv.abs())
        tol_lse[h] = e[:, 0] + torch.where(rows, l, 0.0).abs() * 4 * U32 + 2.0 ** -20
    o[:, ~rows] = 0.0
    return o, lse, tol, tol_lse


def check(o, lse, q, pool_values, lens, news, causal, scale, half_p, extra_k=0.0, fp16_p=False, half_o=None):
    """Holds o [B, H, S, d] and lse [B, H, S] to the bound; pool_values(b, n) gives a
    sequence's keys and values."""
    o, lse, q = o.double().cpu(), lse.double().cpu(), q.cpu()
    S = q.shape[2]
    for b, (n, m) in enumerate(zip(lens, news)):
        k, v = pool_values(b, n)
        lim = limits(n, m, causal)
        ro, rl, to, tl = attention(q[b, :, :m], k, v, lim, scale, half_p, extra_k, fp16_p)
        tol = to + half_o * (ro.abs() + to) + 2.0 ** -25
        assert torch.isfinite(o[b]).all(), f"sequence {b}"
        bad = (o[b, :, :m] - ro).abs() - tol
        assert m == 0 or (bad <= 0).all(), f"sequence {b} ({n} tokens, {m} new): {bad.max():.3e} over the bound"
        real = lim >= 0
        assert ((lse[b, :, :m] - rl).abs() <= tl)[:, real].all(), f"sequence {b}: lse"
        for rows in (torch.arange(m)[~real], torch.arange(m, S)):
            assert (o[b, :, rows] == 0).all() and torch.isneginf(lse[b, :, rows]).all(), f"sequence {b}: padding"
