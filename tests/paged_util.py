"""Plain 64-bit forms of the operators around a paged cache, on the CPU, the
pages that their tests use, and the bounds that the tests hold the kernels to.

u(dtype) = eps / 2 is the largest relative error of one rounding; U32 = 2^-24
that of one fp32 operation.  Every bound below counts roundings:

* a rotated element a c - b s rounds two products and a sum in fp32 and the
  result once: u |y| + 3 U32 (|a c| + |b s|);
* a normed one: the mean of d squares is a chain of 16 fused adds and 4 tree
  steps (20 U32 of the sum, half of it in the root), rsqrt within 2 units,
  three products: below 16 U32 of each operand of the rotation, so with the
  rotation 20 U32 (|a c| + |b s|);
* attention: P is rounded before P V, to one fp16 over a 4-bit cache (u(fp16)),
  to two terms of the cache's type over a 16-bit one (u^2: the second term
  rounds the first's remainder): that times sum p |v|, and, with fp16 terms,
  2^-25 |v| for each term below the smallest normal number, the largest p
  being 1.  O rounds once more: u |o|.  A score is a sum of d exact products,
  each add of the tensor core within 2 U32 of the running magnitude:
  e = 2 d U32 scale sum |q k|, a relative error of p.  exp2, its argument and
  the rescalings: below 2^-20 of p together.
"""
import numpy as np
import torch

U32 = 2.0 ** -24


def u(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def turn(x, table, pos, interleaved, back=False):
    """x [..., S, d] rotated by the rows pos [S] of table (any float type); and
    the magnitude sum |a c| + |b s| behind each element."""
    rot = table.shape[1]
    t = table[pos].to(x.dtype)
    c, s = t[:, :rot // 2], t[:, rot // 2:]
    if back:
        s = -s
    i = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    j = i + (1 if interleaved else rot // 2)
    a, b = x[..., i], x[..., j]
    y, mag = x.clone(), x.abs().clone()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    mag[..., i], mag[..., j] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def norm_rope(x, w, table, pos, eps, interleaved):
    """Forward for x [heads, S, d] in 64 bits: (y, magnitude)."""
    z = x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return (z, z.abs()) if table is None else turn(z, table, pos, interleaved)


def norm_rope_bwd(dy, x, w, table, pos, eps, interleaved):
    """Backward: (dx, dw, magnitude of dx, magnitude of dw)."""
    dz, mag = (dy, dy.abs()) if table is None else turn(dy, table, pos, interleaved, back=True)
    if w is None:
        return dz, None, mag, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    g = dz * w
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    mag_dx = r * (mag * w.abs() + n.abs() * (mag * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (dz * n).sum((0, 1)), mag_dx, (mag * n.abs()).sum((0, 1))


E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def quantise(x, descale):
    """x [..., d] fp32 -> (codes [..., d/2] uint8, factors [..., d/16] E4M3) by
    the header's formula in IEEE fp32; descale [...] broadcasts over the rows."""
    g = x.unflatten(-1, (-1, 16))
    descale = torch.as_tensor(descale, dtype=torch.float32)[..., None]
    f = (g.abs().amax(-1) / (6.0 * descale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    inv = torch.where(f.float() > 0, 1.0 / (f.float() * descale), torch.zeros(()))
    y = g * inv[..., None]
    # nearest of the eight magnitudes, ties to the even code
    m = y.abs().clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    near = (m / step).round() * step
    code = torch.searchsorted(E2M1[:8].contiguous(), near) + 8 * torch.signbit(y)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), f


def dequantise(codes, factors, descale):
    """The fp32 values (code * factor) * descale; exact in 64 bits up to the last product."""
    v = torch.stack([E2M1[(codes & 15).long()], E2M1[(codes >> 4).long()]], -1).flatten(-2)
    v = v.unflatten(-1, (-1, 16)) * factors.float()[..., None]
    return (v * torch.as_tensor(descale, dtype=torch.float32)[..., None, None]).flatten(-2)


def page_table(lens, page, n_pages, width, gen, beyond=-1):
    """Scattered distinct pages for every sequence; entries behind its last page are `beyond`."""
    order = torch.randperm(n_pages, generator=gen).tolist()
    table = torch.full((len(lens), width), beyond, dtype=torch.int32)
    for b, n in enumerate(lens):
        for i in range((n + page - 1) // page):
            table[b, i] = order.pop()
    return table


def sequence(pool, table_row, page, n):
    """Rows 0 .. n-1 of a sequence, [Hkv, n, w], from a pool [n_pages, Hkv, page, w]."""
    pages = table_row[: (n + page - 1) // page].long()
    return pool[pages].transpose(0, 1).flatten(1, 2)[:, :n]


def attention(q, k, v, scale, half_p, extra_k=0.0, fp16_p=False):
    """One sequence's decode in 64 bits.  q [Hq, d], k and v [Hkv, n, d].
    Returns o, lse and the bounds of their errors before o's last rounding,
    where P's rounding is off by half_p at most, relative to p (fp16_p: it has
    fp16's smallest numbers too).  extra_k: error of an element of q relative to
    its row's largest."""
    Hq, d = q.shape
    Hkv, n, _ = k.shape
    if n == 0:
        zero = torch.zeros(Hq, d, dtype=torch.float64)
        return zero, torch.full((Hq,), -np.inf, dtype=torch.float64), zero, torch.zeros(Hq, dtype=torch.float64)
    g = Hq // Hkv
    kk, vv = k.double().repeat_interleave(g, 0), v.double().repeat_interleave(g, 0)
    q = q.double()
    s = torch.einsum("hd,hnd->hn", q, kk) * scale
    e = 2 * d * U32 * scale * torch.einsum("hd,hnd->hn", q.abs(), kk.abs())
    e = e + extra_k * scale * q.abs().amax(-1, keepdim=True) * kk.abs().sum(-1)
    e = e.amax(-1, keepdim=True) + s.abs().amax(-1, keepdim=True) * 4 * U32 + 2.0 ** -20
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    o = torch.einsum("hn,hnd->hd", p, vv)
    a = torch.einsum("hn,hnd->hd", p, vv.abs())
    tol = (half_p + 2 * e) * a
    if fp16_p:
        tol = tol + 2.0 ** -25 * vv.abs().sum(1)
    return o, lse, tol, e[:, 0] + lse.abs() * 4 * U32 + 2.0 ** -20
