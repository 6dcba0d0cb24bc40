"""Attention of a chunk of new tokens over a paged cache, and rotary positions of several axes on the
way into it, in their plain form and as the library runs them.

Three kinds of pass, named by a case's "op":

  rope    norms of queries and keys for each head with a rotation whose pairs follow the positions of
          several axes (time, height, width); with "train" its backward pass too
  append  new keys and values into a paged cache of 16 or 4 bits, keys and queries rotated on the way
          by positions of several axes, which are not the cache's slots; from 4 bits the cached
          sequences are read back, since what is held there counts as the values it stands for
  chunk   the last `new` tokens of every sequence attend to the whole cached sequence and to each
          other (causal, or all to all), over a cache of 16 or 4 bits

`run` computes them with elementary torch operations in 32 bits, or (where `own` is set) with the
calls that a program makes of the library.  `exact` states the definitions once more in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
# The magnitudes that the eight 3-bit E2M1 codes stand for.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One new token for each of 64 sequences of text and images: a serving step, where latency counts.
        dict(name="rope_token", op="rope", train=False, norm=True, B=64, S=1, H=32, Hkv=8, d=128, rot=128,
             sections="16,24,24", cycle=False, interleaved=False, dtype="bf16", far=32768),
        # A training step's forward and backward over images at the 8192-token shape.
        dict(name="rope_train", op="rope", train=True, norm=True, B=4, S=8192, H=16, Hkv=16, d=128, rot=128,
             sections="16,24,24", cycle=False, interleaved=False, dtype="bf16", far=1024),
        # An odd length in half precision, axes taking turns, adjacent pairs of half of each head, no norms.
        dict(name="rope_train_odd", op="rope", train=True, norm=False, B=3, S=1001, H=8, Hkv=2, d=64, rot=32,
             sections="6,5,5", cycle=True, interleaved=True, dtype="fp16", far=0),
        # A serving step's append: one token for each of 64 sequences, queries rotated with them.
        dict(name="append_token", op="append", bits=16, B=64, S=1, H=32, Hkv=8, d=128, rot=128,
             sections="24,20,20", cycle=True, interleaved=False, dtype="bf16", page=64, lo=1, hi=2048, new_lo=1,
             far=32768),
        # Chunks of up to 2048 tokens of four sequences with images, written into a 4-bit cache.
        dict(name="append_fp4_chunk", op="append", bits=4, B=4, S=2048, H=32, Hkv=8, d=128, rot=128,
             sections="16,24,24", cycle=False, interleaved=False, dtype="bf16", page=64, lo=2048, hi=4096,
             new_lo=1500, far=1024),
        # The last 16 tokens of one user's prompt of a thousand: the latency of a short chunk.
        dict(name="chunk_short", op="chunk", bits=16, causal=True, B=1, S=16, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, lo=1000, hi=1000, new_lo=16),
        # Five drafted tokens of each of 64 sequences, 1024 to 32768 tokens long, checked at once.
        dict(name="chunk_verify", op="chunk", bits=16, causal=True, B=64, S=5, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, lo=1024, hi=32768, new_lo=1),
        # Chunks of 2048 tokens of four prompts, behind contexts of up to 16384.
        dict(name="chunk_prompts", op="chunk", bits=16, causal=True, B=4, S=2048, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, lo=4096, hi=16384, new_lo=1500),
        # One long prompt's last 4096 tokens of 32768.
        dict(name="chunk_long", op="chunk", bits=16, causal=True, B=1, S=4096, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, lo=32768, hi=32768, new_lo=4096),
        # A short ragged batch in half precision, three query heads on a KV head, small pages, idle slots, all to all.
        dict(name="chunk_odd", op="chunk", bits=16, causal=False, B=6, S=33, H=6, Hkv=2, d=64, dtype="fp16", page=16,
             lo=0, hi=1500, new_lo=0),
        # The prompts' chunks over a cache held in 4 bits.
        dict(name="chunk_fp4_prompts", op="chunk", bits=4, causal=True, B=4, S=2048, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, lo=4096, hi=16384, new_lo=1500),
        # The drafted tokens over a cache held in 4 bits.
        dict(name="chunk_fp4_verify", op="chunk", bits=4, causal=True, B=64, S=5, H=32, Hkv=8, d=128, dtype="bf16",
             page=64, lo=1024, hi=32768, new_lo=1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    d = rng.choice([64, 128])
    H = Hkv * rng.choice([n for n in (1, 2, 3, 4, 5, 7, 8, 16) if n * Hkv <= 128])
    c = dict(H=H, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "fp16"]))
    kind = rng.choice(["rope", "rope", "append", "append", "chunk", "chunk", "chunk", "chunk"])
    rot = rng.choice([16, d // 2, d, d, d])
    n = rot // 2
    a = rng.randint(1, n - 2)
    b = rng.randint(1, n - 1 - a)
    sections = rng.choice([(n,), (n // 2, n - n // 2), (a, b, n - a - b), (n // 4, n // 8 * 3, n - n // 4 - n // 8 * 3)])
    rope = dict(rot=rot, sections=",".join(map(str, sections)), cycle=rng.random() < 0.4, interleaved=rng.random() < 0.3,
                far=rng.choice([0, 1024, 32768]))
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "rope":
        tokens = _log(rng, 1, min(65536, (1 << 28) // (2 * d * (H + Hkv))))
        B = _log(rng, 1, min(64, tokens))
        return dict(op=kind, train=rng.random() < 0.5, norm=rng.random() < 0.7, B=B, S=max(1, tokens // B), **c, **rope)
    bits = rng.choice([16, 4])
    if kind == "append":
        tokens = _log(rng, 1, 16384)
        B = _log(rng, 1, min(64, tokens))
        S = max(1, tokens // B)
        hi = S + _log(rng, 1, max(1, min(8192, (1 << 27) // (B * Hkv * d))))
        return dict(op=kind, bits=bits, B=B, S=S, page=page, lo=rng.choice([S, hi]), hi=hi,
                    new_lo=rng.choice([S, S // 2, 0]), **c, **rope)
    B = _log(rng, 1, 64)
    S = _log(rng, 1, 4096)
    # A chunk's products and its cache stay below those of the largest listed cases.
    hi = _log(rng, 1, max(1, min(65536, (1 << 30) // (B * Hkv * d), (1 << 39) // (B * H * S * d))))
    S = min(S, hi)
    return dict(op=kind, bits=bits, causal=rng.random() < 0.8, B=B, S=S, page=page,
                lo=rng.choice([0, S, (S + hi + 1) // 2, hi]), hi=hi, new_lo=rng.choice([S, S, S // 2, 0]), **c)


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(lo, hi, n, g):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def _frequencies(rot):
    return 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)


def _table(rows, rot):
    """cos and sin of position * 10000^(-2 i / rot), formed in 64 bits: [rows, rot], cosines first."""
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * _frequencies(rot)
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _sections(c):
    """Pairs of each axis."""
    return [int(n) for n in c["sections"].split(",")]


def _pair_axes(c):
    """The axis that each of the rot / 2 pairs follows: sections one behind another, or axes in turn
    until their shares are used up."""
    if not c["cycle"]:
        return tuple(a for a, n in enumerate(_sections(c)) for _ in range(n))
    left, order = _sections(c), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                order.append(a)
                left[a] -= 1
    return tuple(order)


def _positions(c, g):
    """Positions [axes, B, S] of sequences of images: each image's tokens share a time and lie on a
    grid; whatever the number of axes, they start at a place of the sequence's own."""
    axes, B, S = len(_sections(c)), c["B"], c["S"]
    start = _ints(0, c["far"], B, g).long()[:, None]
    width = 8 + 8 * _ints(0, 3, B, g).long()[:, None]
    s = torch.arange(S, device="cuda")[None, :].expand(B, S)
    grid = [s // (width * width), s // width % width, s % width]
    pick = {1: [s], 2: grid[1:], 3: grid}[axes]
    return torch.stack([start + x for x in pick]).to(torch.int32).contiguous()


def _heads(c, g, dtype):
    """q, k, v as views [B, heads, S, d] of one projection output [B, S, (H + 2 Hkv) d]."""
    B, S, H, Hkv, d = c["B"], c["S"], c["H"], c["Hkv"], c["d"]
    x = _randn((B, S, H + 2 * Hkv, d), dtype, g).transpose(1, 2)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def _pages(c, lens, g):
    """Every sequence's pages, scattered over a pool with room for the longest batch; entries behind a
    sequence's last page are -1."""
    need = (lens.long() + c["page"] - 1) // c["page"]
    width = max(1, (c["hi"] + c["page"] - 1) // c["page"])
    used = torch.arange(width, device="cuda")[None, :] < need[:, None]
    n_pages = c["B"] * width + 3
    order = torch.randperm(n_pages, generator=g, device="cuda")
    slot = (torch.cumsum(used.flatten(), 0) - 1).view(used.shape).clamp(min=0)
    return torch.where(used, order[slot], -1).to(torch.int32).contiguous(), n_pages


def _fp4_pool(c, n_pages, g, spread):
    """A pool of normal values in 4 bits: E2M1 codes (two to a byte, the even element in the low half)
    and one E4M3 scale for each 16 of them."""
    shape = (n_pages, c["Hkv"], c["page"])
    codes = torch.empty(*shape, c["d"] // 2, device="cuda", dtype=torch.uint8)
    scales = torch.empty(*shape, c["d"] // 16, device="cuda", dtype=torch.float8_e4m3fn)
    step = max(1, (1 << 27) // (c["Hkv"] * c["page"] * c["d"]))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        x = torch.randn((n, *shape[1:], c["d"]), generator=g, device="cuda") * spread
        codes[i:i + n], scales[i:i + n] = _quantise(x, torch.ones(1, device="cuda"))
    return codes, scales


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[c["dtype"]]
    s = dict(case=c)
    if c["op"] == "chunk":
        s["q"] = _randn((c["B"], c["H"], c["S"], c["d"]), dtype, g)
    else:
        s["q"], s["k"], s["v"] = _heads(c, g, dtype)
        s["pos"] = _positions(c, g)
        s["axes"] = _pair_axes(c)
        s["rope"] = _table(c["far"] + c["S"] + 32, c["rot"])
    if c["op"] == "rope":
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"] = 1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")
            s["kw"] = 1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")
        if c["train"]:
            s["dqo"] = _randn((c["B"], c["H"], c["S"], c["d"]), dtype, g)
            s["dko"] = _randn((c["B"], c["Hkv"], c["S"], c["d"]), dtype, g)
        return s
    s["lens"] = lens = _ints(c["lo"], c["hi"], c["B"], g)
    s["new"] = torch.minimum(_ints(min(c["new_lo"], c["S"]), c["S"], c["B"], g), lens)
    s["table"], n_pages = _pages(c, lens, g)
    pool = (n_pages, c["Hkv"], c["page"], c["d"])
    if c["bits"] == 16:
        s["kc"], s["vc"] = _randn(pool, dtype, g), _randn(pool, dtype, g)
    else:
        s["kc"], s["ks"] = _fp4_pool(c, n_pages, g, 4.0)
        s["vc"], s["vs"] = _fp4_pool(c, n_pages, g, 2.0)
        s["kd"] = 0.2 + 0.1 * torch.rand(c["Hkv"], generator=g, device="cuda")
        s["vd"] = 0.4 + 0.2 * torch.rand(c["Hkv"], generator=g, device="cuda")
    return s


def work(case):
    """Bytes and operations of one pass: every input read once, every output written once."""
    c = case
    H, Hkv, d, B, S = c["H"], c["Hkv"], c["d"], c["B"], c["S"]
    if c["op"] == "rope":
        n = B * S * (H + Hkv) * d
        # the table's rows are shared by tokens at one place; what has to come is the positions
        side = 4 * len(_sections(c)) * B * S + 4 * c["rot"] * min(B * S, c["far"] + S)
        if not c["train"]:
            return {"bytes": 4 * n + side, "flops": (6 if c["norm"] else 3) * n}
        # x and dy read (x twice only by a program that runs the two calls apart), y and dx written
        return {"bytes": 8 * n + side, "flops": (20 if c["norm"] else 6) * n}
    held = 2 * Hkv * (2 * d if c["bits"] == 16 else d / 2 + d / 16)  # bytes of one cached token
    mean = (c["lo"] + c["hi"]) / 2
    new = min((min(c["new_lo"], S) + S) / 2, mean)
    if c["op"] == "append":
        token = 4 * Hkv * d + held + 4 * len(_sections(c)) + 4 * c["rot"]
        back = (mean - new) * held + c["hi"] * 4 * Hkv * d if c["bits"] == 4 else 0
        return {"bytes": B * (H * d * 2 * (new + S) + new * token + back), "flops": 3 * B * new * (H + Hkv) * d}
    keys = mean - (new - 1) / 2 if c["causal"] else mean
    return {"bytes": B * (mean * held + H * d * 2 * (new + S) + 4 * H * S), "flops": 4 * B * H * new * max(keys, 0) * d}


def run(s):
    c = s["case"]
    return {"rope": _rope, "append": _append, "chunk": _chunk}[c["op"]](s, c)


# ---------------------------------------------------------------- the plain forms, and the library's calls


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _joined(a, b, x, rot, interleaved):
    y = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _rotate(x, cos, sin, rot, interleaved, back=False):
    """x [B, heads, S, d] rotated by cos, sin [B, 1, S, rot / 2]; `back` by the negative angles."""
    a, b = _pairs(x, rot, interleaved)
    if back:
        return _joined(a * cos + b * sin, b * cos - a * sin, x, rot, interleaved)
    return _joined(a * cos - b * sin, b * cos + a * sin, x, rot, interleaved)


def _angles(s, c):
    """Cosines and sines [B, 1, S, rot / 2]: each pair's from its own axis's position."""
    half = c["rot"] // 2
    rows = torch.stack([s["pos"][a] for a in s["axes"]], dim=-1).long()  # [B, S, rot / 2]
    i = torch.arange(half, device="cuda")
    return s["rope"][rows, i][:, None], s["rope"][rows, half + i][:, None]


def _rope(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_qk_norm_rope, attn_qk_norm_rope_bwd

        out = attn_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], rope=s["rope"], positions=s["pos"], eps=EPS,
                                interleaved=c["interleaved"], axes=s["axes"])
        if c["train"]:
            grads = attn_qk_norm_rope_bwd(s["dqo"], s["dko"], s["q"], s["k"], s["qw"], s["kw"], rope=s["rope"],
                                          positions=s["pos"], eps=EPS, interleaved=c["interleaved"], axes=s["axes"])
            out += grads if c["norm"] else grads[:2]
        return out
    cos, sin = _angles(s, c)
    outs, grads, wgrads = [], [], []
    for x16, w, dy in ((s["q"], s["qw"], s.get("dqo")), (s["k"], s["kw"], s.get("dko"))):
        x = x16.float()
        if c["norm"]:
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            x = x * r
        outs.append(_rotate(x * w if c["norm"] else x, cos, sin, c["rot"], c["interleaved"]).to(x16.dtype))
        if c["train"]:
            dz = _rotate(dy.float(), cos, sin, c["rot"], c["interleaved"], back=True)
            if c["norm"]:
                wgrads.append((dz * x).sum((0, 1, 2)))
                dn = dz * w
                dz = r * (dn - x * (dn * x).mean(-1, keepdim=True))
            grads.append(dz.to(x16.dtype))
    return tuple(outs + grads + wgrads)


def _places(s, c):
    """Positions [B, S] of the new tokens (the last `new` of each sequence) and which of them exist."""
    i = torch.arange(c["S"], device="cuda")[None, :]
    pos = (s["lens"] - s["new"]).long()[:, None] + i
    return pos, (i < s["new"][:, None]) & (pos >= 0)


def _append(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_cache_append, attn_cache_append_fp4, attn_cache_gather_fp4

        same = dict(new_lens=s["new"], rope=s["rope"], interleaved=c["interleaved"], q=s["q"], positions=s["pos"],
                    axes=s["axes"])
        if c["bits"] == 16:
            q = attn_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], **same)
            return q, s["kc"], s["vc"]
        q = attn_cache_append_fp4(s["k"], s["v"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                  k_descale=s["kd"], v_descale=s["vd"], **same)
        return (q,) + attn_cache_gather_fp4(s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"], c["hi"],
                                            k_descale=s["kd"], v_descale=s["vd"], dtype=s["q"].dtype)
    pos, real = _places(s, c)
    cos, sin = _angles(s, c)
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"])
    q = torch.where(real[:, None, :, None], q, 0.0).to(s["q"].dtype)
    k = _rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"])
    b, i = real.nonzero(as_tuple=True)
    p = pos[b, i]
    page, row = s["table"][b, p // c["page"]].long(), p % c["page"]
    if c["bits"] == 16:
        s["kc"][page, :, row] = k.to(s["kc"].dtype)[b, :, i]
        s["vc"][page, :, row] = s["v"][b, :, i]
        return q, s["kc"], s["vc"]
    out = [q]
    for x, codes, scales, descale in ((k, s["kc"], s["ks"], s["kd"]), (s["v"].float(), s["vc"], s["vs"], s["vd"])):
        new_codes, new_scales = _quantise(x[b, :, i], descale[:, None])
        codes[page, :, row] = new_codes
        scales.view(torch.uint8)[page, :, row] = new_scales.view(torch.uint8)
    for x in "kv":
        v = _cached(s, c, x, slice(None), slice(None))[:, :, :c["hi"]]
        present = torch.arange(c["hi"], device="cuda") < s["lens"][:, None]
        out.append(torch.where(present[:, None, :, None], v, 0.0).to(q.dtype))
    return tuple(out)


def _quantise(x, descale):
    """[..., d] in 32 bits -> codes [..., d / 2], scales [..., d / 16]: each group of 16 gets the E4M3
    scale nearest to its largest magnitude / 6, each element the E2M1 code nearest to its value over
    scale * descale, ties to the even code.  descale broadcasts over [..., d / 16]."""
    g = x.unflatten(-1, (-1, 16))
    scale = (g.abs().amax(-1) / (6.0 * descale)).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = scale.float()
    y = g * torch.where(f > 0, 1.0 / (f * descale), 0.0)[..., None]
    m = y.abs()
    code = (m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
    code = (code + 8 * torch.signbit(y)).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scales, descale, dtype=torch.float32):
    """Codes and scales -> the values they stand for, [..., d]; descale broadcasts over [..., d / 16, 16]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda", dtype=dtype)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], dim=-1).flatten(-2)
    return ((v.unflatten(-1, (-1, 16)) * scales.to(dtype)[..., None]) * descale).flatten(-2)


def _cached(s, c, x, b, h):
    """Keys ("k") or values ("v") of sequences b and KV heads h (slices) in 32 bits: [., ., width * page, d]."""
    def rows(pool):
        return pool[:, h][s["table"][b].long().clamp(min=0)].transpose(1, 2).flatten(2, 3)

    if c["bits"] == 16:
        return rows(s[x + "c"]).float()
    scales = rows(s[x + "s"].view(torch.uint8)).view(torch.float8_e4m3fn)
    return _values(rows(s[x + "c"]), scales, s[x + "d"][h][:, None, None, None])


def _chunk(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_fwd_paged, attn_fwd_paged_fp4

        if c["bits"] == 16:
            return attn_fwd_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], new_lens=s["new"],
                                  causal=c["causal"])
        return attn_fwd_paged_fp4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                  new_lens=s["new"], k_descale=s["kd"], v_descale=s["vd"], causal=c["causal"])
    B, H, Hkv, S, d = c["B"], c["H"], c["Hkv"], c["S"], c["d"]
    g = H // Hkv
    pos, real = _places(s, c)
    limit = torch.where(real, pos if c["causal"] else s["lens"].long()[:, None] - 1, -1)  # last key of each token
    o = torch.empty_like(s["q"])
    lse = torch.empty(B, H, S, device="cuda")
    width = s["table"].shape[1] * c["page"]
    # Scores of at most 2^29 elements at a time: all sequences and heads, or one sequence's, or one KV head's.
    whole = B * H * S * width <= 1 << 29
    heads = Hkv if H * S * width <= 1 << 29 else 1
    for b in [slice(0, B)] if whole else [slice(i, i + 1) for i in range(B)]:
        for h0 in range(0, Hkv, heads):
            h, hq = slice(h0, h0 + heads), slice(h0 * g, (h0 + heads) * g)
            k, v = _cached(s, c, "k", b, h), _cached(s, c, "v", b, h)
            q = s["q"][b, hq].float().unflatten(1, (heads, g)).flatten(2, 3)  # [., heads, g S, d]
            score = (q @ k.transpose(-1, -2) / math.sqrt(d)).unflatten(2, (g, S))
            key = torch.arange(width, device="cuda")
            score = torch.where(key <= limit[b][:, None, None, :, None], score, -math.inf)
            top = score.amax(-1, keepdim=True).clamp(min=-1e30)
            p = torch.exp(score - top)
            total = p.sum(-1, keepdim=True)
            v = torch.where((key < s["lens"][b][:, None])[:, None, :, None], v, 0.0)
            y = (p.flatten(2, 3) @ v).unflatten(2, (g, S))
            o[b, hq] = torch.where(total > 0, y / total, 0.0).flatten(1, 2).to(o.dtype)
            lse[b, hq] = (top + total.log())[..., 0].flatten(1, 2)
    return o, lse


# ---------------------------------------------------------------- the definitions in 64 bits


def _turned(x, c, pos, axes):
    """x [heads, n, d] in 64 bits, its pairs as complex numbers times exp(i * angle); pos [axes, n]."""
    rot = c["rot"]
    angle = torch.stack([pos[a].double() * f for a, f in zip(axes, _frequencies(rot).tolist())], dim=-1)
    w = torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    if c["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * w
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * w
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    return {"rope": _rope_64, "append": _append_64, "chunk": _chunk_64}[c["op"]](c, s)


def _rope_64(c, s):
    outs, grads, wgrads = [], [], []
    for x16, w, dy in ((s["q"], s["qw"], s.get("dqo")), (s["k"], s["kw"], s.get("dko"))):
        y = torch.empty(x16.shape, device="cuda", dtype=torch.float64)
        dx, dw = torch.empty_like(y), torch.zeros(c["d"], device="cuda", dtype=torch.float64)
        for b in range(c["B"]):
            pos, x = s["pos"][:, b], x16[b].double()
            if c["norm"]:
                size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
                r = 1.0 / torch.sqrt(size * size / c["d"] + EPS)
                y[b] = _turned(x * r * w.double(), c, pos, s["axes"])
            else:
                y[b] = _turned(x, c, pos, s["axes"])
            if c["train"]:
                dz = _turned(dy[b].double(), c, -pos, s["axes"])
                if c["norm"]:
                    dw += torch.einsum("hsd,hsd->d", dz, x * r)
                    g = dz * w.double()
                    dz = r * g - x * r ** 3 * torch.einsum("hsd,hsd->hs", g, x)[..., None] / c["d"]
                dx[b] = dz
        outs.append(y)
        grads.append(dx)
        wgrads.append(dw)
    return tuple(outs + (grads if c["train"] else []) + (wgrads if c["train"] and c["norm"] else []))


def _append_64(c, s):
    q = torch.zeros(c["B"], c["H"], c["S"], c["d"], device="cuda", dtype=torch.float64)
    if c["bits"] == 16:
        kv = [s["kc"].double(), s["vc"].double()]
    else:
        kv = [torch.zeros(c["B"], c["Hkv"], c["hi"], c["d"], device="cuda", dtype=torch.float64) for _ in "kv"]
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        pos, pages = s["pos"][:, b, :m], s["table"][b].long()
        q[b, :, :m] = _turned(s["q"][b, :, :m].double(), c, pos, s["axes"])
        fresh = _turned(s["k"][b, :, :m].double(), c, pos, s["axes"]), s["v"][b, :, :m].double()
        at = torch.arange(n - m, n, device="cuda")
        for j in range(2):
            if c["bits"] == 16:
                kv[j][pages[at // c["page"]], :, at % c["page"]] = fresh[j].transpose(0, 1)
            elif n:
                used = pages[:(n + c["page"] - 1) // c["page"]]
                kv[j][b, :, :n] = _sequence(s, c, used, n, "kv"[j])
                kv[j][b, :, n - m:n] = _nearest(fresh[j], (s["kd"], s["vd"])[j].double())
    return (q, *kv)


def _nearest(x, descale):
    """x [Hkv, n, d] in 64 bits -> the values that its 4-bit form stands for."""
    g = x.unflatten(-1, (-1, 16))
    descale = descale[:, None, None, None]
    scale = (g.abs().amax(-1, keepdim=True) / descale / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).double()
    y = torch.where(scale > 0, g / (scale * descale), 0.0)
    m = y.abs().clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))  # spacing of E2M1 around m
    near = (m / step).round() * step  # ties go to the even multiple, which is the even code
    return (torch.sign(y) * near * scale * descale).flatten(-2)


def _sequence(s, c, pages, n, x):
    """A sequence's first n cached keys ("k") or values ("v"), [Hkv, n, d] in 64 bits."""
    def rows(pool):
        return pool[pages].transpose(0, 1).flatten(1, 2)[:, :n]

    if c["bits"] == 16:
        return rows(s[x + "c"]).double()
    scales = rows(s[x + "s"].view(torch.uint8)).view(torch.float8_e4m3fn)
    return _values(rows(s[x + "c"]), scales, s[x + "d"].double()[:, None, None, None], torch.float64)


def _chunk_64(c, s):
    if work(c)["flops"] > 4e12:  # the 64-bit products would take too long
        return None
    o = torch.zeros(c["B"], c["H"], c["S"], c["d"], device="cuda", dtype=torch.float64)
    lse = torch.full((c["B"], c["H"], c["S"]), -math.inf, device="cuda", dtype=torch.float64)
    g = c["H"] // c["Hkv"]
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        if m == 0:
            continue
        pages = s["table"][b, :(n + c["page"] - 1) // c["page"]].long()
        k, v = (_sequence(s, c, pages, n, x) for x in "kv")
        hidden = torch.ones(m, n, device="cuda", dtype=torch.bool).triu(n - m + 1) if c["causal"] else None
        for h in range(c["H"]):
            score = s["q"][b, h, :m].double() @ k[h // g].T / math.sqrt(c["d"])
            if c["causal"]:
                score.masked_fill_(hidden, -math.inf)
            lse[b, h, :m] = torch.logsumexp(score, -1)
            o[b, h, :m] = torch.softmax(score, -1) @ v[h // g]
    return o, lse
