"""The operators around a paged key/value cache, in their plain form and as the library runs them.

Four kinds of pass, named by a case's "op":

  norm_rope   norms of queries and keys for each head with the position rotation; with "train" its
              backward pass too
  append      new keys and values into a paged 16-bit cache, rotated on the way, with the queries
  context     new keys and values into a paged 4-bit cache, and the whole cached context read back
              as 16-bit keys and values (what a chunk of a prompt attends to)
  decode      one query per sequence over a paged cache held in 16 bits or in 4

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
        # One new token for each of 64 sequences in flight: a serving step, where latency counts.
        dict(name="norm_rope_token", op="norm_rope", train=False, B=64, S=1, H=32, Hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16", far=32768),
        # Two prompts of 4096 tokens, read from the fused projection's output.
        dict(name="norm_rope_prompt", op="norm_rope", train=False, B=2, S=4096, H=32, Hkv=8, d=128, rot=128,
             interleaved=False, dtype="bf16", far=0),
        # A training step's forward and backward at the 8192-token shape.
        dict(name="norm_rope_train", op="norm_rope", train=True, B=4, S=8192, H=16, Hkv=16, d=128, rot=128,
             interleaved=False, dtype="bf16", far=0),
        # An odd length in half precision, adjacent pairs rotated in half of each head.
        dict(name="norm_rope_train_odd", op="norm_rope", train=True, B=3, S=1001, H=8, Hkv=2, d=64, rot=32,
             interleaved=True, dtype="fp16", far=0),
        # A serving step's append: one token for each of 64 sequences, queries rotated with them.
        dict(name="append_token", op="append", B=64, S=1, H=32, Hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", page=64, lo=1, hi=2048, new_lo=1),
        # Eight prompts of different lengths, padded to 4096, written at once.
        dict(name="append_prompts", op="append", B=8, S=4096, H=32, Hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", page=64, lo=4096, hi=8192, new_lo=1),
        # A chunk of 2048 tokens behind contexts of up to 16384, held in 4 bits and read back for the prefill.
        dict(name="context_fp4_chunk", op="context", B=4, S=2048, H=32, Hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", page=64, lo=4096, hi=16384, new_lo=1500),
        # A short ragged batch in half precision with small pages.
        dict(name="context_fp4_small", op="context", B=3, S=33, H=8, Hkv=2, d=64, rot=32, interleaved=True,
             dtype="fp16", page=16, lo=33, hi=700, new_lo=0),
        # One sequence of a thousand tokens: the latency of a single user's token.
        dict(name="decode_one", op="decode", bits=16, B=1, H=32, Hkv=8, d=128, dtype="bf16", page=64, lo=1000,
             hi=1000),
        # 64 sequences of 1024 to 32768 tokens, the batch of the decode benchmark.
        dict(name="decode_batch", op="decode", bits=16, B=64, H=32, Hkv=8, d=128, dtype="bf16", page=64, lo=1024,
             hi=32768),
        # The same batch over a cache held in 4 bits.
        dict(name="decode_fp4_batch", op="decode", bits=4, B=64, H=32, Hkv=8, d=128, dtype="bf16", page=64, lo=1024,
             hi=32768),
        # Sixteen query heads on one KV head, small pages, idle slots among the sequences.
        dict(name="decode_fp4_small", op="decode", bits=4, B=6, H=16, Hkv=1, d=64, dtype="fp16", page=16, lo=0,
             hi=1500),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 16])
    d = rng.choice([64, 128])
    H = Hkv * rng.choice([n for n in (1, 2, 3, 4, 5, 7, 8, 16) if n * Hkv <= 128])
    c = dict(H=H, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "fp16"]))
    kind = rng.choice(["norm_rope", "norm_rope", "append", "context", "decode", "decode", "decode"])
    rope = dict(rot=rng.choice([0, 16, d // 2, d, d, d]), interleaved=rng.random() < 0.3)
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "norm_rope":
        tokens = _log(rng, 1, min(65536, (1 << 28) // (2 * d * (H + Hkv))))
        B = _log(rng, 1, min(64, tokens))
        return dict(op=kind, train=rng.random() < 0.5, B=B, S=max(1, tokens // B), far=rng.choice([0, 0, 32768]),
                    **c, **rope)
    if kind == "decode":
        bits = rng.choice([16, 4])
        B = _log(rng, 1, 96)
        hi = _log(rng, 1, min(65536, (1 << 30) // (B * Hkv * d)))
        return dict(op=kind, bits=bits, B=B, page=page, lo=rng.choice([0, (hi + 1) // 2, hi]), hi=hi, **c)
    tokens = _log(rng, 1, 16384)
    B = _log(rng, 1, min(64, tokens))
    S = max(1, tokens // B)
    hi = S + _log(rng, 1, max(1, min(8192, (1 << 27) // (B * Hkv * d))))
    return dict(op=kind, B=B, S=S, page=page, lo=rng.choice([S, hi]), hi=hi, new_lo=rng.choice([S, S // 2, 0]),
                **c, **rope)


def _randn(shape, dtype, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _ints(lo, hi, n, g):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def _table(rows, rot):
    """cos and sin of position * 10000^(-2 i / rot), formed in 64 bits: [rows, rot], cosines first."""
    if rot == 0:
        return None
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _heads(c, g, dtype, S):
    """q, k, v as views [B, heads, S, d] of one projection output [B, S, (H + 2 Hkv) d]."""
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
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
    if c["op"] == "norm_rope":
        s["q"], s["k"], _ = _heads(c, g, dtype, c["S"])
        s["qw"] = 1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")
        s["kw"] = 1 + 0.1 * torch.randn(c["d"], generator=g, device="cuda")
        s["pos"] = None
        rows = c["S"]
        if c["far"]:
            rows = c["far"] + c["S"]
            start = _ints(0, c["far"], c["B"], g)
            s["pos"] = start[:, None] + torch.arange(c["S"], device="cuda", dtype=torch.int32)
        s["rope"] = _table(rows, c["rot"])
        if c["train"]:
            s["dqo"] = _randn((c["B"], c["H"], c["S"], c["d"]), dtype, g)
            s["dko"] = _randn((c["B"], c["Hkv"], c["S"], c["d"]), dtype, g)
        return s
    s["lens"] = lens = _ints(c["lo"], c["hi"], c["B"], g)
    s["table"], n_pages = _pages(c, lens, g)
    pool = (n_pages, c["Hkv"], c["page"], c["d"])
    if c["op"] == "decode":
        s["q"] = _randn((c["B"], c["H"], 1, c["d"]), dtype, g)
    else:
        s["q"], s["k"], s["v"] = _heads(c, g, dtype, c["S"])
        s["new"] = torch.minimum(_ints(min(c["new_lo"], c["S"]), c["S"], c["B"], g), lens)
        s["rope"] = _table(c["hi"] + 1, c["rot"])
    if c["op"] == "append" or (c["op"] == "decode" and c["bits"] == 16):
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
    H, Hkv, d, B = c["H"], c["Hkv"], c["d"], c["B"]
    if c["op"] == "norm_rope":
        row = B * c["S"]
        table = (row if c["far"] else c["S"]) * c["rot"] * 4
        n = row * (H + Hkv) * d
        if c["train"]:  # x and dy read; y and dx written
            return {"bytes": 2 * n * 4 + table, "flops": 20 * n}
        return {"bytes": 2 * n * 2 + table, "flops": 6 * n}
    mean = (c["lo"] + c["hi"]) / 2
    if c["op"] == "decode":
        row = {16: 2 * d, 4: d / 2 + d / 16}[c["bits"]]
        return {"bytes": B * (2 * mean * Hkv * row + 4 * H * d), "flops": 4 * B * H * mean * d}
    new = (min(c["new_lo"], c["S"]) + c["S"]) / 2
    bytes_q = B * H * d * 2 * (new + c["S"])
    if c["op"] == "append":  # tokens read and written in 16 bits, the table's rows
        return {"bytes": bytes_q + B * new * (8 * Hkv * d + 4 * c["rot"]), "flops": 3 * B * new * (H + Hkv) * d}
    held = 2 * Hkv * (d / 2 + d / 16)
    return {"bytes": bytes_q + B * (new * (4 * Hkv * d + held + 4 * c["rot"]) + (mean - new) * held
                                    + c["hi"] * 4 * Hkv * d), "flops": 4 * B * mean * Hkv * d}


def run(s):
    c = s["case"]
    return {"norm_rope": _norm_rope, "append": _append, "context": _context, "decode": _decode}[c["op"]](s, c)


# ---------------------------------------------------------------- the plain forms, and the library's calls


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _joined(a, b, x, rot, interleaved):
    y = torch.stack([a, b], dim=-1).flatten(-2) if interleaved else torch.cat([a, b], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _rotate(x, cos, sin, rot, interleaved, back=False):
    """x [B, heads, S, d] rotated by cos, sin [B or 1, 1, S, rot / 2]; `back` by the negative angles."""
    if rot == 0:
        return x
    a, b = _pairs(x, rot, interleaved)
    if back:
        return _joined(a * cos + b * sin, b * cos - a * sin, x, rot, interleaved)
    return _joined(a * cos - b * sin, b * cos + a * sin, x, rot, interleaved)


def _angles(rope, pos, S, rot):
    if rot == 0:
        return None, None
    t = rope[:S][None, None] if pos is None else rope[pos.long()][:, None]
    return t[..., :rot // 2], t[..., rot // 2:]


def _norm_rope(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_qk_norm_rope, attn_qk_norm_rope_bwd

        out = attn_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], rope=s["rope"], positions=s["pos"], eps=EPS,
                                interleaved=c["interleaved"])
        if c["train"]:
            out += attn_qk_norm_rope_bwd(s["dqo"], s["dko"], s["q"], s["k"], s["qw"], s["kw"], rope=s["rope"],
                                         positions=s["pos"], eps=EPS, interleaved=c["interleaved"])
        return out
    cos, sin = _angles(s["rope"], s["pos"], c["S"], c["rot"])
    outs, grads, wgrads = [], [], []
    for x16, w, dy in ((s["q"], s["qw"], s.get("dqo")), (s["k"], s["kw"], s.get("dko"))):
        x = x16.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        outs.append(_rotate(x * r * w, cos, sin, c["rot"], c["interleaved"]).to(x16.dtype))
        if c["train"]:
            dz = _rotate(dy.float(), cos, sin, c["rot"], c["interleaved"], back=True)
            n = x * r
            wgrads.append((dz * n).sum((0, 1, 2)))
            dn = dz * w
            grads.append((r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x16.dtype))
    return tuple(outs + grads + wgrads)


def _places(s, c):
    """Positions [B, S] of the new tokens (the last `new` of each sequence) and which of them exist."""
    i = torch.arange(c["S"], device="cuda")[None, :]
    pos = (s["lens"] - s["new"]).long()[:, None] + i
    return pos, (i < s["new"][:, None]) & (pos >= 0)


def _rotated(s, c, pos, real):
    """Queries (0 where a token is padding) and keys after the rotation, in 32 bits."""
    cos, sin = _angles(s["rope"], pos.clamp(0, c["hi"]), c["S"], c["rot"])
    q = _rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"])
    return torch.where(real[:, None, :, None], q, 0.0), _rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"])


def _slots(s, c, pos, real):
    b, i = real.nonzero(as_tuple=True)
    p = pos[b, i]
    return b, i, s["table"][b, p // c["page"]].long(), p % c["page"]


def _append(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_cache_append

        q = attn_cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["lens"], new_lens=s["new"],
                              rope=s["rope"], interleaved=c["interleaved"], q=s["q"])
        return q, s["kc"], s["vc"]
    pos, real = _places(s, c)
    q, k = _rotated(s, c, pos, real)
    b, i, page, row = _slots(s, c, pos, real)
    s["kc"][page, :, row] = k.to(s["kc"].dtype)[b, :, i]
    s["vc"][page, :, row] = s["v"][b, :, i]
    return q.to(s["q"].dtype), s["kc"], s["vc"]


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


def _gathered(pool, s, c):
    """Pages [n_pages, Hkv, page, w] in the order of the sequences: [B, Hkv, width * page, w]."""
    return pool[s["table"].long().clamp(min=0)].transpose(1, 2).flatten(2, 3)


def _present(s, n):
    return torch.arange(n, device="cuda")[None, :] < s["lens"][:, None]


def _context(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_cache_append_fp4, attn_cache_gather_fp4

        q = attn_cache_append_fp4(s["k"], s["v"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                  new_lens=s["new"], k_descale=s["kd"], v_descale=s["vd"], rope=s["rope"],
                                  interleaved=c["interleaved"], q=s["q"])
        return (q,) + attn_cache_gather_fp4(s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"], c["hi"],
                                            k_descale=s["kd"], v_descale=s["vd"], dtype=s["q"].dtype)
    pos, real = _places(s, c)
    q, k = _rotated(s, c, pos, real)
    b, i, page, row = _slots(s, c, pos, real)
    out = [q.to(s["q"].dtype)]
    for x, codes, scales, descale in ((k, s["kc"], s["ks"], s["kd"]), (s["v"].float(), s["vc"], s["vs"], s["vd"])):
        new_codes, new_scales = _quantise(x[b, :, i], descale[:, None])
        codes[page, :, row] = new_codes
        scales.view(torch.uint8)[page, :, row] = new_scales.view(torch.uint8)
        seq_codes = _gathered(codes, s, c)[:, :, :c["hi"]]
        seq_scales = _gathered(scales.view(torch.uint8), s, c)[:, :, :c["hi"]].view(torch.float8_e4m3fn)
        v = _values(seq_codes, seq_scales, descale[:, None, None, None])
        out.append(torch.where(_present(s, c["hi"])[:, None, :, None], v, 0.0).to(s["q"].dtype))
    return tuple(out)


def _decode(s, c):
    if own:
        from exact_tiled_attention_gb300 import attn_decode_paged, attn_decode_paged_fp4

        if c["bits"] == 16:
            return attn_decode_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"])
        return attn_decode_paged_fp4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"],
                                     k_descale=s["kd"], v_descale=s["vd"])
    if c["bits"] == 16:
        k, v = _gathered(s["kc"], s, c).float(), _gathered(s["vc"], s, c).float()
    else:
        k = _values(_gathered(s["kc"], s, c), _gathered(s["ks"].view(torch.uint8), s, c).view(torch.float8_e4m3fn),
                    s["kd"][:, None, None, None])
        v = _values(_gathered(s["vc"], s, c), _gathered(s["vs"].view(torch.uint8), s, c).view(torch.float8_e4m3fn),
                    s["vd"][:, None, None, None])
    real = _present(s, k.shape[2])[:, None, None, :]
    q = s["q"].float().view(c["B"], c["Hkv"], c["H"] // c["Hkv"], c["d"])
    score = torch.where(real, q @ k.transpose(-1, -2) / math.sqrt(c["d"]), -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(real.transpose(-1, -2), v, 0.0)
    o = torch.where(total > 0, (p @ v) / total, 0.0)
    return o.to(s["q"].dtype).view(s["q"].shape), (top + total.log()).view(c["B"], c["H"])


# ---------------------------------------------------------------- the definitions in 64 bits


def _turned(x, c, pos):
    """x [..., n, d] in 64 bits at positions pos [n], as complex numbers times exp(i * angle)."""
    rot = c["rot"]
    if rot == 0:
        return x.clone()
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    w = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), pos.double()[:, None] * inv)
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
    if c["op"] == "norm_rope":
        outs, grads, wgrads = [], [], []
        for x16, w, dy in ((s["q"], s["qw"], s.get("dqo")), (s["k"], s["kw"], s.get("dko"))):
            y = torch.empty(x16.shape, device="cuda", dtype=torch.float64)
            dx, dw = torch.empty_like(y), torch.zeros(c["d"], device="cuda", dtype=torch.float64)
            for b in range(c["B"]):
                pos = torch.arange(c["S"], device="cuda") if s["pos"] is None else s["pos"][b]
                x = x16[b].double()
                size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
                r = 1.0 / torch.sqrt(size * size / c["d"] + EPS)
                y[b] = _turned(x * r * w.double(), c, pos)
                if c["train"]:
                    dz = _turned(dy[b].double(), c, -pos)
                    dw += torch.einsum("hsd,hsd->d", dz, x * r)
                    g = dz * w.double()
                    dx[b] = r * g - x * r ** 3 * torch.einsum("hsd,hsd->hs", g, x)[..., None] / c["d"]
            outs.append(y)
            grads.append(dx)
            wgrads.append(dw)
        return tuple(outs + grads + wgrads) if c["train"] else tuple(outs)
    lens = s["lens"].tolist()
    if c["op"] == "decode":
        o = torch.zeros(c["B"], c["H"], 1, c["d"], device="cuda", dtype=torch.float64)
        lse = torch.full((c["B"], c["H"]), -math.inf, device="cuda", dtype=torch.float64)
        for b, n in enumerate(lens):
            if n == 0:
                continue
            pages = s["table"][b, :(n + c["page"] - 1) // c["page"]].long()
            k, v = (_sequence(s, c, pages, n, x) for x in "kv")
            q = s["q"][b, :, 0].double().view(c["Hkv"], -1, c["d"])
            score = torch.bmm(q, k.transpose(1, 2)) / math.sqrt(c["d"])
            lse[b] = torch.logsumexp(score, -1).flatten()
            o[b, :, 0] = torch.bmm(torch.softmax(score, -1), v).view(c["H"], c["d"])
        return o, lse
    new = s["new"].tolist()
    q = torch.zeros(c["B"], c["H"], c["S"], c["d"], device="cuda", dtype=torch.float64)
    pools = [s["kc"].double(), s["vc"].double()] if c["op"] == "append" else []
    whole = [torch.zeros(c["B"], c["Hkv"], c["hi"], c["d"], device="cuda", dtype=torch.float64) for _ in "kv"]
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n - m, n, device="cuda")
        q[b, :, :m] = _turned(s["q"][b, :, :m].double(), c, pos)
        fresh = _turned(s["k"][b, :, :m].double(), c, pos), s["v"][b, :, :m].double()
        pages = s["table"][b].long()
        for j in range(2):
            if c["op"] == "append":
                pools[j][pages[pos // c["page"]], :, pos % c["page"]] = fresh[j].transpose(0, 1)
            elif n:
                used = pages[:(n + c["page"] - 1) // c["page"]]
                whole[j][b, :, :n] = _sequence(s, c, used, n, "kv"[j])
                whole[j][b, :, n - m:n] = _nearest(fresh[j], (s["kd"], s["vd"])[j].double())
    return (q, *pools) if c["op"] == "append" else (q, *whole)


def _sequence(s, c, pages, n, x):
    """A sequence's first n cached keys ("k") or values ("v"), [Hkv, n, d] in 64 bits."""
    def rows(pool):
        return pool[pages].transpose(0, 1).flatten(1, 2)[:, :n]

    if x + "s" not in s:
        return rows(s[x + "c"]).double()
    scales = rows(s[x + "s"].view(torch.uint8)).view(torch.float8_e4m3fn)
    return _values(rows(s[x + "c"]), scales, s[x + "d"].double()[:, None, None, None], torch.float64)


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
