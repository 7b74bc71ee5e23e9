"""Measured cases of the paged key/value cache operators: head norms with position rotation,
appending to the cache, reading it back densely, and attention of one new token over it.

`run` computes each operator either in plain torch operations (``own = False``) or through the
package's entry points (``own = True``), from the same state.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
# E2M1: magnitudes by code, sign in bit 3.
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------------------ cases --

def _case(op, name=None, **kw):
    c = {"op": op}
    if name:
        c["name"] = name
    c.update(kw)
    return c


def listed():
    return [
        # The queries and keys of one step of a small running batch: latency is all of it.
        _case("norm_rope", "norm_rope_step", layout="packed", B=1, N=8, Hq=32, Hkv=8, D=128, rot=128,
              interleaved=False, norm=True, dtype="bf16"),
        # The long video sequence the benchmark runs attention on, with adjacent-pair rotation.
        _case("norm_rope", "norm_rope_video", layout="HND", B=1, N=32768, Hq=24, Hkv=24, D=128, rot=128,
              interleaved=True, norm=True, dtype="bf16"),
        # A packed prompt of odd length, grouped heads, half of the channels rotated, no norm.
        _case("norm_rope", "norm_rope_prompt", layout="packed", B=1, N=8191, Hq=32, Hkv=8, D=128, rot=64,
              interleaved=False, norm=False, dtype="fp16"),
        # One step of 64 running sequences: norm, rotation and append in one call.
        _case("append", "append_step", fmt="16bit", layout="HND", B=64, mix=41, new_lo=1, new_hi=1, len_lo=256,
              len_hi=2048, page=16, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, norm=True, dtype="bf16"),
        # 16 prompts of mixed length quantized into an FP4 cache, then read back.
        _case("append", "append_prompts_fp4", fmt="fp4", layout="HND", B=16, mix=41, new_lo=256, new_hi=2048,
              len_lo=256, len_hi=4096, page=64, Hq=32, Hkv=8, D=128, rot=128, interleaved=False, norm=True,
              dtype="bf16"),
        # The cached tokens of 16 mixed sequences as dense keys and values (a prompt that continues a cache).
        _case("gather", "gather_prefix_fp4", fmt="fp4", layout="HND", B=16, mix=41, new_lo=256, new_hi=16384,
              page=64, Hkv=8, D=128, dtype="bf16"),
        # A few short sequences from a token-major 16-bit cache with small heads and an uncommon page size.
        _case("gather", "gather_short_nhd", fmt="16bit", layout="NHD", B=5, mix=41, new_lo=1, new_hi=333,
              page=24, Hkv=16, D=64, dtype="fp16"),
        # One sequence, about a thousand tokens: the smallest attention step.
        _case("decode", "decode_one", fmt="16bit", layout="HND", B=1, mix=41, len_lo=1000, len_hi=1000, page=16,
              Hq=32, Hkv=8, D=128, dtype="bf16"),
        # The mixed batch of prompt lengths of the packed workload, at its decode steps.
        _case("decode", "decode_mix", fmt="16bit", layout="HND", B=16, mix=41, len_lo=256, len_hi=16384,
              page=16, Hq=32, Hkv=8, D=128, dtype="bf16"),
        # No head sharing, small heads, token-major pages.
        _case("decode", "decode_heads_d64", fmt="16bit", layout="NHD", B=8, mix=41, len_lo=2000, len_hi=8192,
              page=64, Hq=16, Hkv=16, D=64, dtype="fp16"),
        # A large batch over an FP4 cache.
        _case("decode", "decode_batch_fp4", fmt="fp4", layout="HND", B=64, mix=41, len_lo=128, len_hi=8192,
              page=64, Hq=32, Hkv=8, D=128, dtype="bf16"),
        # One very long sequence over an FP4 cache.
        _case("decode", "decode_long_fp4", fmt="fp4", layout="HND", B=1, mix=41, len_lo=131071, len_hi=131071,
              page=128, Hq=32, Hkv=8, D=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm_rope", "append", "gather", "decode", "decode"))
    D = rng.choice((64, 128))
    dtype = rng.choice(("bf16", "fp16"))
    Hkv = rng.choice((1, 2, 3, 4, 8, 8, 16))
    group = rng.choice((1, 2, 4, 4, 7, 8, 12, 16))
    if Hkv * group > 64:
        group = 4
    rot = rng.choice([r for r in (0, 32, 64, 96, 128) if r <= D] + [D, D])
    common = {"D": D, "dtype": dtype, "Hkv": Hkv}
    rope = {"rot": rot, "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.6}
    if op == "norm_rope":
        layout = rng.choice(("packed", "HND", "NHD"))
        most = 32768 * 24 * 2 * 128 // ((Hkv * group + Hkv) * D)
        tokens = _log(rng, 1, min(most, 65536))
        B = 1 if layout == "packed" else rng.randint(1, min(4, tokens))
        return _case(op, layout=layout, B=B, N=tokens // B, Hq=Hkv * group, **common, **rope)
    paged = {"fmt": rng.choice(("16bit", "fp4")), "layout": rng.choice(("HND", "NHD")),
             "page": rng.choice((8, 16, 16, 24, 32, 64, 128, 256)), "mix": rng.randint(0, 1 << 20)}
    if op in ("append", "gather"):
        B = _log(rng, 1, 128)
        most = 32768 * 24 * 2 * 128 // (Hkv * (group + 2) * D)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, min(32768, most) // B)
        lo = rng.randint(1, new)
        if op == "gather":
            return _case(op, B=B, new_lo=lo, new_hi=new, **paged, **common)
        return _case(op, B=B, new_lo=lo, new_hi=new, len_lo=new, len_hi=new + _log(rng, 1, 2048),
                     Hq=Hkv * group, **paged, **common, **rope)
    B = _log(rng, 1, 128)
    most = min(131072, 64 * 8192 * 8 * 128 // (B * Hkv * D * (4 if paged["fmt"] == "16bit" else 1)))
    hi = _log(rng, 1, most)
    return _case(op, B=B, len_lo=rng.randint(max(1, hi // 8), hi), len_hi=hi, Hq=Hkv * group, **paged, **common)


# ------------------------------------------------------------------------------ inputs --

def _lens(c, lo, hi):
    """The lengths belong to the case: two seeds differ in what the tokens hold and where they lie."""
    g = torch.Generator().manual_seed(c["mix"])
    return torch.randint(c[lo], c[hi] + 1, (c["B"],), generator=g).tolist()


def _rope_table(positions, rot):
    """cos of the rot/2 angles, then their sin, for every position: [positions, rot]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def _pages(s, g, lens, page):
    """A page table whose pages lie in random order, as in a cache that has been in use."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["page_table"] = table.cuda()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    return pages


def _cache(s, c, gen, pages):
    """The cache's buffers with keys and values of a running model in them."""
    H, P, D, dt = c["Hkv"], c["page"], c["D"], DTYPES[c["dtype"]]
    shape = (pages, H, P) if c["layout"] == "HND" else (pages, P, H)
    bias = torch.randn((H, D), generator=gen, device="cuda") * 2.0
    bias = bias[:, None, :] if c["layout"] == "HND" else bias
    for name in ("k", "v"):
        if c["fmt"] == "16bit":
            x = torch.randn(shape + (D,), generator=gen, device="cuda", dtype=dt)
            s[name + "_cache"] = x.add_(bias.to(dt)) if name == "k" else x
        else:
            codes = torch.empty(shape + (D // 2,), dtype=torch.uint8, device="cuda")
            scales = torch.empty(shape + (D // 16,), dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 26) // (H * P * D))
            for p in range(0, pages, step):
                x = torch.randn((min(step, pages - p),) + shape[1:] + (D,), generator=gen, device="cuda")
                codes[p:p + step], scales[p:p + step] = _quantize(x + bias if name == "k" else x)
            s[name + "_cache"], s[name + "_sf"] = codes, scales


def _rope_inputs(s, c, gen, positions):
    dt = DTYPES[c["dtype"]]
    s["rope"] = _rope_table(positions, c["rot"]) if c["rot"] else None
    for name in ("q_weight", "k_weight"):
        s[name] = (1.0 + 0.1 * torch.randn(c["D"], generator=gen, device="cuda")).to(dt) if c["norm"] else None


def prepare(case, seed):
    c = case
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    D, dt = c["D"], DTYPES[c["dtype"]]
    s = {"case": c}

    def rows(*shape):
        return torch.randn(shape + (D,), generator=gen, device="cuda", dtype=dt)

    if c["op"] == "norm_rope":
        B, N = c["B"], c["N"]
        if c["layout"] == "packed":
            s["q"], s["k"] = rows(N, c["Hq"]), rows(N, c["Hkv"])
            s["positions"] = torch.randint(0, 2 * N, (N,), generator=g).to(torch.int32).cuda()
        else:
            hnd = c["layout"] == "HND"
            s["q"], s["k"] = (rows(B, h, N) if hnd else rows(B, N, h) for h in (c["Hq"], c["Hkv"]))
            s["positions"] = None
        _rope_inputs(s, c, gen, 2 * N)
        return s
    if c["op"] == "decode":
        lens = _lens(c, "len_lo", "len_hi")
        s["q"] = rows(c["B"], c["Hq"])
    else:
        new = _lens(c, "new_lo", "new_hi")
        old = _lens(c, "len_lo", "len_hi") if c["op"] == "append" else new
        lens = [max(n, o) for n, o in zip(new, old)]
        s["total"] = sum(new)
        s["cu_seqlens"] = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()
        if c["new_hi"] == 1:
            s["cu_seqlens"] = None  # one token of each sequence
    pages = _pages(s, g, lens, c["page"])
    _cache(s, c, gen, pages)
    if c["op"] == "append":
        T = s["total"]
        s["q"], s["k"], s["v"] = rows(T, c["Hq"]), rows(T, c["Hkv"]), rows(T, c["Hkv"])
        _rope_inputs(s, c, gen, max(lens))
    if own:  # the handle that a program keeps for its cache
        import microscaling_fp4_quantized_b200 as sage
        s["cache"] = sage.PagedKVCache(s["k_cache"], s["v_cache"], s.get("k_sf"), s.get("v_sf"), dtype=dt,
                                       tensor_layout=c["layout"])
    return s


# -------------------------------------------------------------------------- plain forms --

def _norm(x, w, wide):
    """x / rms(x) * w over the last axis, in 32 bits; the mean square in 64 where the result
    goes on to a 4-bit rounding."""
    if w is None:
        return x
    t = x.double() if wide else x
    r = torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS).float()
    return x * r * w.float()


def _rotate(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    y = x.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _norm_rotate(x, w, rope, pos, head_axis, interleaved, wide=False):
    """x with tokens on the axes of `pos` (the last of them may be broadcast) and heads on head_axis."""
    x = _norm(x.float(), w, wide)
    if rope is None:
        return x
    cs = rope[pos.long()].unsqueeze(head_axis)
    half = cs.shape[-1] // 2
    return _rotate(x, cs[..., :half], cs[..., half:], interleaved)


def _quantize(x):
    """E2M1 codes (two per byte, even element low) and E4M3 scales, one per 16 elements: scale
    = absmax / 6, codes = x / scale, both to the nearest with ties to even, in IEEE 32-bit steps."""
    b = x.unflatten(-1, (-1, 16))
    a = b.abs().amax(-1)
    sf = (a / torch.full_like(a, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = sf.float().unsqueeze(-1)
    y = torch.where(s > 0, b / s, torch.zeros_like(b)).abs()
    code = (y > 0.25).to(torch.uint8)
    code += y >= 0.75
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5.0
    code += 8 * (torch.signbit(b) & (s > 0)).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sf.view(torch.uint8)


def _decode(codes, sf):
    lut = torch.tensor(E2M1, device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), dim=-1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * sf.view(torch.float8_e4m3fn).float().unsqueeze(-1)).flatten(-2)


def _slots(s, c):
    """Page and slot of every new token, and its position."""
    lens, table, dev = s["seq_lens"].long(), s["page_table"], s["page_table"].device
    cu = torch.arange(len(lens) + 1, device=dev) if s["cu_seqlens"] is None else s["cu_seqlens"].long()
    tok = torch.arange(s["total"], device=dev)
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = tok - cu[b + 1] + lens[b]
    return table[b, pos // c["page"]].long(), pos % c["page"], pos


def _at(x, page, slot, layout):
    """Rows [tokens, heads, .] of a cache buffer."""
    return x[page, :, slot] if layout == "HND" else x[page, slot]


def _put(x, page, slot, layout, rows):
    if layout == "HND":
        x[page, :, slot] = rows
    else:
        x[page, slot] = rows


def _plain_gather(s, c, page, slot):
    out = []
    for name in ("k", "v"):
        x = _at(s[name + "_cache"], page, slot, c["layout"])
        if c["fmt"] == "fp4":
            x = _decode(x, _at(s[name + "_sf"], page, slot, c["layout"])).to(DTYPES[c["dtype"]])
        out.append(x)
    return out


def _plain_decode(s, c):
    q, table, lens = s["q"], s["page_table"].long(), s["seq_lens"]
    B, Hq, D = q.shape
    kv = []
    for name in ("k", "v"):
        x = s[name + "_cache"][table]
        x = _decode(x, s[name + "_sf"][table]) if c["fmt"] == "fp4" else x.float()
        x = x.transpose(2, 3) if c["layout"] == "NHD" else x  # [B, pages, H, page, D]
        kv.append(x.transpose(1, 2).flatten(2, 3))             # [B, H, tokens, D]
    k, v = kv
    qg = q.float().view(B, c["Hkv"], Hq // c["Hkv"], D)
    sc = qg @ k.transpose(-1, -2) * (1.0 / math.sqrt(D))
    off = torch.arange(k.shape[2], device=q.device)[None, :] >= lens[:, None]
    sc = sc.masked_fill(off[:, None, None, :], float("-inf"))
    p = (sc - sc.amax(-1, keepdim=True)).exp()
    return ((p @ v) / p.sum(-1, keepdim=True)).view(B, Hq, D).to(q.dtype)


def _plain(s, c):
    dt = DTYPES[c["dtype"]]
    if c["op"] == "norm_rope":
        pos = s["positions"] if c["layout"] == "packed" else torch.arange(c["N"], device=s["q"].device)
        axis = 0 if c["layout"] == "HND" else 1
        return [_norm_rotate(s[n], s[n + "_weight"], s["rope"], pos, axis, c["interleaved"]).to(dt) for n in ("q", "k")]
    if c["op"] == "decode":
        return _plain_decode(s, c)
    page, slot, pos = _slots(s, c)
    if c["op"] == "gather":
        return _plain_gather(s, c, page, slot)
    q, k = (_norm_rotate(s[n], s[n + "_weight"], s["rope"], pos, 1, c["interleaved"], c["fmt"] == "fp4")
            for n in ("q", "k"))
    for name, x in (("k", k), ("v", s["v"].float())):
        if c["fmt"] == "16bit":
            _put(s[name + "_cache"], page, slot, c["layout"], x.to(dt))
        else:
            codes, sf = _quantize(x)
            _put(s[name + "_cache"], page, slot, c["layout"], codes)
            _put(s[name + "_sf"], page, slot, c["layout"], sf)
    if c["fmt"] == "16bit":
        return [q.to(dt), s["k_cache"], s["v_cache"]]
    return [q.to(dt)] + _plain_gather(s, c, page, slot)


# ---------------------------------------------------------------------------------- run --

def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain(s, c)
    import microscaling_fp4_quantized_b200 as sage
    if c["op"] == "norm_rope":
        return sage.qk_norm_rope(s["q"], s["k"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, rope=s["rope"],
                                 positions=s["positions"], interleaved=c["interleaved"],
                                 tensor_layout="HND" if c["layout"] == "packed" else c["layout"])
    if c["op"] == "decode":
        return sage.sageattn_decode(s["q"], s["cache"], s["page_table"], s["seq_lens"])
    if c["op"] == "gather":
        return sage.cache_gather(s["cache"], s["page_table"], s["seq_lens"], cu_seqlens=s["cu_seqlens"],
                                 total=s["total"])
    q = sage.cache_append(s["cache"], s["k"], s["v"], s["page_table"], s["seq_lens"], cu_seqlens=s["cu_seqlens"],
                          q=s["q"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, rope=s["rope"],
                          interleaved=c["interleaved"])
    if c["fmt"] == "16bit":
        return [q, s["k_cache"], s["v_cache"]]
    # What 4-bit pages hold is read back as the values it stands for.
    k, v = sage.cache_gather(s["cache"], s["page_table"], s["seq_lens"], cu_seqlens=s["cu_seqlens"], total=s["total"])
    return [q, k, v]


def work(case):
    c = case
    D, esz = c["D"], (9 / 16 if c.get("fmt") == "fp4" else 2.0)
    if c["op"] == "norm_rope":
        rows = c["B"] * c["N"] * (c["Hq"] + c["Hkv"])
        table = c["N"] * c["rot"] * 4
        return {"bytes": rows * D * 4 + table, "flops": rows * D * ((4 if c["norm"] else 0) + 3)}
    if c["op"] == "decode":
        tokens = sum(_lens(c, "len_lo", "len_hi"))
        return {"bytes": tokens * c["Hkv"] * D * 2 * esz + c["B"] * c["Hq"] * D * 4 + tokens / c["page"] * 4,
                "flops": 4.0 * tokens * c["Hq"] * D}
    tokens = sum(_lens(c, "new_lo", "new_hi"))
    if c["op"] == "gather":
        return {"bytes": tokens * c["Hkv"] * D * 2 * (2 + esz), "flops": 0}
    rows = tokens * (c["Hq"] + c["Hkv"])
    moved = tokens * D * (4 * c["Hq"] + 2 * c["Hkv"] * (2 + esz)) + tokens * c["rot"] * 4
    if c["fmt"] == "fp4":
        moved += tokens * c["Hkv"] * D * 2 * (2 + esz)  # read back
    return {"bytes": moved, "flops": rows * D * ((4 if c["norm"] else 0) + 3)}


# -------------------------------------------------------------------------------- exact --

def _exact_rows(x, w, rope, pos, interleaved):
    """x [tokens, heads, D] in 64 bits: each token's heads normed, then turned as complex numbers."""
    z = x.to(torch.float64)
    if w is not None:
        z = z / (z.pow(2).sum(-1, keepdim=True) / z.shape[-1] + EPS).sqrt() * w.to(torch.float64)
    if rope is not None:
        R = rope.shape[1]
        turn = torch.complex(*rope.to(torch.float64)[pos.long()].chunk(2, dim=1))[:, None, :]
        head = z[..., :R]
        pairs = head.reshape(*head.shape[:-1], R // 2, 2) if interleaved else \
            head.reshape(*head.shape[:-1], 2, R // 2).transpose(-1, -2)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        y = y.flatten(-2) if interleaved else y.transpose(-1, -2).flatten(-2)
        z = torch.cat((y, z[..., R:]), dim=-1)
    return z


def _exact_rows_of(s, name, b, n, c):
    """The first n cached rows of sequence b, [n, heads, D], in 64 bits."""
    idx = s["page_table"][b, :-(-n // c["page"])].long()

    def dense(x):
        x = x[idx] if c["layout"] == "NHD" else x[idx].permute(0, 2, 1, 3)
        return x.reshape(-1, *x.shape[2:])[:n]

    x = dense(s[name + "_cache"])
    if c["fmt"] == "16bit":
        return x.to(torch.float64)
    sf = dense(s[name + "_sf"]).view(torch.float8_e4m3fn).to(torch.float64)
    lut = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    both = torch.stack((x % 16, x // 16), dim=-1).reshape(*x.shape[:-1], -1)
    return lut[both.long()] * sf.repeat_interleave(16, dim=-1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    D = c["D"]
    if c["op"] == "norm_rope":
        out = []
        for n in ("q", "k"):
            x = s[n]
            if c["layout"] == "packed":
                out.append(_exact_rows(x, s[n + "_weight"], s["rope"], s["positions"], c["interleaved"]))
                continue
            t = x if c["layout"] == "NHD" else x.transpose(1, 2)
            pos = torch.arange(c["N"], device=x.device).repeat(c["B"])
            y = _exact_rows(t.reshape(-1, *t.shape[2:]), s[n + "_weight"], s["rope"], pos, c["interleaved"])
            y = y.reshape(t.shape)
            out.append(y if c["layout"] == "NHD" else y.transpose(1, 2))
        return out
    lens = s["seq_lens"].tolist()
    if c["op"] == "decode":
        out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            k, v = (_exact_rows_of(s, name, b, n, c) for name in ("k", "v"))
            qh = s["q"][b].to(torch.float64).reshape(c["Hkv"], -1, D)
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", qh, k) / D ** 0.5, dim=-1)
            out[b] = torch.einsum("hgn,nhd->hgd", w, v).reshape(-1, D)
        return out
    new = [1] * len(lens) if s["cu_seqlens"] is None else s["cu_seqlens"].diff().tolist()
    if c["op"] == "gather":
        return [torch.cat([_exact_rows_of(s, name, b, n, c)[n - m:] for b, (n, m) in enumerate(zip(lens, new))])
                for name in ("k", "v")]
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, new)]).cuda()
    q, k = (_exact_rows(s[n], s[n + "_weight"], s["rope"], pos, c["interleaved"]) for n in ("q", "k"))
    if c["fmt"] == "fp4":
        return [q, None, None]  # what a 4-bit rounding leaves has no value of its own in 64 bits
    out = [q]
    for name, rows in (("k", k), ("v", s["v"].to(torch.float64))):
        buf = s[name + "_cache"].to(torch.float64)
        at = 0
        for b, (n, m) in enumerate(zip(lens, new)):
            p = torch.arange(n - m, n)
            page, slot = s["page_table"][b].cpu()[p // c["page"]].long().cuda(), (p % c["page"]).cuda()
            if c["layout"] == "HND":
                buf[page, :, slot] = rows[at:at + m]
            else:
                buf[page, slot] = rows[at:at + m]
            at += m
        out.append(buf)
    return out
