"""Paged cache operators on the GPU against plain 64-bit implementations.

Tolerances. u = eps / 2 of the output type (one rounding: half a step, relative). Norm and rotation run in
binary32: the mean square is a sum of at most 4 fused steps per accumulator, 3 additions in the lane and 3 over
lanes, its scaling and eps (12 roundings of 2^-24, halved by the root), the reciprocal root is good to 2 units
in the last place (4 x 2^-24), then two products, the rotation's product and its sum: 14, bounded by 16;
attention adds its own terms (decode_tolerance). FP4 codes and scales, copies and reads are exact.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half a step of fp16's subnormals
BF, HF = torch.bfloat16, torch.float16
EPS = 1e-6


@pytest.fixture(scope="module")
def sage():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import microscaling_fp4_quantized_b200 as s
    s.lib()
    s.device_error()
    return s


@pytest.fixture(autouse=True)
def no_device_error(sage):
    yield
    assert sage.device_error() == 0


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, dtype=BF):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------- plain implementations --

def rows64(x, w, rope, pos, interleaved):
    """[tokens, heads, D] in binary64 (tables and weights as given); and the bound on the 32-bit steps."""
    z = x.double()
    if w is not None:
        z = z / torch.sqrt((z * z).mean(-1, keepdim=True) + EPS) * w.double()
    mag = z.abs()
    if rope is not None:
        R = rope.shape[1]
        c, s = (t[:, None, :] for t in rope.double()[pos.long()].split(R // 2, dim=1))
        a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        y, m = z.clone(), mag.clone()
        y[..., a], y[..., b] = z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s
        m[..., a] = mag[..., a] * c.abs() + mag[..., b] * s.abs()
        m[..., b] = mag[..., b] * c.abs() + mag[..., a] * s.abs()
        z, mag = y, m
    return z, 16 * 2.0 ** -24 * mag


def assert_rounded(got, want, slack, dtype):
    tol = U[dtype] * (want.abs() + slack) + slack + TINY[dtype]
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() - tol).max()))


def rows32(x, w, rope, pos, interleaved):
    """The same steps in binary32, each rounded on its own and the mean square in binary64 (on the CPU)."""
    z = x.float().cpu()
    if w is not None:
        ms = (z.double() * z.double()).mean(-1, keepdim=True) + float(np.float32(EPS))
        z = z * (1.0 / torch.sqrt(ms)).float() * w.float().cpu()
    if rope is not None:
        R = rope.shape[1]
        c, s = (t[:, None, :] for t in rope.cpu()[pos.long().cpu()].split(R // 2, dim=1))
        a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        y = z.clone()
        y[..., a], y[..., b] = z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s
        z = y
    return z


def quantized(oracle_mod, x):
    """Oracle codes and scale bytes of float rows [tokens, heads, D]."""
    return oracle_mod.quantize_rows(x.numpy())


def decoded(oracle_mod, codes, sf):
    v = oracle_mod.e2m1_decode(oracle_mod.unpack_fp4(codes))
    return v * np.repeat(oracle_mod.e4m3_decode(sf), 16, axis=-1)


class Case:
    """Sequences in a paged cache: pages in random order, slots never written hold NaN (FP4: the NaN scale)."""

    def __init__(self, sage, lens, page, Hkv, D, dtype=BF, fmt="16bit", layout="HND", spare=2, pad=0, seed=0, width=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), max([1] + need) if width is None else width), 2 ** 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.lens, self.page, self.Hkv, self.D, self.dtype, self.fmt, self.layout = lens, page, Hkv, D, dtype, fmt, layout
        self.table, self.seq_lens = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        shape = (self.pages, Hkv, page) if layout == "HND" else (self.pages, page, Hkv)

        def buf(width, fill, dt):
            # `pad` extra heads (HND) or rows make the strides larger than the shape
            full = torch.full((shape[0], shape[1] + pad, shape[2], width), fill, dtype=dt, device="cuda")
            return full[:, :shape[1]]

        if fmt == "16bit":
            self.k, self.v = (buf(D, float("nan"), dtype) for _ in range(2))
            self.cache = sage.PagedKVCache(self.k, self.v, tensor_layout=layout)
        else:
            self.k, self.v = (buf(D // 2, 0x77, torch.uint8) for _ in range(2))
            self.ks, self.vs = (buf(D // 16, 0x7F, torch.uint8) for _ in range(2))
            self.cache = sage.PagedKVCache(self.k, self.v, self.ks, self.vs, dtype=dtype, tensor_layout=layout)

    def cu(self, new):
        return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32).cuda()

    def places(self, new):
        """(page, slot, position) of the last new[b] tokens of every sequence."""
        table = self.table.cpu()
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(self.lens, new)] or [torch.zeros(0)]).long()
        b = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
        return table[b, pos // self.page].long().cuda(), (pos % self.page).cuda(), pos.cuda()

    def at(self, x, new):
        page, slot, _ = self.places(new)
        return x[page, :, slot] if self.layout == "HND" else x[page, slot]

    def fill(self, oracle_mod, seed, scale=1.0):
        """Keys and values of all tokens; kv64[b] = (k, v) in binary64 as the cache holds them."""
        g = gen(seed)
        T = sum(self.lens)
        page, slot, _ = self.places(self.lens)
        dense = []
        for name in ("k", "v"):
            x = torch.randn((T, self.Hkv, self.D), generator=g, device="cuda") * scale
            if name == "k":
                x += torch.randn((self.Hkv, self.D), generator=g, device="cuda")
            if self.fmt == "16bit":
                x = x.to(self.dtype)
                put(getattr(self, name), page, slot, self.layout, x)
                dense.append(x.double())
            else:
                codes, sf = quantized(oracle_mod, x.cpu())
                put(getattr(self, name), page, slot, self.layout, torch.from_numpy(codes).cuda())
                put(getattr(self, name + "s"), page, slot, self.layout, torch.from_numpy(sf).cuda())
                dense.append(torch.from_numpy(decoded(oracle_mod, codes, sf)).cuda())
        self.kv64 = list(zip(*(x.split(self.lens) for x in dense)))
        return self


def put(x, page, slot, layout, rows):
    if layout == "HND":
        x[page, :, slot] = rows
    else:
        x[page, slot] = rows


def decode64(q, k, v, sm):
    """One sequence: q [Hq, D], k, v [n, Hkv, D] -> out [Hq, D] and its tolerance, all binary64.

    Weights w~ = w (1 + d): |d| <= u_p (their rounding: U[fp16] on FP4 caches; on 16-bit ones a second operand holds
    what the first rounding left, U^2) + e (error of the exponent: the
    score's binary32 sums, D steps and the scaling, relative to the sum of magnitudes, and the exp2
    approximation's 2^-22, plus the magnitude of the exponent itself times 2^-23). Normalised by their
    own sum, the result is off by at most 2 max|d| sum w |v|; the binary32 accumulation over n / 16 steps per
    warp adds n 2^-24 of it, and weights below fp16's subnormals at most 2^-29 |v| each."""
    Hq, D = q.shape
    n, Hkv = k.shape[:2]
    qd = q.double().view(Hkv, Hq // Hkv, D)
    s = torch.einsum("hgd,nhd->hgn", qd, k) * sm
    w = torch.softmax(s, dim=-1)
    out = torch.einsum("hgn,nhd->hgd", w, v)
    amag = torch.einsum("hgn,nhd->hgd", w, v.abs())
    smag = (torch.einsum("hgd,nhd->hgn", qd.abs(), k.abs()) * sm).amax(-1, keepdim=True)
    d = smag * (D + 8) * 2.0 ** -23 + 2.0 ** -21
    vmax = v.abs().amax(0)[:, None, :]
    return out.reshape(Hq, D), amag.reshape(Hq, D), (2 * d * amag + n * 2.0 ** -24 * amag + n * 2.0 ** -29 * vmax).reshape(Hq, D)


def check_decode(case, q, out, sm=None):
    sm = sm or case.D ** -0.5
    up = U[HF] if case.fmt == "fp4" else U[case.dtype] ** 2
    u = U[case.dtype]
    worst = 0.0
    for b, n in enumerate(case.lens):
        if n == 0:
            assert not out[b].any()
            continue
        k, v = case.kv64[b]
        want, amag, slack = decode64(q[b], k, v, sm)
        tol = u * want.abs() + (2 * up * amag + slack) * (1 + u) + TINY[case.dtype]
        err = (out[b].double() - want).abs()
        assert torch.isfinite(out[b]).all(), b
        worst = max(worst, float((err / tol).max()))
        assert (err <= tol).all(), (b, n, float((err / tol).max()))
    return worst


# ------------------------------------------------------------------------- norm and rotation --

@pytest.mark.parametrize("layout,B,N,Hq,Hkv,D,rot,inter,norm,dtype", [
    ("HND", 2, 37, 3, 1, 64, 64, False, True, BF), ("NHD", 1, 130, 8, 2, 128, 128, True, True, HF),
    ("packed", 1, 1, 1, 1, 128, 128, False, True, BF), ("packed", 1, 5, 5, 5, 64, 32, True, True, HF),
    ("HND", 3, 17, 6, 2, 128, 96, False, True, BF), ("NHD", 2, 9, 20, 4, 128, 32, False, False, HF),
    ("packed", 1, 1000, 17, 1, 128, 64, True, False, BF), ("HND", 1, 300, 2, 2, 64, 0, False, True, HF),
    ("NHD", 1, 2050, 24, 8, 128, 128, False, True, BF),
])
def test_norm_rope(sage, layout, B, N, Hq, Hkv, D, rot, inter, norm, dtype):
    g = gen(N)
    shape = lambda H: {"HND": (B, H, N, D), "NHD": (B, N, H, D), "packed": (N, H, D)}[layout]  # noqa: E731
    q, k = randn(g, *shape(Hq), dtype=dtype), randn(g, *shape(Hkv), dtype=dtype)
    qw, kw = (randn(g, D, dtype=dtype) if norm else None for _ in range(2))
    rope = sage.rope_table(4 * N, rot) if rot else None
    pos = torch.randint(0, 4 * N, (N,) if layout == "packed" else (B, N), generator=g, device="cuda", dtype=torch.int32)
    lay = "HND" if layout == "packed" else layout
    kw_args = dict(q_weight=qw, k_weight=kw, rope=rope, interleaved=inter, tensor_layout=lay, positions=pos, eps=EPS)
    qo, ko = sage.qk_norm_rope(q, k, **kw_args)
    for x, w, y in ((q, qw, qo), (k, kw, ko)):
        t = lambda z: (z if layout == "packed" else z.transpose(1, 2) if layout == "HND" else z).reshape(-1, x.shape[1 if layout != "NHD" else 2], D)  # noqa: E731,B023
        want, slack = rows64(t(x), w, rope, pos.reshape(-1), inter)
        assert_rounded(t(y), want, slack, dtype)
    # in place, queries alone
    q2 = q.clone()
    kw_args["k_weight"] = None
    got, none = sage.qk_norm_rope(q2, q_out=q2, **kw_args)
    assert got is q2 and none is None and torch.equal(q2, qo)


@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 128, True), (128, 96, False), (64, 32, True)])
def test_rotation_rounds_every_step(sage, D, rot, inter):
    """Without a norm a rotation is two products and their sum, each rounded to binary32, and the rounding to fp16: bit for
    bit, over enough elements (two million) that a product left unrounded in the sum would show in hundreds of them."""
    N, H = 4096, 1024 // D // 2
    q, pos = randn(gen(7), N, H, D, dtype=HF), torch.arange(N, dtype=torch.int32, device="cuda")
    rope = sage.rope_table(N, rot)
    want = rows32(q, None, rope, pos, inter).to(HF).cuda()
    assert torch.equal(sage.qk_norm_rope(q, rope=rope, positions=pos, interleaved=inter)[0], want)
    c = Case(sage, [N], 16, H, D, HF)
    sage.cache_append(c.cache, q, q, c.table, c.seq_lens, cu_seqlens=c.cu([N]), rope=rope, interleaved=inter)
    assert torch.equal(c.at(c.k, [N]), want) and torch.equal(c.at(c.v, [N]), q)


def test_norm_rope_default_positions_strides_and_weights(sage):
    g = gen(5)
    B, N, H, D = 2, 33, 4, 128
    big = randn(g, B, N, 3 * H, D)  # a fused projection: q and k are slices of it
    q, k = big[:, :, :H], big[:, :, H:2 * H]
    rope = sage.rope_table(N, D)
    w = (torch.randn(D, generator=g, device="cuda"))  # float32 weights
    qo, ko = sage.qk_norm_rope(q, k, q_weight=w, k_weight=w, rope=rope, tensor_layout="NHD")
    pos = torch.arange(N, device="cuda").repeat(B)
    for x, y in ((q, qo), (k, ko)):
        want, slack = rows64(x.reshape(-1, H, D), w, rope, pos, False)
        assert_rounded(y.reshape(-1, H, D), want, slack, BF)
    # the norm of q alone; k only turns
    qo, ko = sage.qk_norm_rope(q, k, q_weight=w, rope=rope, tensor_layout="NHD")
    want, slack = rows64(k.reshape(-1, H, D), None, rope, pos, False)
    assert_rounded(ko.reshape(-1, H, D), want, slack, BF)
    # into a strided output, whose other channels stay
    out = torch.full_like(big, 7.0)
    sage.qk_norm_rope(q, rope=rope, tensor_layout="NHD", q_out=out[:, :, :H])
    assert (out[:, :, H:] == 7.0).all()


def test_norm_rope_extremes(sage):
    D = 128
    x = torch.zeros(6, 1, D, dtype=BF, device="cuda")
    x[1] = 1e-20
    x[2] = 3e38          # the mean square leaves binary32
    x[3, 0, 5] = float("inf")
    x[4, 0, 5] = float("nan")
    x[5] = 2.0 ** -133   # subnormal
    w = torch.ones(D, dtype=BF, device="cuda")
    y, _ = sage.qk_norm_rope(x, q_weight=w, eps=0.0)
    assert torch.isnan(y[0]).all()                       # 0 / 0, as the formula has it
    assert (y[1].float() - 1).abs().max() <= 2.0 ** -8 and (y[2].float() - 1).abs().max() <= 2.0 ** -8
    assert torch.isnan(y[3, 0, 5]) and not y[3, 0, :5].any()   # inf / inf; finite / inf
    assert torch.isnan(y[4]).all()
    assert (y[5].float() - 1).abs().max() <= 2.0 ** -8
    y, _ = sage.qk_norm_rope(x, q_weight=w, eps=1e-6)
    assert not y[0].any()


def test_norm_rope_positions_outside_the_table(sage):
    g = gen(6)
    q = randn(g, 5, 2, 64)
    rope = sage.rope_table(10, 64)
    pos = torch.tensor([0, 10, 9, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    sage.qk_norm_rope(q, rope=rope, positions=pos, q_out=out)
    assert sage.device_error() == sage.DEV_ERR_SEQLENS
    assert (out[[1, 3, 4]] == 7.0).all()
    want, slack = rows64(q[[0, 2]], None, rope, pos[[0, 2]], False)
    assert_rounded(out[[0, 2]], want, slack, BF)


# ----------------------------------------------------------------------------- append, gather --

APPEND = [
    # lens (with the new tokens), new, page, Hkv, Hq, D, rot, interleaved, norm, layout, pad
    ([5, 1, 300, 64], [5, 1, 300, 64], 16, 2, 4, 128, 128, False, True, "HND", 0),
    ([70, 33, 0, 129], [1, 0, 0, 65], 7, 1, 3, 64, 64, True, True, "NHD", 1),
    ([1], [1], 1, 3, 0, 128, 96, False, True, "HND", 2),
    ([40, 41, 42], [17, 41, 3], 24, 4, 8, 64, 32, False, False, "NHD", 0),
    ([1000, 3], [999, 2], 256, 5, 0, 128, 0, False, False, "HND", 0),
    ([513, 90], [2, 90], 64, 8, 16, 128, 64, True, True, "HND", 1),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("lens,new,page,Hkv,Hq,D,rot,inter,norm,layout,pad", APPEND)
def test_append_and_gather(sage, oracle_mod, fmt, dtype, lens, new, page, Hkv, Hq, D, rot, inter, norm, layout, pad):
    c = Case(sage, lens, page, Hkv, D, dtype, fmt, layout, pad=pad, seed=len(lens))
    g = gen(sum(lens))
    T = sum(new)
    k, v = randn(g, T + 2, Hkv, D, dtype=dtype), randn(g, T + 2, Hkv, D, dtype=dtype)  # two rows behind the last sequence
    q = randn(g, T + 2, Hq, D, dtype=dtype) if Hq else None
    qw, kw = (randn(g, D, dtype=dtype) if norm else None for _ in range(2))
    rope = sage.rope_table(max(lens), rot) if rot else None
    before = [x.clone() for x in (c.k, c.v)]
    q_out = torch.full_like(q, 7.0) if Hq else None
    got = sage.cache_append(c.cache, k, v, c.table, c.seq_lens, cu_seqlens=c.cu(new), q=q, q_out=q_out,
                            q_weight=qw if Hq else None, k_weight=kw, eps=EPS, rope=rope, interleaved=inter)
    assert got is q_out
    page_, slot, pos = c.places(new)
    if Hq:
        want, slack = rows64(q[:T], qw, rope, pos, inter)
        assert_rounded(q_out[:T], want, slack, dtype)
        assert (q_out[T:] == 7.0).all()
    kd = rows32(k[:T], kw, rope, pos, inter)
    if fmt == "16bit":
        want, slack = rows64(k[:T], kw, rope, pos, inter)
        assert_rounded(c.at(c.k, new), want, slack, dtype)
        if not norm:
            assert torch.equal(c.at(c.k, new).cpu(), kd.to(dtype))     # the steps are rounded as stated
        assert torch.equal(c.at(c.v, new), v[:T])
    else:
        for rows, codes, sf in ((kd, c.k, c.ks), (v[:T].float().cpu(), c.v, c.vs)):
            wc, ws = quantized(oracle_mod, rows)
            np.testing.assert_array_equal(c.at(sf, new).cpu().numpy(), ws)
            np.testing.assert_array_equal(c.at(codes, new).cpu().numpy(), wc)
    # every other slot is as it was
    for x, y in zip((c.k, c.v), before):
        put(y, page_, slot, layout, c.at(x, new))
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
    # and back
    ko, vo = (torch.full((T + 2, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    sage.cache_gather(c.cache, c.table, c.seq_lens, cu_seqlens=c.cu(new), k_out=ko, v_out=vo)
    assert (ko[T:] == 7.0).all() and (vo[T:] == 7.0).all()
    if fmt == "16bit":
        assert torch.equal(ko[:T], c.at(c.k, new)) and torch.equal(vo[:T], v[:T])
    else:
        for rows, codes, sf in ((ko, c.k, c.ks), (vo, c.v, c.vs)):
            want = decoded(oracle_mod, c.at(codes, new).cpu().numpy(), c.at(sf, new).cpu().numpy())
            np.testing.assert_array_equal(rows[:T].double().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_append_one_token_each_from_strided_rows(sage, oracle_mod, fmt):
    lens = [5, 1, 64, 65, 17]
    c = Case(sage, lens, 16, 2, 128, BF, fmt)
    qkv = randn(gen(3), 5, 8, 128)  # q: heads 0-3, k: 4-5, v: 6-7, as one projection leaves them
    rope = sage.rope_table(65, 128)
    q = sage.cache_append(c.cache, qkv[:, 4:6], qkv[:, 6:], c.table, c.seq_lens, q=qkv[:, :4], rope=rope)
    ko, vo = sage.cache_gather(c.cache, c.table, c.seq_lens)
    new = [1] * 5
    pos = c.places(new)[2]
    want, slack = rows64(qkv[:, :4], None, rope, pos, False)
    assert_rounded(q, want, slack, BF)
    kd = rows32(qkv[:, 4:6], None, rope, pos, False)
    if fmt == "16bit":
        assert torch.equal(ko.cpu(), kd.to(BF)) and torch.equal(vo, qkv[:, 6:])
    else:
        for got, x in ((ko, kd), (vo, qkv[:, 6:].float().cpu())):
            np.testing.assert_array_equal(got.double().cpu().numpy(), decoded(oracle_mod, *quantized(oracle_mod, x)))
    # in place on the projection
    alias = qkv.clone()
    assert torch.equal(sage.cache_append(c.cache, qkv[:, 4:6], qkv[:, 6:], c.table, c.seq_lens, q=alias[:, :4],
                                         q_out=alias[:, :4], rope=rope), q)


def test_fp4_saturation(sage, oracle_mod):
    c = Case(sage, [4], 4, 1, 64, BF, "fp4")
    x = torch.zeros(4, 1, 64, dtype=BF, device="cuda")
    x[0, 0, :16] = torch.linspace(-3e38, 3e38, 16)
    x[1, 0, 3], x[1, 0, 4], x[1, 0, 5], x[1, 0, 20] = float("inf"), float("-inf"), float("nan"), 1.0
    x[2, 0, 7] = 1e-38
    sage.cache_append(c.cache, x, x, c.table, c.seq_lens, cu_seqlens=c.cu([4]))
    k, v = sage.cache_gather(c.cache, c.table, c.seq_lens, cu_seqlens=c.cu([4]), total=4)
    assert torch.equal(k, v)
    finite = x.float().nan_to_num(nan=3.3895e38, posinf=3.3895e38, neginf=-3.3895e38).cpu()
    np.testing.assert_array_equal(k.double().cpu().numpy(), decoded(oracle_mod, *quantized(oracle_mod, finite)))
    # the block of 1.0: E4M3(1/6) = 11/64 (neighbours 10/64 and 11/64), 64/11 = 5.8 -> 6, 6 * 11/64
    assert k[1, 0, 3] == 2688 and k[1, 0, 4] == -2688 and k[1, 0, 5] == 2688 and k[1, 0, 20] == 66 / 64


@pytest.mark.parametrize("dtype", [BF, HF])
def test_fp4_every_scale_at_every_border(sage, oracle_mod, dtype):
    """For every scale byte: the block's maximum, values on the borders between codes (ties), one step to either
    side of them, and their negatives; codes and scales bit for bit."""
    byte = torch.arange(1, 127, dtype=torch.uint8)
    s = byte.view(torch.float8_e4m3fn).float()[:, None]
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    on = (s * ties).to(dtype)  # at most 7 significant bits: exact
    step = lambda x, d: (x.view(torch.int16) + d).view(dtype)  # noqa: E731
    top = (s * 6).to(dtype)
    rows = []
    for v in (on, step(on, 1), step(on, -1)):
        half = torch.cat((v, top), dim=1)
        rows.append(torch.cat((half, -half), dim=1))
    x = torch.stack(rows, dim=1).reshape(-1, 16)
    x = torch.cat((x, x.new_zeros((-len(x)) % 8, 16))).reshape(-1, 1, 128).cuda()
    c = Case(sage, [len(x)], 16, 1, 128, dtype, "fp4")
    new = [len(x)]
    sage.cache_append(c.cache, x, x.flip(0), c.table, c.seq_lens, cu_seqlens=c.cu(new))
    for rows, codes, sf in ((x, c.k, c.ks), (x.flip(0), c.v, c.vs)):
        wc, ws = quantized(oracle_mod, rows.float().cpu())
        np.testing.assert_array_equal(c.at(sf, new).cpu().numpy(), ws)
        np.testing.assert_array_equal(c.at(codes, new).cpu().numpy(), wc)


@pytest.mark.parametrize("dtype,inter", [(BF, False), (HF, True)])
def test_fp4_codes_of_many_rows(sage, oracle_mod, dtype, inter):
    """Norm, rotation and quantization of eight million key elements, codes and scales bit for bit: enough for values
    within a step of binary32 of a border between two codes."""
    N, H, D = 8192, 8, 128
    c = Case(sage, [N], 64, H, D, dtype, "fp4")
    g = gen(19)
    k, w = randn(g, N, H, D, dtype=dtype), 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    rope = sage.rope_table(N, D)
    sage.cache_append(c.cache, k, k, c.table, c.seq_lens, cu_seqlens=c.cu([N]), k_weight=w, eps=EPS, rope=rope, interleaved=inter)
    kd = rows32(k, w, rope, torch.arange(N), inter)
    for rows, codes, sf in ((kd, c.k, c.ks), (k.float().cpu(), c.v, c.vs)):
        wc, ws = quantized(oracle_mod, rows)
        np.testing.assert_array_equal(c.at(sf, [N]).cpu().numpy(), ws)
        np.testing.assert_array_equal(c.at(codes, [N]).cpu().numpy(), wc)


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_bad_tables_are_reported_and_not_followed(sage, oracle_mod, fmt):
    lens = [20, 20, 20, 20]
    c = Case(sage, lens, 16, 2, 64, BF, fmt, width=2)
    g = gen(9)
    k, v, q = randn(g, 80, 2, 64), randn(g, 80, 2, 64), randn(g, 80, 4, 64)
    c.table[1, 0], c.table[3, 1] = -1, c.pages
    rope = sage.rope_table(19, 64)  # position 19 is beyond it
    q_out = torch.full_like(q, 7.0)
    before = c.k.clone()
    sage.cache_append(c.cache, k, v, c.table, c.seq_lens, cu_seqlens=c.cu(lens), q=q, rope=rope, q_out=q_out)
    assert sage.device_error() == sage.DEV_ERR_SEQLENS | sage.DEV_ERR_PAGES
    left = torch.zeros(80, dtype=torch.bool)
    left[20:36], left[76:80], left[[19, 39, 59]] = True, True, True
    assert (q_out[left] == 7.0).all() and not (q_out[~left] == 7.0).all(-1).any()
    ko, vo = (torch.full_like(k, 7.0) for _ in range(2))
    sage.cache_gather(c.cache, c.table, c.seq_lens, cu_seqlens=c.cu(lens), k_out=ko, v_out=vo)
    assert sage.device_error() == sage.DEV_ERR_PAGES
    nowhere = torch.zeros(80, dtype=torch.bool)
    nowhere[20:36], nowhere[76:80] = True, True
    assert (ko[nowhere] == 7.0).all() and (vo[nowhere] == 7.0).all()
    # lengths outside the table, tokens at negative positions, offsets that do not rise
    q_out.fill_(7.0)
    for bad_lens, cu in (([33, 20, 20, 20], [0, 20, 20, 20, 20]), ([-5, 20, 20, 20], [0, 2, 2, 2, 2]),
                         ([3, 20, 20, 20], [0, 9, 9, 9, 9]), ([20, 20, 20, 20], [5, 5, 5, 5, 5]),
                         ([20, 20, 20, 20], [-2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1])):
        before = c.k.clone().view(torch.uint8)
        sage.cache_append(c.cache, k[:9], v[:9], c.table, torch.tensor(bad_lens, dtype=torch.int32).cuda(),
                          cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), q=q[:9], q_out=q_out[:9])
        assert sage.device_error() & sage.DEV_ERR_SEQLENS, (bad_lens, cu)
    # attention: a page outside the cache counts as zeros, a length outside the table is clamped
    c2 = Case(sage, [32, 16], 16, 1, 64, BF, fmt, width=2).fill(oracle_mod, 1)
    qd = randn(g, 2, 2, 64)
    c2.table[0, 1] = 10 ** 9
    out = sage.sageattn_decode(qd, c2.cache, c2.table, c2.seq_lens)
    assert sage.device_error() == sage.DEV_ERR_PAGES
    for t in c2.kv64[0]:
        t[16:] = 0
    check_decode(c2, qd, out)
    c2.table[0, 1] = c2.table[0, 0]
    c2.kv64[0] = tuple(torch.cat((t[:16], t[:16])) for t in c2.kv64[0])
    for wrong, lens2 in (([99, -3], [32, 0]), ([2 ** 31 - 1, -2 ** 31], [32, 0])):
        out = sage.sageattn_decode(qd, c2.cache, c2.table, torch.tensor(wrong, dtype=torch.int32).cuda())
        assert sage.device_error() == sage.DEV_ERR_SEQLENS
        c2.lens = lens2
        check_decode(c2, qd, out)


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_left_out_tokens_leave_everything_as_it_was(sage, oracle_mod, fmt):
    """Tokens that are reported, and rows behind the last sequence, change neither codes nor scales nor outputs; those
    beside them in the same call go where they belong."""
    c = Case(sage, [20, 20, 20, 20], 16, 2, 64, BF, fmt, width=2).fill(oracle_mod, 5)
    g = gen(17)
    buffers = (c.k, c.v, c.ks, c.vs) if fmt == "fp4" else (c.k, c.v)
    whole = lambda: [x.clone().view(torch.uint8) for x in buffers]  # noqa: E731
    good = c.table.clone()
    bad_table = good.clone()
    bad_table[1, 0], bad_table[3, 1] = -1, c.pages
    rope19, low, top = sage.rope_table(19, 64), -2 ** 31, 2 ** 31 - 1
    E_LEN, E_PAGE = sage.DEV_ERR_SEQLENS, sage.DEV_ERR_PAGES
    same, none = [20] * 4, []
    for table, lens, cu, rope, err, rows in (  # rows: (row, sequence, position) of what is written
            (bad_table, same, [0, 20, 40, 60, 80], rope19, E_LEN | E_PAGE,
             [(i, 0, i) for i in range(19)] + [(36 + i, 1, 16 + i) for i in range(3)] + [(40 + i, 2, i) for i in range(19)]
             + [(60 + i, 3, i) for i in range(16)]),
            (good, [33, 20, 20, 20], [0, 20, 20, 20, 20], None, E_LEN, none),
            (good, [-5, 20, 20, 20], [0, 2, 2, 2, 2], None, E_LEN, none),
            (good, [3, 20, 20, 20], [0, 9, 9, 9, 9], None, E_LEN, [(6, 0, 0), (7, 0, 1), (8, 0, 2)]),
            (good, same, [5, 5, 5, 5, 5], None, E_LEN, none),
            (good, same, [low, top, top, top, top], None, E_LEN, none),
            (good, [low, top, 20, 20], [0, 1, 2, 2, 2], None, E_LEN, none),
            (good, same, [0, 0, 3, 3, 3], None, 0, [(0, 1, 17), (1, 1, 18), (2, 1, 19)])):
        total = 80 if cu[-1] == 80 else 9
        k, v, q = randn(g, total, 2, 64), randn(g, total, 2, 64), randn(g, total, 4, 64)
        q_out = torch.full_like(q, 7.0)
        want = whole()
        sage.cache_append(c.cache, k, v, table, torch.tensor(lens, dtype=torch.int32).cuda(),
                          cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), q=q, q_out=q_out, rope=rope)
        assert sage.device_error() == err, (lens, cu)
        row, b, pos = (torch.tensor([r[i] for r in rows], dtype=torch.long) for i in range(3))
        page, slot = table.cpu()[b, pos // 16].long().cuda(), (pos % 16).cuda()
        kd, vd = rows32(k.cpu()[row], None, rope, pos, False), v.float().cpu()[row]
        new = []
        if rows and fmt == "fp4":
            codes, scales = zip(quantized(oracle_mod, kd), quantized(oracle_mod, vd))
            new = [torch.from_numpy(x).cuda() for x in codes + scales]
        elif rows:
            new = [x.to(BF).cuda().view(torch.uint8) for x in (kd, vd)]
        for x, y in zip(want, new):
            put(x, page, slot, "HND", y)
        assert all(torch.equal(x, y) for x, y in zip(whole(), want)), (lens, cu)
        out = torch.full_like(q, 7.0).cpu()
        out[row] = rows32(q.cpu()[row], None, rope, pos, False).to(BF)
        assert torch.equal(q_out.cpu(), out), (lens, cu)


# -------------------------------------------------------------------------------------- decode --

DECODE = [
    # lens, page, Hkv, group, D, layout
    ([1], 16, 1, 1, 128, "HND"),
    ([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 0], 16, 2, 4, 128, "HND"),
    ([1000], 16, 8, 4, 128, "HND"),
    ([5, 333, 64], 7, 3, 7, 64, "NHD"),
    ([100, 3, 257], 1, 1, 8, 128, "NHD"),
    ([2000, 1, 900], 64, 2, 12, 128, "HND"),
    ([700, 50], 24, 2, 16, 64, "HND"),
    ([130, 64], 32, 1, 20, 128, "HND"),
    ([90, 77], 256, 2, 33, 64, "NHD"),
    ([0, 0], 16, 2, 2, 64, "HND"),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("lens,page,Hkv,group,D,layout", DECODE)
def test_decode(sage, oracle_mod, fmt, dtype, lens, page, Hkv, group, D, layout):
    c = Case(sage, lens, page, Hkv, D, dtype, fmt, layout, pad=1, seed=3).fill(oracle_mod, 11)
    q = randn(gen(12), len(lens), Hkv * group, D, dtype=dtype) * 2
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    check_decode(c, q, out)
    ws = torch.full((sage.decode_workspace_bytes(c.cache, c.table, c.seq_lens, q.shape[1]),), 0xFF, dtype=torch.uint8,
                    device="cuda")  # NaN wherever nothing was written
    assert torch.equal(out, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, workspace=ws))


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("B,Hkv,width", [(1, 1, 16), (1, 8, 64), (3, 8, 128), (16, 8, 40), (70, 8, 30), (300, 3, 8), (9, 2, 4096)])
def test_decode_by_pairs_and_by_shares(sage, oracle_mod, fmt, B, Hkv, width):
    """Tables of widths that take one CTA, a cluster of 2, 4 or 8 per pair, and (the last) shares: the split follows
    the table, the lengths may be anything in it, down to nothing."""
    g = torch.Generator().manual_seed(B)
    top = min(width * 16, 1200)
    lens = torch.randint(0, top + 1, (B,), generator=g).tolist()
    lens[0] = top
    c = Case(sage, lens, 16, Hkv, 64, BF, fmt, width=width).fill(oracle_mod, B)
    q = randn(gen(B + 1), B, Hkv * 3, 64)
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    check_decode(c, q, out)
    ws = torch.full((sage.decode_workspace_bytes(c.cache, c.table, c.seq_lens, q.shape[1]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    assert torch.equal(out, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, workspace=ws))


@pytest.mark.parametrize("fmt,D", [("16bit", 64), ("16bit", 128), ("fp4", 64), ("fp4", 128)])
@pytest.mark.parametrize("layout,Hkv,group,lens", [
    ("HND", 8, 2, [3000, 0, 1, 129, 64, 700]), ("NHD", 8, 2, [3000, 0, 1, 129, 64, 700]),
    ("HND", 24, 2, [0, 1500, 300]), ("NHD", 24, 2, [0, 1500, 300]),  # blocks left over
    ("NHD", 3, 40, [2000, 33]), ("HND", 2, 33, [2000, 33]),          # heads of a group in several chunks
    ("NHD", 100, 1, [500, 0, 90]), ("HND", 67, 3, [500, 1]), ("NHD", 601, 1, [200]),
])
def test_decode_heads_side_by_side_or_end_to_end(sage, oracle_mod, fmt, D, layout, Hkv, group, lens):
    """Wide tables, so that the tokens are dealt in shares: of one head each, with the blocks of all heads side by
    side, or, where the heads do not fill the machine, of all heads' tiles end to end."""
    c = Case(sage, lens, 16, Hkv, D, BF, fmt, layout, seed=5, width=4096).fill(oracle_mod, 35)
    q = randn(gen(36), len(lens), Hkv * group, D)
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    check_decode(c, q, out)
    ws = torch.full((sage.decode_workspace_bytes(c.cache, c.table, c.seq_lens, q.shape[1]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    assert torch.equal(out, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, workspace=ws))


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_decode_one_long_sequence(sage, oracle_mod, fmt):
    """More shares than any other case; the last tokens matter as much as the first."""
    c = Case(sage, [70001], 64, 1, 128, BF, fmt).fill(oracle_mod, 21)
    q = randn(gen(22), 1, 4, 128)
    check_decode(c, q, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens))


@pytest.mark.parametrize("fmt,D", [("16bit", 64), ("fp4", 128)])
def test_decode_more_pairs_than_shares(sage, oracle_mod, fmt, D):
    """Joins are then recorded per share."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 200, (700,), generator=g).tolist()
    c = Case(sage, lens, 16, 2, D, BF, fmt).fill(oracle_mod, 31)
    q = randn(gen(32), 700, 4, D)
    check_decode(c, q, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens))


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("qscale,kscale", [(40.0, 1.0), (1e-3, 1.0), (1.0, 30.0), (0.0, 1.0)])
def test_decode_peaked_and_flat_scores(sage, oracle_mod, fmt, qscale, kscale):
    """One key holding all the weight, and all keys the same; the running maximum rises often."""
    c = Case(sage, [513, 64, 2], 16, 2, 128, BF, fmt).fill(oracle_mod, 41, scale=kscale)
    q = randn(gen(42), 3, 8, 128) * qscale
    check_decode(c, q, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, sm_scale=0.1), sm=0.1)


def test_decode_identical_values_and_one_key(sage, oracle_mod):
    """All values equal: the output is that value, for any scores; a single key: its value, exactly."""
    for fmt in ("16bit", "fp4"):
        c = Case(sage, [777, 1], 16, 1, 64, HF, fmt).fill(oracle_mod, 51)
        page, slot, _ = c.places(c.lens)
        row = c.v[page[0], :, slot[0]].clone()
        put(c.v, page, slot, "HND", row.expand(778, *row.shape))
        if fmt == "fp4":
            srow = c.vs[page[0], :, slot[0]].clone()
            put(c.vs, page, slot, "HND", srow.expand(778, *srow.shape))
        _, v = sage.cache_gather(c.cache, c.table, c.seq_lens)
        out = sage.sageattn_decode(randn(gen(52), 2, 8, 64, dtype=HF), c.cache, c.table, c.seq_lens)
        assert torch.equal(out[1], v[1].expand(8, 64))
        assert ((out[0] - v[0]).abs().double() <= 2 * U[HF] * v[0].abs().double()).all()


@pytest.mark.parametrize("dtype,size", [(BF, 3.38e38), (BF, 2.0 ** -126), (HF, 65504.0), (HF, 2.0 ** -24)])
@pytest.mark.parametrize("lens,width", [([1, 900], 64), ([1, 9000], 1024)])
def test_decode_values_at_the_limits(sage, oracle_mod, dtype, size, lens, width):
    """Values at the type's largest and smallest magnitudes, of both signs per channel: an average of equal
    values neither overflows nor vanishes."""
    c = Case(sage, lens, 16, 2, 64, dtype, width=width).fill(oracle_mod, 65)
    row = torch.where(torch.arange(64) % 3 == 0, -size, size).to(dtype).cuda()
    page, slot, _ = c.places(c.lens)
    put(c.v, page, slot, "HND", row)
    c.kv64 = [(k, row.double().expand(v.shape)) for k, v in c.kv64]
    q = randn(gen(66), 2, 6, 64, dtype=dtype) * 0.05  # weights of like size: sums over many keys
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    assert torch.equal(out[0], row.expand(6, 64))
    check_decode(c, q, out)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("D,group,width", [(64, 4, None), (64, 12, 4096), (128, 4, 4096), (128, 12, None),
                                           (64, 7, 4096), (128, 8, None), (128, 1, None)])
def test_decode_weights_on_fp4_are_as_exact_as_on_16_bits(sage, dtype, D, group, width):
    """Two kinds of keys, all of a kind alike, whose values nearly cancel: a rounding of the weights to 11 bits would
    be the same for each of them and stand out in the sum (up to 1e-3 where 1.3e-4 and the output's rounding are
    allowed). The bound is decode64's with what a second operand leaves of the weights' rounding."""
    B, n, first = 6, 128, 53
    c = Case(sage, [n] * B, 16, 1, D, dtype, "fp4", width=width)
    g = gen(77)
    kind = torch.stack([torch.randperm(n, generator=g, device="cuda") < first for _ in range(B)]).view(-1)
    k = torch.zeros(B * n, 1, D, dtype=dtype, device="cuda")
    k[~kind, 0, 0] = -6.0                       # codes and scales are exact
    v = torch.where(kind, 6.0, -6.0).to(dtype)[:, None, None].expand(-1, 1, D).contiguous()
    sage.cache_append(c.cache, k, v, c.table, c.seq_lens, cu_seqlens=c.cu(c.lens))
    kk, vv = sage.cache_gather(c.cache, c.table, c.seq_lens, cu_seqlens=c.cu(c.lens), total=B * n)
    assert torch.equal(kk, k) and torch.equal(vv, v)
    q = torch.zeros(B, group, D, device="cuda")
    q[..., 0] = 5.78 + 0.3 * (2 * torch.rand(B, group, generator=g, device="cuda") - 1)
    q = q.to(dtype)
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, sm_scale=0.01)
    for b in range(B):
        want, amag, slack = decode64(q[b], k.double().view(B, n, 1, D)[b], v.double().view(B, n, 1, D)[b], 0.01)
        tol = U[dtype] * want.abs() + (2 * U[HF] ** 2 * amag + slack) * (1 + U[dtype]) + TINY[dtype]
        err = (out[b].double() - want).abs()
        assert (err <= tol).all(), (b, float(err.max()), float((err / tol).max()))

@pytest.mark.parametrize("fmt,dtype,size", [("16bit", BF, 2e3), ("16bit", BF, 3e4), ("16bit", HF, 6e3), ("fp4", BF, 3e4),
                                            ("fp4", HF, 6e3)])
@pytest.mark.parametrize("lens,width", [([100, 3], 16), ([2000, 700], 128), ([5000, 900], 4096)])
def test_decode_scores_beyond_the_steps_of_32_bits(sage, oracle_mod, fmt, dtype, size, lens, width):
    """Scores of 10^7 to 10^10, where a step of binary32 is many powers of e: the best key takes all (in the first
    sequence it shares with its double in the second half). The next one is further below than decode64's bound on
    the sums, and by more than 100 (heads where it is not are left out), so its weight is nothing."""
    c = Case(sage, lens, 16, 2, 128, dtype, fmt, width=width).fill(oracle_mod, 45, scale=size / 4)
    page, slot, _ = c.places(lens)
    half = lens[0] // 2
    for x in (c.k, c.ks) if fmt == "fp4" else (c.k,):
        put(x, page[half:2 * half], slot[half:2 * half], "HND", x[page[:half], :, slot[:half]])
    c.kv64[0][0][half:2 * half] = c.kv64[0][0][:half]
    q = randn(gen(46), 2, 6, 128, dtype=dtype) * size
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, sm_scale=1.0)
    assert torch.isfinite(out).all()
    seen = 0
    for b, n in enumerate(lens):
        k, v = c.kv64[b]
        many = 2 if b == 0 else 1
        for h in range(6):
            s = k[:, h // 3] @ q[b, h].double()
            top, at = s.topk(many + 1)
            bound = float((k[:, h // 3].abs() @ q[b, h].double().abs()).max()) * 136 * 2.0 ** -23
            if top[many - 1] - top[many] <= bound + 100 or (many == 2 and top[0] != top[1]):
                continue
            seen += 1
            mean = v[at[:many], h // 3].mean(0)
            assert ((out[b, h].double() - mean).abs() <= U[dtype] * mean.abs() + TINY[dtype]).all(), (b, h)
    assert seen >= 6

@pytest.mark.parametrize("B,pages,first", [(1, 1024, False), (512, 1024, False), (512, 64, True)])
def test_decode_sums_over_many_large_values(sage, B, pages, first):
    """Values at bf16's limit, more of them than a sum of weights near one could hold: many parts of one sequence (1),
    2^16 keys of one weight in each warp's sum (2), and 2^12 of them with 15 times the first keys' weight, which is
    not yet enough to raise the running maximum (3). An average of equal values is that value; its binary32 sum
    over n keys is off by at most n 2^-24 of it."""
    D, P, n = 64, 256, 256 * pages
    c = Case(sage, [2 * P], P, 1, D, BF)  # two pages, of which every sequence has many copies
    row = torch.where(torch.arange(D) % 3 == 0, -3.38e38, 3.38e38).to(BF).cuda()
    k = torch.zeros(2 * P, 1, D, dtype=BF, device="cuda")
    k[P:, 0, 0] = 1.0
    sage.cache_append(c.cache, k, row.expand(2 * P, 1, D).contiguous(), c.table, c.seq_lens, cu_seqlens=c.cu([2 * P]))
    table = c.table[0, 1].expand(B, pages).contiguous()
    table[:, 0] = c.table[0, 0]
    q = torch.zeros(B, 1, D, dtype=BF, device="cuda")
    if first:
        q[..., 0] = 2.703125  # ln 2^3.9: exact in 8 bits
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    out = sage.sageattn_decode(q, c.cache, table, lens, sm_scale=1.0)
    want = row.double()
    assert torch.isfinite(out).all()
    assert ((out.double() - want).abs() <= (U[BF] + n * 2.0 ** -24) * want.abs()).all()

def test_decode_large_queries_on_fp4(sage, oracle_mod):
    """bf16 queries beyond fp16's range, and rows of very different size, are rescaled exactly."""
    c = Case(sage, [100], 16, 1, 128, BF, "fp4").fill(oracle_mod, 61)
    q = randn(gen(62), 1, 3, 128) * torch.tensor([1e6, 1e-6, 1.0], device="cuda")[None, :, None].to(BF)
    sm = 1e-6
    check_decode(c, q, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, sm_scale=sm), sm=sm)
    tiny = torch.full((1, 3, 128), 2.0 ** -133, dtype=BF, device="cuda")
    check_decode(c, tiny, sage.sageattn_decode(tiny, c.cache, c.table, c.seq_lens))


def test_decode_nan_in_cached_token_reaches_only_its_sequence(sage, oracle_mod):
    c = Case(sage, [70, 70], 16, 1, 64, BF).fill(oracle_mod, 71)
    page, slot, _ = c.places(c.lens)
    c.v[page[30], :, slot[30]] = float("nan")
    q = randn(gen(72), 2, 2, 64)
    out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("lens,width", [([9000, 70], 1024), ([900, 70], 64), ([40, 3], 4)])
def test_decode_nan_queries_and_keys(sage, oracle_mod, fmt, lens, width):
    """A query that is not a number gives outputs that are not, however its sequence is split; the others are untouched.
    A key that is not (16-bit) takes its heads with it."""
    c = Case(sage, lens, 16, 2, 64, BF, fmt, width=width).fill(oracle_mod, 75)
    q = randn(gen(76), 2, 6, 64)
    want = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    check_decode(c, q, want)
    bad = q.clone()
    bad[0, 4, 9] = float("nan")
    out = sage.sageattn_decode(bad, c.cache, c.table, c.seq_lens)
    assert torch.isnan(out[0, 4]).all()
    out[0, 4] = want[0, 4]
    assert torch.equal(out, want)
    if fmt == "16bit":
        page, slot, _ = c.places(c.lens)
        c.k[page[lens[0] - 2], 1, slot[lens[0] - 2], 5] = float("nan")
        out = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
        assert torch.isnan(out[0, 3:]).all() and torch.equal(out[0, :3], want[0, :3]) and torch.equal(out[1], want[1])


def test_decode_strided_queries_outputs_and_tables(sage, oracle_mod):
    c = Case(sage, [70, 130, 5], 16, 2, 128, BF).fill(oracle_mod, 81)
    big = randn(gen(82), 3, 12, 128)
    q = big[:, 2:10]
    out = torch.full((3, 12, 128), 7.0, dtype=BF, device="cuda")
    table = torch.full((3, 40), -1, dtype=torch.int32, device="cuda")
    table[:, 8:8 + c.table.shape[1]] = c.table
    ws = torch.empty(sage.decode_workspace_bytes(c.cache, table[:, 8:20], c.seq_lens, 8), dtype=torch.uint8, device="cuda")
    got = sage.sageattn_decode(q, c.cache, table[:, 8:20], c.seq_lens, out=out[:, 2:10], workspace=ws.fill_(0xFF))
    check_decode(c, q, got)
    assert (out[:, :2] == 7.0).all() and (out[:, 10:] == 7.0).all()
    assert torch.equal(got, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens))


def test_decode_in_place(sage, oracle_mod):
    for lens, width in (([3000, 5, 700], None), ([90, 64], None), ([9000], 1024)):
        c = Case(sage, lens, 16, 2, 128, BF, "fp4", width=width).fill(oracle_mod, 85)
        q = randn(gen(86), len(lens), 40, 128)  # 20 heads a group: two chunks
        want = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
        assert sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, out=q) is q
        assert torch.equal(q, want)


def test_decode_in_place_needs_the_same_strides(sage, oracle_mod):
    c = Case(sage, [90, 64, 3, 1], 16, 2, 128).fill(oracle_mod, 87)
    q = randn(gen(88), 4, 4, 128)
    kept = q.clone()
    with pytest.raises(sage.SageError) as e:
        sage.sageattn_decode(q, c.cache, c.table, c.seq_lens, out=q.transpose(0, 1))
    assert e.value.status == sage.SAGE_ERR_INVALID_ARG and torch.equal(q, kept)
    # strides of a dimension of one do not count
    want = sage.sageattn_decode(q[:1], c.cache, c.table[:1], c.seq_lens[:1])
    out = q.as_strided((1, 4, 128), (8, 128, 1))
    sage.sageattn_decode(q[:1], c.cache, c.table[:1], c.seq_lens[:1], out=out)
    assert torch.equal(q[:1], want) and torch.equal(q[1:], kept[1:])


def test_many_sequences(sage, oracle_mod):
    """More sequences than threads of a block, most of them short or empty; steps for all of them at once."""
    B = 5000
    g = torch.Generator().manual_seed(7)
    lens = torch.where(torch.rand(B, generator=g) < 0.3, 0, torch.randint(0, 40, (B,), generator=g)).tolist()
    lens = [n + 1 for n in lens]
    c = Case(sage, lens, 8, 1, 64, HF).fill(oracle_mod, 95)
    w = torch.randn(64, generator=gen(96), device="cuda")
    k, v, q = (randn(gen(97 + i), B, 1 + i, 64, dtype=HF) for i in range(3))
    v, q = v[:, :1], q[:, :2]
    qr = sage.cache_append(c.cache, k, v, c.table, c.seq_lens, q=q, q_weight=w, k_weight=w, rope=sage.rope_table(64, 64))
    pos = c.places([1] * B)[2]
    want, slack = rows64(q, w, sage.rope_table(64, 64), pos, False)
    assert_rounded(qr, want, slack, HF)
    kk, vv = sage.cache_gather(c.cache, c.table, c.seq_lens, cu_seqlens=c.cu(lens), total=sum(lens))
    c.kv64 = list(zip(kk.double().split(lens), vv.double().split(lens)))
    check_decode(c, qr, sage.sageattn_decode(qr, c.cache, c.table, c.seq_lens))


FIRST = """
import torch, microscaling_fp4_quantized_b200 as sage
BF = torch.bfloat16
cache = sage.PagedKVCache.empty(200, 16, 2, 128, dtype=BF, format=%r)
table = torch.arange(200, dtype=torch.int32, device='cuda').view(2, 100)
lens = torch.tensor([1600, 900], dtype=torch.int32, device='cuda')
cu = torch.tensor([0, 1600, 2500], dtype=torch.int32, device='cuda')
g = torch.Generator('cuda').manual_seed(1)
k, v = (torch.randn(2500, 2, 128, generator=g, device='cuda').to(BF) for _ in range(2))
q = torch.randn(2500, 8, 128, generator=g, device='cuda').to(BF)
rope = sage.rope_table(1600, 128)
pos = torch.cat((torch.arange(1600), torch.arange(900))).int().cuda()

def step():
    sage.cache_append(cache, k, v, table, lens, cu_seqlens=cu, rope=rope)
    qr, kr = sage.qk_norm_rope(q, k, rope=rope, positions=pos)
    dense = sage.cache_gather(cache, table, lens, cu_seqlens=cu, total=2500)
    short = sage.sageattn_decode(qr[:2], cache, table[:, :4], lens.clamp(max=64))
    return qr, kr, *dense, short, sage.sageattn_decode(qr[:2], cache, table, lens)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and sage.device_error() == 0
print('same')
"""


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_first_call_of_a_process_is_captured(sage, fmt):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % fmt], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_shared_prefix_pages(sage, oracle_mod):
    """Two sequences whose tables name the same pages."""
    c = Case(sage, [48, 48], 16, 2, 64, BF).fill(oracle_mod, 91)
    c.table[1] = c.table[0]
    c.kv64[1] = c.kv64[0]
    q = randn(gen(92), 2, 4, 64)
    check_decode(c, q, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens))


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_offsets_beyond_32_bits(sage, oracle_mod, fmt):
    """A pool of more than 2^32 elements (and code bytes), of which the last pages are used."""
    H, P, D = 8, 64, 128
    pages = 2 ** 33 // (H * P * D) + 9 if fmt == "fp4" else 2 ** 32 // (H * P * D) + 9
    lens, dt = [130, 64], BF
    c = Case(sage, lens, P, H, D, dt, fmt, spare=4)
    small = c.table.clone()
    c.cache = sage.PagedKVCache.empty(pages, P, H, D, dtype=dt, format=fmt)
    used = small.cpu() < 2 ** 30
    c.table = torch.where(used, pages - 1 - small.cpu(), small.cpu()).cuda()
    g = gen(101)
    k, v = randn(g, 194, H, D), randn(g, 194, H, D)
    sage.cache_append(c.cache, k, v, c.table, c.seq_lens, cu_seqlens=c.cu(lens))
    ko, vo = sage.cache_gather(c.cache, c.table, c.seq_lens, cu_seqlens=c.cu(lens), total=194)
    if fmt == "16bit":
        assert torch.equal(ko, k) and torch.equal(vo, v)
    c.kv64 = list(zip(*(x.double().split(lens) for x in (ko, vo))))
    q = randn(g, 2, 16, D)
    check_decode(c, q, sage.sageattn_decode(q, c.cache, c.table, c.seq_lens))


# -------------------------------------------------------------------- streams, graphs, together --

def test_other_stream_and_two_workspaces_at_once(sage, oracle_mod):
    c = Case(sage, [3000, 129], 16, 2, 128, BF).fill(oracle_mod, 111)
    q = randn(gen(112), 2, 8, 128)
    want = sage.sageattn_decode(q, c.cache, c.table, c.seq_lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs.append([sage.sageattn_decode(q, c.cache, c.table, c.seq_lens) for _ in range(20)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for group in outs for o in group)


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_captured_steps(sage, oracle_mod, fmt):
    """Append and attention captured once, replayed over growing sequences; two graphs side by side."""
    B, H, Hq, D, P, steps = 3, 2, 8, 128, 16, 40
    start = [0, 30, 60]
    c = Case(sage, [n + steps for n in start], P, H, D, BF, fmt)
    rope = sage.rope_table(200, D)
    g = gen(121)
    w = randn(g, D)
    xs = randn(g, steps, B, Hq + 2 * H, D)
    old = randn(g, 90, 2, H, D)
    first = torch.tensor(start, dtype=torch.int32).cuda()

    def reset():
        sage.cache_append(c.cache, old[:, 0], old[:, 1], c.table, first, cu_seqlens=c.cu(start))

    def step(x, lens):
        q = sage.cache_append(c.cache, x[:, Hq:Hq + H], x[:, Hq + H:], c.table, lens, q=x[:, :Hq], q_weight=w, k_weight=w,
                              rope=rope)
        return sage.sageattn_decode(q, c.cache, c.table, lens)

    reset()
    lens = first.clone()
    want = []
    for i in range(steps):
        lens += 1
        want.append(step(xs[i], lens).clone())
    reset()
    lens = first.clone()
    x = xs[0].clone()
    graphs = []
    for _ in range(2):  # both captured with private workspaces; the second one's pool is its own
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step(x, lens)
        graphs.append((gr, out))
    for i in range(steps):
        x.copy_(xs[i])
        lens += 1
        gr, out = graphs[i % 2]
        gr.replay()
        assert torch.equal(out, want[i]), i


@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_prompt_continued_prompt_and_tokens(sage, oracle_mod, fmt):
    """The operators as they are used: prompts, a second part of the prompts over the cached first, then
    tokens one by one; every attention held to binary64 attention over what the cache holds."""
    H, Hq, D, P = 2, 8, 128, 16
    one, two = [150, 33, 1], [40, 129, 70]
    total = [a + b + 3 for a, b in zip(one, two)]
    c = Case(sage, total, P, H, D, BF, fmt)
    rope, g = sage.rope_table(400, D), gen(131)
    w = randn(g, D)
    opts = dict(q_weight=w, k_weight=w, rope=rope)

    def lens_of(*parts):
        return torch.tensor([sum(t) for t in zip(*parts)], dtype=torch.int32).cuda()

    def rows(n, heads):
        return randn(g, n, heads, D)

    q, k, v = rows(184, Hq), rows(184, H), rows(184, H)
    out = sage.sageattn_prefill(q, k, v, c.cache, c.table, lens_of(one), c.cu(one), max(one), **opts)
    qr, kr = sage.qk_norm_rope(q, k, positions=torch.cat([torch.arange(n) for n in one]).int().cuda(), **opts)
    dense = sage.cache_gather(c.cache, c.table, lens_of(one), cu_seqlens=c.cu(one), total=184)
    if fmt == "16bit":
        assert torch.equal(dense[0], kr) and torch.equal(dense[1], v)
    assert torch.equal(out, sage.sageattn_varlen(qr, *dense, c.cu(one), c.cu(one), max(one), max(one), is_causal=True))
    q, k, v = rows(239, Hq), rows(239, H), rows(239, H)
    both = [a + b for a, b in zip(one, two)]
    out = sage.sageattn_prefill(q, k, v, c.cache, c.table, lens_of(both), c.cu(two), max(two), cu_seqlens_kv=c.cu(both),
                                max_seqlen_kv=max(both), total_kv=sum(both), smooth_q=True, **opts)
    assert out.shape == (239, Hq, D) and torch.isfinite(out).all()
    lens = lens_of(both)
    for _ in range(3):
        lens += 1
        q = sage.cache_append(c.cache, rows(3, H), rows(3, H), c.table, lens, q=rows(3, Hq), **opts)
        got = sage.sageattn_decode(q, c.cache, c.table, lens)
        n = lens.tolist()
        kk, vv = sage.cache_gather(c.cache, c.table, lens, cu_seqlens=c.cu(n), total=sum(n))
        c.lens, c.kv64 = n, list(zip(kk.double().split(n), vv.double().split(n)))
        check_decode(c, q, got)



@pytest.mark.parametrize("precision", ["fp4", "8bit"])
@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
@pytest.mark.parametrize("one,two", [([0, 0, 0], [150, 33, 1]), ([150, 33, 1], [40, 129, 70]),
                                     ([128, 0, 16, 300], [1, 128, 5, 15])])
def test_every_prompt_token_attends_up_to_itself(sage, oracle_mod, fmt, precision, one, two):
    """The second part of each prompt over the cached first one. Keys are random signs, and the query of a token is its
    own key and, a little stronger, the next one: after the rotation to their true positions the own key leads all earlier
    ones by far (scores 181 against 24 z, z normal), and only the causal mask keeps the next one out. So a token's
    output is its own value, and any other offset, position, length or prefix shows. The values are signs too: FP4 holds them as 6 E4M3(1/6) = 1.03125, the 8-bit
    path to 2^-4, the FP4 cache to 2^-5 first; weights sum to one within 2^-4 (E4M3) and the others' stay
    below 0.01: 0.2 in all, where another value is off by 2."""
    H, Hq, D, P = 2, 8, 128, 16
    n = [a + b for a, b in zip(one, two)]
    c = Case(sage, n, P, H, D, BF, fmt)
    g = gen(161)
    rope = sage.rope_table(max(n), D)
    sign = lambda *s: torch.randint(0, 2, s, generator=g, device="cuda").float() * 2 - 1  # noqa: E731
    keys, values = [sign(m, H, D) for m in n], [sign(m, H, D) for m in n]
    queries = []
    for k in keys:
        nxt = torch.cat((k[1:], torch.zeros_like(k[:1])))
        queries.append((16 * (k + 1.1 * nxt)).repeat_interleave(Hq // H, dim=1))
    part = lambda xs, lo, hi: torch.cat([x[a:b] for x, a, b in zip(xs, lo, hi)]).to(BF)  # noqa: E731
    zero = [0] * len(n)
    if sum(one):
        sage.cache_append(c.cache, part(keys, zero, one), part(values, zero, one), c.table,
                          torch.tensor(one, dtype=torch.int32).cuda(), cu_seqlens=c.cu(one), rope=rope)
    q, k, v = part(queries, one, n), part(keys, one, n), part(values, one, n)
    kv = {} if not sum(one) else dict(cu_seqlens_kv=c.cu(n), max_seqlen_kv=max(n), total_kv=sum(n))
    out = sage.sageattn_prefill(q, k, v, c.cache, c.table, c.seq_lens, c.cu(two), max(two), rope=rope, precision=precision,
                                **kv)
    assert (out.float() - v.float().repeat_interleave(Hq // H, dim=1)).abs().max() <= 0.2
    # the same, from inputs put together here: rows read from the pages, queries turned to their positions
    pos = torch.cat([torch.arange(a, b) for a, b in zip(one, n)]).int().cuda()
    qr, _ = sage.qk_norm_rope(q, rope=rope, positions=pos)
    if fmt == "16bit":
        dense = [c.at(x, n).contiguous() for x in (c.k, c.v)]
    else:
        dense = [torch.from_numpy(decoded(oracle_mod, c.at(x, n).cpu().numpy(), c.at(s, n).cpu().numpy())).to(BF).cuda()
                 for x, s in ((c.k, c.ks), (c.v, c.vs))]
    assert torch.equal(out, sage.sageattn_varlen(qr, *dense, c.cu(two), c.cu(n), max(two), max(n), is_causal=True,
                                                 precision=precision))

@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_padded_prompts(sage, fmt):
    """Rows behind the last prompt, whatever they hold, change nothing in the cache; attention over packed
    rows wants them cut off, and says so."""
    lens, H, Hq, D = [70, 1, 33], 2, 4, 64
    n, rope, g = sum(lens), sage.rope_table(128, 64), gen(141)
    q, k, v = randn(g, n, Hq, D), randn(g, n, H, D), randn(g, n, H, D)
    held = []
    for pad in (0, 25):
        c = Case(sage, lens, 16, H, D, BF, fmt)
        qp, kp, vp = (torch.cat((t, torch.full((pad,) + t.shape[1:], float("nan"), dtype=BF, device="cuda")))
                      for t in (q, k, v))
        out = sage.sageattn_prefill(qp, kp, vp, c.cache, c.table, c.seq_lens, c.cu(lens), max(lens), rope=rope)
        assert out.shape == qp.shape and sage.device_error() == (sage.DEV_ERR_SEQLENS if pad else 0)
        held.append((c.k.view(torch.uint8).clone(), c.v.view(torch.uint8).clone()))
    assert all(torch.equal(a, b) for a, b in zip(*held))


def test_two_threads_at_once(sage, oracle_mod):
    """Calls from two Python threads, each on its own stream."""
    c = Case(sage, [2000, 31, 500], 16, 8, 128).fill(oracle_mod, 151)
    q = [randn(gen(152 + i), 3, 32, 128) for i in range(2)]
    want = [sage.sageattn_decode(x, c.cache, c.table, c.seq_lens) for x in q]
    torch.cuda.synchronize()
    same = [0, 0]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                same[i] += int(torch.equal(sage.sageattn_decode(q[i], c.cache, c.table, c.seq_lens), want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [50, 50]


def test_refusals_on_the_gpu(sage):
    cache = sage.PagedKVCache.empty(8, 16, 2, 128)
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    q, k = torch.zeros(2, 4, 128, dtype=BF, device="cuda"), torch.zeros(2, 2, 128, dtype=BF, device="cuda")
    bad = [
        lambda: sage.sageattn_decode(q.half(), cache, table, lens),
        lambda: sage.sageattn_decode(q[:, :3], cache, table, lens),
        lambda: sage.sageattn_decode(q[:1], cache, table, lens),
        lambda: sage.sageattn_decode(q.cpu(), cache, table, lens),
        lambda: sage.sageattn_decode(q, cache, table.long(), lens),
        lambda: sage.sageattn_decode(q, cache, table.t(), lens),
        lambda: sage.sageattn_decode(q, cache, table, lens.float()),
        lambda: sage.sageattn_decode(q, cache, table, lens[:1]),
        lambda: sage.sageattn_decode(q, cache, table, lens, out=q[:, :2]),
        lambda: sage.sageattn_decode(q, cache, table, lens, workspace=torch.empty(8, device="cuda")),
        lambda: sage.cache_append(cache, k, k[:, :1], table, lens),
        lambda: sage.cache_append(cache, k[:1], k[:1], table, lens),
        lambda: sage.cache_append(cache, k, k, table, lens, q=q[:1]),
        lambda: sage.cache_append(cache, k, k, table, lens, q_weight=k[0, 0]),
        lambda: sage.cache_append(cache, k, k, table, lens, k_weight=k[0, 0, :64]),
        lambda: sage.cache_append(cache, k, k, table, lens, k_weight=k[0, 0].half()),
        lambda: sage.cache_append(cache, k, k, table, lens, rope=torch.zeros(4, 128, dtype=BF, device="cuda")),
        lambda: sage.cache_append(cache, k, k, table, lens, cu_seqlens=lens),
        lambda: sage.cache_gather(cache, table, lens, cu_seqlens=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: sage.cache_gather(cache, table, lens, k_out=k),
        lambda: sage.cache_gather(cache, table, lens, total=3),
        lambda: sage.qk_norm_rope(q, rope=torch.zeros(4, 128, device="cuda")),
        lambda: sage.qk_norm_rope(q, k[:1]),
        lambda: sage.qk_norm_rope(q, q_out=q[:, :2]),
        lambda: sage.qk_norm_rope(q, k_weight=q[0, 0]),
        lambda: sage.PagedKVCache(cache.k, cache.v[:4]),
        lambda: sage.PagedKVCache(cache.k, cache.v, dtype=HF),
        lambda: sage.PagedKVCache(cache.k.transpose(2, 3), cache.v.transpose(2, 3)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(sage.SageError) as e:
        sage.sageattn_decode(q, cache, table, lens, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == sage.SAGE_ERR_INVALID_ARG
    with pytest.raises(sage.SageError):
        sage.sageattn_decode(q, cache, table, lens, sm_scale=float("nan"))
    with pytest.raises(sage.SageError):
        sage.cache_append(cache, k, k, table, lens, rope=torch.zeros(4, 48, device="cuda"))
    with pytest.raises(sage.SageError):
        sage.cache_append(cache, k.transpose(0, 1).contiguous().view(-1)[4:4 + 2 * 128].view(1, 2, 128), k[:1], table[:1], lens[:1])
    with pytest.raises(sage.SageError) as e:
        c96 = sage.PagedKVCache.empty(2, 16, 2, 96)  # building it is fine; using it is refused
        z = torch.zeros(2, 2, 96, dtype=BF, device="cuda")
        sage.cache_append(c96, z, z, table, lens)
    assert e.value.status == sage.SAGE_ERR_UNSUPPORTED


@pytest.mark.parametrize("layout", ["HND", "NHD"])
@pytest.mark.parametrize("fmt", ["16bit", "fp4"])
def test_caches_without_heads_or_slots_are_refused(sage, fmt, layout):
    for pages, slots, heads in ((4, 16, 0), (4, 0, 2), (0, 16, 0)):
        with pytest.raises(ValueError):
            sage.PagedKVCache.empty(pages, slots, heads, 128, format=fmt, tensor_layout=layout)
    sage.PagedKVCache.empty(0, 16, 2, 128, format=fmt, tensor_layout=layout)  # no pages yet: a cache like any other


def test_empty_calls(sage):
    cache = sage.PagedKVCache.empty(4, 16, 2, 64)
    table, lens = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    z = torch.zeros(0, 4, 64, dtype=BF, device="cuda")
    assert sage.sageattn_decode(z, cache, table, lens).shape == (0, 4, 64)
    assert sage.cache_append(cache, z[:, :2], z[:, :2], table, lens, q=z).shape == (0, 4, 64)
    assert sage.cache_gather(cache, table, lens)[0].shape == (0, 2, 64)
    assert sage.qk_norm_rope(z)[0].shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, dtype=BF, device="cuda")
    out = sage.sageattn_decode(q, cache, torch.zeros(2, 0, dtype=torch.int32, device="cuda"),
                               torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert not out.any()
