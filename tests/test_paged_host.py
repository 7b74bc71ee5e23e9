"""Paged cache, host side (no GPU): what the C entry points refuse before any launch, workspace
sizes, empty problems, and the arithmetic of the page division."""
import ctypes

import pytest

FAKE = 0x10000  # a 16- and 256-byte aligned address that is never followed


@pytest.fixture(scope="module")
def sage():
    from microscaling_fp4_quantized_b200 import build
    build.build()
    import microscaling_fp4_quantized_b200 as s
    s.lib()
    return s


def s3(*v):
    return (ctypes.c_int64 * 3)(*v)


def s2(*v):
    return (ctypes.c_int64 * 2)(*v)


def make_cache(sage, **kw):
    d = dict(k=FAKE, v=FAKE, k_sf=None, v_sf=None, num_pages=10, page_size=16, Hkv=2, D=128, dtype=0, format=0)
    d.update(kw)
    D, P, H = d["D"], d["page_size"], d["Hkv"]
    d.setdefault("k_stride", s3(H * P * D, P * D, D))
    d.setdefault("v_stride", s3(H * P * D, P * D, D))
    return sage.paged._Cache(**d)


def make_batch(sage, **kw):
    d = dict(B=3, page_table=FAKE, table_stride=4, table_width=4, seq_lens=FAKE, cu_seqlens=None)
    d.update(kw)
    return sage.paged._Batch(**d)


def decode(sage, cache=None, batch=None, q=FAKE, qs=None, out=FAKE, os=None, Hq=8, scale=0.0, ws=FAKE, ws_bytes=1 << 40):
    c, b = cache or make_cache(sage), batch or make_batch(sage)
    return sage.lib().sage_fp4_attn_decode(c, b, q, qs or s2(Hq * c.D, c.D), out, os or s2(Hq * c.D, c.D), Hq, scale, ws,
                                           ws_bytes, None)


INV, UNS = 1, 2


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), UNS), (dict(dtype=2), INV), (dict(format=2), INV), (dict(num_pages=-1), INV), (dict(page_size=0), INV),
    (dict(page_size=65537), UNS), (dict(Hkv=0), INV), (dict(k=FAKE + 8), INV), (dict(v=None), INV),
    (dict(format=1), INV),                                           # no scales
    (dict(format=1, k_sf=FAKE, v_sf=FAKE + 4), INV),                 # scales not 8-byte aligned
    (dict(k_stride=s3(4096, 2048, 100)), INV),                       # slot stride not 16-byte granular
    (dict(k_stride=s3(4096, 2048, -128)), INV),
    (dict(v_stride=s3(4096, 2048, 64)), INV),                        # rows would overlap
    (dict(v_stride=s3(4096, 0, 128)), INV),
    (dict(format=1, k_sf=FAKE, v_sf=FAKE, k_stride=s3(4096, 2048, 136)), INV),  # FP4: multiples of D
    (dict(num_pages=2 ** 25), UNS),                                  # 2^37 elements: beyond 2^32 units of 16 bytes
])
def test_cache_refusals(sage, kw, status):
    c = make_cache(sage, **kw)
    b = make_batch(sage)
    L = sage.lib()
    assert decode(sage, cache=c) == status
    assert L.sage_fp4_decode_workspace_bytes(c, b, 8) == 0
    st = s2(c.D or 1, 2 * c.D)
    assert L.sage_fp4_cache_append(c, b, FAKE, st, FAKE, st, 3, None, None, None) == status
    assert L.sage_fp4_cache_gather(c, b, FAKE, st, FAKE, st, 3, None) == status


def test_largest_cache_is_accepted(sage):
    # the last row just inside 2^32 - 1 units of 8 elements
    pages = (2 ** 35 - 8) // 4096
    assert sage.lib().sage_fp4_decode_workspace_bytes(make_cache(sage, num_pages=pages), make_batch(sage), 8) > 0


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INV), (dict(table_width=-1), INV), (dict(table_stride=-4), INV), (dict(page_table=None), INV),
    (dict(page_table=FAKE + 2), INV), (dict(seq_lens=None), INV), (dict(table_width=2 ** 26 + 1), UNS),
])
def test_batch_refusals(sage, kw, status):
    b = make_batch(sage, **kw)
    assert decode(sage, batch=b) == status
    st = s2(128, 256)
    assert sage.lib().sage_fp4_cache_append(make_cache(sage), b, FAKE, st, FAKE, st, 3, None, None, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(Hq=7), INV), (dict(Hq=-2), INV), (dict(q=None), INV), (dict(q=FAKE + 2), INV), (dict(out=FAKE + 8), INV),
    (dict(qs=s2(1024, 100)), INV), (dict(os=s2(1024, 0)), INV), (dict(os=s2(64, 128)), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV), (dict(ws=FAKE + 16), INV), (dict(ws=None), INV),
    (dict(ws_bytes=1000), INV),
])
def test_decode_refusals(sage, kw, status):
    assert decode(sage, **kw) == status


@pytest.mark.parametrize("kw", [dict(Hkv=0), dict(Hkv=-2), dict(page_size=0)])
def test_a_cache_without_heads_or_slots_gets_no_handle(sage, kw):
    """The calls divide by both; a handle is made for caches that have them."""
    with pytest.raises(ValueError):
        sage.paged._n().make_cache(ctypes.addressof(make_cache(sage, **kw)), 0)
    sage.paged._n().make_cache(ctypes.addressof(make_cache(sage)), 0)


def test_decode_in_place_with_other_strides_is_refused(sage):
    """Output rows would lie on query rows that other blocks have yet to read."""
    for qs, os in (((1024, 128), (128, 384)), ((1024, 128), (2048, 128)), ((1024, 128), (1024, 256)), ((0, 128), (1024, 128))):
        assert decode(sage, qs=s2(*qs), os=s2(*os)) == INV, (qs, os)


def test_append_and_gather_refusals(sage):
    L, c, b, st = sage.lib(), make_cache(sage), make_batch(sage), s2(128, 256)

    def append(k=FAKE, ks=st, v=FAKE, vs=st, total=3, rope=None, q=None, batch=b):
        return L.sage_fp4_cache_append(c, batch, k, ks, v, vs, total, rope, q, None)

    assert append(k=None) == INV and append(v=FAKE + 4) == INV and append(ks=s2(128, 100)) == INV and append(ks=None) == INV
    assert append(total=-1) == INV
    assert append(total=4) == INV                       # one token per sequence without offsets
    assert append(total=4, batch=make_batch(sage, cu_seqlens=FAKE + 1)) == INV
    R, Q = sage.paged._Rope, sage.paged._Rows
    for bad, status in ((dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(q_weight=FAKE + 4), INV),
                        (dict(rope=FAKE + 8, rope_len=4, rotary_dim=64), INV), (dict(rope=FAKE, rope_len=-1, rotary_dim=64), INV),
                        (dict(rope=FAKE, rope_len=4, rotary_dim=48), UNS), (dict(rope=FAKE, rope_len=4, rotary_dim=160), UNS),
                        (dict(rope=FAKE, rope_len=4, rotary_dim=0), UNS)):
        assert append(rope=R(**bad)) == status, bad
        rows = Q(FAKE, FAKE, 2, s3(0, 128, 256), s3(0, 128, 256))
        assert L.sage_fp4_norm_rope(rows, None, 1, 3, 128, 0, R(**bad), None, None) == status, bad
    assert append(q=Q(FAKE, None, 2, s3(0, 128, 256), s3(0, 128, 256))) == INV
    assert append(q=Q(FAKE, FAKE, 2, s3(0, 128, 256), s3(0, 256, 128))) == INV  # in place, other strides
    assert append(q=Q(FAKE, FAKE + 4096, 2, s3(0, 128, 256), s3(0, 128, 0))) == INV  # outputs overlap
    assert append(q=Q(FAKE, FAKE, -1)) == INV

    def gather(k=FAKE, ks=st, v=FAKE, vs=st, total=3):
        return L.sage_fp4_cache_gather(c, b, k, ks, v, vs, total, None)

    assert gather(k=None) == INV and gather(vs=s2(128, 0)) == INV and gather(ks=s2(64, 256)) == INV and gather(total=2) == INV


def test_norm_rope_refusals(sage):
    L, Q = sage.lib(), sage.paged._Rows
    ok = Q(FAKE, FAKE, 2, s3(768, 384, 128), s3(768, 384, 128))
    call = lambda q=ok, k=None, B=2, N=3, D=128, dtype=0, pos=None: L.sage_fp4_norm_rope(q, k, B, N, D, dtype, None, pos, None)  # noqa: E731
    assert call(D=80) == UNS and call(dtype=5) == INV and call(B=-1) == INV and call(B=2 ** 16, N=2 ** 15) == UNS
    assert call(pos=FAKE + 2) == INV
    assert call(k=Q(FAKE, FAKE + 8, 2, s3(768, 384, 128), s3(768, 384, 128))) == INV
    assert call(k=Q(FAKE, FAKE + 16, 2, s3(768, 384, 12), s3(768, 384, 128))) == INV


def test_empty_problems_launch_nothing(sage):
    L, c, st = sage.lib(), make_cache(sage), s2(128, 256)
    empty = make_batch(sage, B=0, page_table=None, seq_lens=None)
    assert decode(sage, batch=empty, q=None, out=None, ws=None, ws_bytes=0) == 0
    assert decode(sage, Hq=0, q=None, out=None, ws=None, ws_bytes=0) == 0
    assert L.sage_fp4_cache_append(c, empty, None, st, None, st, 0, None, None, None) == 0
    b = make_batch(sage, cu_seqlens=FAKE)
    assert L.sage_fp4_cache_append(c, b, None, st, None, st, 0, None, None, None) == 0
    assert L.sage_fp4_cache_gather(c, b, None, st, None, st, 0, None) == 0
    rows = sage.paged._Rows(heads=0)
    assert L.sage_fp4_norm_rope(rows, None, 2, 3, 128, 0, None, None, None) == 0
    assert L.sage_fp4_norm_rope(None, None, 0, 3, 128, 0, None, None, None) == 0


def test_decode_workspace(sage):
    L = sage.lib()
    size = lambda Hq=8, cache=None, **kw: L.sage_fp4_decode_workspace_bytes(cache or make_cache(sage), make_batch(sage, **kw), Hq)  # noqa: E731
    # 3 sequences x 2 heads of one 64-key tile, each pair counted as one tile more: at most 12 shares,
    # two partials of 8 heads each
    rows = 12 * 2 * 8
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert size() == up(12 * 16) + up(rows * 8) + rows * 128 * 4
    assert size(Hq=32) == up(12 * 16) + up(2 * rows * 8) + 2 * rows * 128 * 4  # 16 heads a group
    assert size(Hq=0) == 0 and size(B=0) == 0 and size(Hq=7) == 0
    # bounded by the number of shares the kernel ever uses
    assert size(B=4096, table_width=4096, table_stride=4096) == size(B=8192, table_width=8192, table_stride=8192)


def test_page_division_multiplier():
    """n // d = (n m) >> (31 + L), m = floor(2^(31+L) / d) + 1, at the ends of every quotient."""
    for d in list(range(1, 300)) + [4095, 4096, 4097, 65535, 65536]:
        L = (d - 1).bit_length()
        m = (1 << (31 + L)) // d + 1
        assert m < 1 << 32
        top = (2 ** 31 - 1) // d
        for k in {0, 1, 2, top // 2, top - 1, top}:
            for n in (k * d - 1, k * d, k * d + d - 1):
                if 0 <= n < 2 ** 31:
                    assert (n * m) >> (31 + L) == n // d, (n, d)


def test_python_refusals_without_a_gpu(sage):
    import torch
    t = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sage.PagedKVCache(t, t)                                       # not on a GPU
    with pytest.raises(ValueError):
        sage.PagedKVCache(t, t, tensor_layout="DHN")
    with pytest.raises(ValueError):
        sage.PagedKVCache(t.view(torch.uint8), t.view(torch.uint8))   # FP4 without scales
    with pytest.raises(ValueError):
        sage.PagedKVCache.empty(4, 16, 2, 128, format="int4", device="cpu")
    with pytest.raises(ValueError):
        sage.qk_norm_rope(t)
    with pytest.raises(ValueError):
        sage.rope_table(16, 48, device="cpu")
    tab = sage.rope_table(1000, 64, device="cpu")
    ang = 999.0 * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    assert torch.equal(tab[999], torch.cat((ang.cos(), ang.sin())).float())
