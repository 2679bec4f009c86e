"""What the entry points around the cache refuse on the host, before any CUDA call, and
the tables of rotary frequencies (host arithmetic)."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import quantized_attention_diffusion_gb300 as qad
from quantized_attention_diffusion_gb300 import build as qbuild
from quantized_attention_diffusion_gb300.sage import _KV4Cache, _KVCache, _Rope

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, NOMEM, TIMEOUT, WORKSPACE, BAD_PAGE, NO_PAGES = range(10)
FAKE = 0x10000          # 256-byte aligned, never dereferenced
OUT, KOUT = 0x4000000, 0x8000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qad.load_library()


def cache4(kc=FAKE, kb=FAKE, ks=FAKE, vc=FAKE, vb=FAKE, vs=FAKE, pages=4, H=2, page=16):
    return ctypes.byref(_KV4Cache(kc, kb, ks, vc, vb, vs, pages, H, page))


def rope(freq=FAKE, dim=128, interleaved=0, axes=1, sections=(64, 0, 0, 0), factor=1.0):
    return ctypes.byref(_Rope(freq, dim, interleaved, axes, (ctypes.c_int32 * 4)(*sections), factor))


def write(lib, c=None, D=128, B=1, table=FAKE, width=1):
    return lib.sage_kv4_cache_write(c or cache4(), P(FAKE), P(FAKE), 256, 256, 256, 256, B, 1, D, P(table), width, 1, P(FAKE), None, None)


def read(lib, c=None, D=128, B=1, table=FAKE, width=1):
    return lib.sage_kv4_cache_read(c or cache4(), P(table), width, 1, P(FAKE), P(FAKE), P(FAKE), B, 1, D, None)


def attn(lib, c=None, D=128, B=1, table=FAKE, width=1, prefix=None, Hq=4):
    tail = (P(table), width, 1, P(FAKE), P(FAKE), None, B, 1, Hq, D, 0.1, 1, None, 0, None)
    if prefix is None:
        return lib.sage_attn_fwd_kv4_cache(P(FAKE), 256, 256, c or cache4(), *tail)
    return lib.sage_attn_fwd_kv4_cache_prefix(P(FAKE), 256, 256, c or cache4(), P(prefix[0]), prefix[1], *tail)


def turn(lib, q=FAKE, k=FAKE, qs=(512, 512), ks=(256, 256), B=1, S=1, Hq=4, Hk=2, D=128, r=None, pos=FAKE, ps=(1, 1), qw=None, kw=None,
         eps=1e-6, qo=OUT, ko=KOUT):
    return lib.sage_qk_norm_rope(P(q), P(k), *qs, *ks, B, S, Hq, Hk, D, r, P(pos), *ps, P(qw), P(kw), eps, P(qo), P(ko), None)


def append(lib, c=None, q=FAKE, k=FAKE, v=FAKE, qs=(512, 512), ks=(256, 256), vs=(256, 256), B=1, S=1, Hq=4, D=128, r=None, pos=FAKE,
           ps=(1, 1), qw=None, kw=None, eps=1e-6, slots=FAKE, qo=OUT, bits=4):
    if bits == 8:
        c, fn = c or ctypes.byref(_KVCache(FAKE, FAKE, FAKE, FAKE, 4, 2, 16)), lib.sage_kv_cache_append
    else:
        c, fn = c or cache4(), lib.sage_kv4_cache_append
    return fn(c, P(q), P(k), P(v), *qs, *ks, *vs, B, S, Hq, D, r, P(pos), *ps, P(qw), P(kw), eps, P(slots), P(qo), None)


def reserve(lib, pages=8, page=16, B=1, width=2, stride=2, layout=0, tokens=1, **ptr):
    names = ("free_pages", "free_count", "lens", "counts", "table", "start", "taken", "new_lens", "first", "left", "slots", "positions")
    p = {n: P(ptr.get(n, FAKE)) for n in names}
    return lib.sage_kv_pages_reserve(p["free_pages"], p["free_count"], pages, page, p["lens"], p["counts"], B, p["table"], width, stride,
                                     layout, tokens, p["start"], p["taken"], p["new_lens"], p["first"], p["left"], p["slots"], p["positions"], None)


def release(lib, pages=8, page=16, B=1, width=2, stride=2, **ptr):
    p = {n: P(ptr.get(n, FAKE)) for n in ("free_pages", "free_count", "lens", "keep", "table")}
    return lib.sage_kv_pages_release(p["free_pages"], p["free_count"], pages, page, p["lens"], p["keep"], B, p["table"], width, stride, None)


@pytest.mark.parametrize("kw,want,text", [
    (dict(kc=0), INVALID, b"k_codes"), (dict(kb=0), INVALID, b"k_block"), (dict(vb=FAKE + 8), MISALIGNED, b"v_block"),
    (dict(vs=FAKE + 4), MISALIGNED, b"v_scale"), (dict(pages=0), INVALID, b"num_pages"), (dict(page=8), UNSUPPORTED, b"page_size"),
    (dict(pages=1 << 26), INVALID, b"2^31-1"),
])
def test_bad_caches(lib, kw, want, text):
    for call in (write, read, attn, append):
        assert call(lib, c=cache4(**kw)) == want
        assert text in lib.sage_last_error()
    assert attn(lib, c=cache4(**kw), prefix=(FAKE, 1)) == want


def test_what_the_4_bit_calls_refuse(lib):
    for call in (write, read, attn):
        assert call(lib, D=64) == UNSUPPORTED and call(lib, B=0) == INVALID
        assert call(lib, table=0) == INVALID and call(lib, width=0) == INVALID
    assert attn(lib, Hq=3) == INVALID and b"multiple" in lib.sage_last_error()
    assert attn(lib, prefix=(0, 5)) == INVALID and attn(lib, prefix=(FAKE, 0)) == INVALID
    assert lib.sage_status_string(NO_PAGES) == b"SAGE_ERR_NO_PAGES"


@pytest.mark.parametrize("bits", [0, 4, 8])
def test_what_norm_and_rotation_refuse(lib, bits):
    def call(**kw):
        return turn(lib, **kw) if bits == 0 else append(lib, bits=bits, **kw)

    assert call(D=64) == UNSUPPORTED and call(S=0) == INVALID and call(B=0) == INVALID and call(Hq=-1) == INVALID
    assert call(q=0) == INVALID and call(k=FAKE + 8) == MISALIGNED and call(qo=0) == INVALID and call(qo=OUT + 2) == MISALIGNED
    assert call(qs=(512, 12)) == MISALIGNED and call(ks=(-8, 256)) == INVALID
    assert call(B=1 << 15, S=1 << 15) == INVALID and b"2^31-1" in lib.sage_last_error()
    for eps in (math.nan, math.inf, -0.5, -2.0):
        assert call(eps=eps) == INVALID and b"eps" in lib.sage_last_error()
    assert call(eps=-1.0, kw=FAKE) == INVALID and b"weights without a norm" in lib.sage_last_error()
    assert call(qw=FAKE + 8) == MISALIGNED and call(kw=FAKE + 2) == MISALIGNED
    for dim in (0, 16, 48, 160):
        assert call(r=rope(dim=dim)) == UNSUPPORTED and b"rotated channels" in lib.sage_last_error()
    assert call(r=rope(axes=0)) == UNSUPPORTED and call(r=rope(axes=5)) == UNSUPPORTED
    assert call(r=rope(sections=(63, 0, 0, 0))) == INVALID and call(r=rope(axes=2, sections=(65, -1, 0, 0))) == INVALID
    assert call(r=rope(factor=math.nan)) == INVALID and call(r=rope(freq=0)) == INVALID and call(r=rope(freq=FAKE + 4)) == MISALIGNED
    assert call(r=rope(), pos=0) == INVALID and b"positions" in lib.sage_last_error()
    assert call(r=rope(), pos=FAKE + 2) == MISALIGNED and call(r=rope(), ps=(-1, 1)) == INVALID
    # outputs in inputs' places: k's, or a shifted q's
    assert call(q=2 * OUT, k=OUT) == INVALID and b"overlaps" in lib.sage_last_error()
    assert call(q=OUT + 256) == INVALID and b"overlaps" in lib.sage_last_error()
    assert call(q=OUT, S=2, qs=(4096, 2048)) == INVALID and b"overlaps" in lib.sage_last_error()     # rows of q are apart
    if bits == 0:
        assert call(ko=OUT + 512) == INVALID and b"overlaps" in lib.sage_last_error()
        assert call(Hk=-1) == INVALID and call(ko=0) == INVALID
    else:
        assert call(v=0) == INVALID and call(vs=(256, 4)) == MISALIGNED and call(slots=0) == INVALID and call(slots=FAKE + 1) == MISALIGNED
        assert call(q=2 * OUT, v=OUT) == INVALID and b"overlaps" in lib.sage_last_error()


def test_what_the_page_calls_refuse(lib):
    for call in (reserve, release):
        assert call(lib, pages=0) == INVALID and call(lib, pages=1 << 28) == INVALID
        assert call(lib, page=24) == UNSUPPORTED and call(lib, page=8) == UNSUPPORTED
        assert call(lib, B=0) == INVALID and call(lib, B=(1 << 20) + 1) == INVALID
        assert call(lib, table=0) == INVALID and call(lib, width=0) == INVALID and call(lib, B=2, stride=1) == INVALID
        for name in ("free_pages", "free_count", "lens"):
            assert call(lib, **{name: 0}) == INVALID and name.encode() in lib.sage_last_error()
            assert call(lib, **{name: FAKE + 2}) == MISALIGNED
    assert release(lib, keep=0) == INVALID
    for name in ("counts", "start", "taken", "new_lens", "first", "slots", "positions"):
        assert reserve(lib, **{name: 0}) == INVALID and name.encode() in lib.sage_last_error()
    assert reserve(lib, left=0) == INVALID and b"free_left" in lib.sage_last_error()
    assert reserve(lib, layout=3) == UNSUPPORTED and reserve(lib, layout=-1) == UNSUPPORTED
    assert reserve(lib, tokens=0) == INVALID and reserve(lib, B=1 << 16, layout=1, tokens=1 << 15) == INVALID


# ------------------------------------------------------------- frequencies --

TWO_PI = 2 * Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)


def table(lib, dim, base=10000.0, scaling=0, factor=1.0, length=0.0, low=1.0, high=32.0):
    f, a = (ctypes.c_uint64 * (dim // 2))(), ctypes.c_double()
    assert lib.sage_rope_frequencies(dim, base, scaling, factor, length, low, high, f, ctypes.byref(a)) == OK
    return list(f), a.value


def test_a_frequency_is_the_nearest_2_64th_of_a_revolution(lib):
    for f in (1.0, 0.1, 1e-4, 2.9999, 1e-9, 0.7071067811865476, 5e-324, 0.0, -1.0, -0.3):
        want = Fraction(f) / TWO_PI * 2 ** 64
        got = lib.sage_rope_frequency(f)
        got -= (1 << 64) if got >> 63 else 0
        assert abs(got - want) <= Fraction(1, 2) + Fraction(1, 2 ** 20)
    for f in (math.nan, math.inf, 3.5):
        assert lib.sage_rope_frequency(f) == 0


@pytest.mark.parametrize("dim", [2, 32, 96, 128])
def test_frequencies_of_each_scaling(lib, dim):
    """Powers and logarithms are within some ulp of Python's: 2^-45 of a frequency."""
    n = dim // 2
    plain = [10000.0 ** (-2.0 * i / dim) for i in range(n)]

    def check(got, want):
        for g, w in zip(got, want):
            assert abs(g - Fraction(w) / TWO_PI * 2 ** 64) <= Fraction(w) * 2 ** 17 + 1

    got, factor = table(lib, dim)
    check(got, plain)
    assert factor == 1.0
    check(table(lib, dim, scaling=1, factor=4.0)[0], [f / 4 for f in plain])
    base = 10000.0 * (8.0 ** (dim / (dim - 2)) if dim > 2 else 1.0)
    check(table(lib, dim, scaling=2, factor=8.0)[0], [base ** (-2.0 * i / dim) for i in range(n)])
    lo, hi = (f(dim * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(10000.0))) for f, t in ((math.floor, 32.0), (math.ceil, 1.0)))
    lo, hi = max(0, lo), min(dim - 1, hi)
    ramp = [min(1.0, max(0.0, (i - lo) / max(1e-3, hi - lo))) for i in range(n)]
    got, factor = table(lib, dim, scaling=3, factor=4.0, length=4096.0)
    check(got, [f / 4 * r + f * (1 - r) for f, r in zip(plain, ramp)])
    assert abs(factor - (0.1 * math.log(4.0) + 1)) < 1e-15
    keep = [min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1) / 3)) for f in plain]
    check(table(lib, dim, scaling=4, factor=8.0, length=8192.0, low=1.0, high=4.0)[0], [f / 8 * (1 - k) + f * k for f, k in zip(plain, keep)])


def test_what_the_frequencies_refuse(lib):
    f, a = (ctypes.c_uint64 * 64)(), ctypes.c_double()

    def call(dim=64, base=1e4, scaling=0, factor=1.0, length=100.0, low=1.0, high=4.0, f=f, a=ctypes.byref(a)):
        return lib.sage_rope_frequencies(dim, base, scaling, factor, length, low, high, f, a)

    assert call() == OK
    for dim in (0, 7, 130, -2):
        assert call(dim=dim) == INVALID
    for base in (1.0, 0.0, math.nan, math.inf):
        assert call(base=base) == INVALID
    assert call(scaling=5) == UNSUPPORTED and call(scaling=-1) == UNSUPPORTED
    assert call(scaling=1, factor=0.5) == INVALID and call(scaling=3, length=0.0) == INVALID
    assert call(scaling=4, low=4.0, high=4.0) == INVALID and call(scaling=3, low=0.0) == INVALID
    assert call(f=None) == INVALID and call(a=None) == INVALID


def test_binding_makes_and_refuses_ropes():
    r = qad.Rope(64, interleaved=True, sections=(8, 24), device="cpu")
    assert r.freq.shape == (32,) and r.sections == (8, 24) and r.factor == 1.0
    assert r.freq[0] == r.freq[8]                       # each axis begins at one radian
    y = qad.Rope(128, scaling=("yarn", 4.0, 4096), device="cpu")
    assert abs(y.factor - (0.1 * math.log(4.0) + 1)) < 1e-15
    own = qad.Rope(32, freqs=[1.0] * 16, factor=2.0, device="cpu")
    assert own.factor == 2.0 and own.freq.unique().numel() == 1 and own.freq[0] == r.freq[0]
    for kw in (dict(dim=48), dict(sections=(10, 10)), dict(sections=(1,) * 5), dict(sections=(64, 0)), dict(scaling=("yarn", 2.0)),
               dict(scaling=("none", 2.0)), dict(scaling=("linear",)), dict(freqs=[1.0]), dict(freqs=[4.0] * 64),
               dict(freqs=[1.0] * 64, scaling=("linear", 2.0))):
        with pytest.raises(ValueError):
            qad.Rope(**{"dim": 128, "device": "cpu", **kw})
    with pytest.raises(qad.SageError, match="factor"):
        qad.Rope(scaling=("linear", 0.5), device="cpu")
    with pytest.raises(ValueError, match="bits"):
        qad.kv_cache_alloc(4, 2, 16, device="cpu", bits=6)
    c = qad.kv_cache_alloc(4, 2, 16, device="cpu", bits=4)
    assert [(tuple(t.shape), t.dtype) for t in c[:3]] == [((4, 2, 16, 64), torch.uint8), ((4, 2, 16, 8), torch.float8_e4m3fn), ((4, 2, 16), torch.float32)]
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        qad.attn_fwd_cache(q, c, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        qad.qk_norm_rope(q)


# ------------------------------------------------------------ index bounds --

@pytest.mark.parametrize("rot", [0, 32, 64, 96, 128])
def test_lanes_hold_every_channel_once_and_both_of_their_pairs(rot):
    """The lanes of qk_rope.cu: chunks of 8 channels c0, c1 of lane l, n = rot / 16."""
    n = rot // 16
    c0 = [l if l < n else n + l for l in range(8)]
    c1 = [n + l if l < n else 8 + l for l in range(8)]
    assert sorted(c0 + c1) == list(range(16))
    for l in range(8):
        assert c0[l] // 2 == c0[l ^ 1] // 2 and c1[l] // 2 == c1[l ^ 1] // 2      # blocks of 16 channels, for 4 bits
        if l < n:
            assert 8 * c1[l] == 8 * c0[l] + rot // 2 and 8 * c0[l] + 7 < rot // 2
            assert 4 * c1[l] + 3 < rot // 2                                         # interleaved pairs
        else:
            assert 8 * c0[l] >= rot and 8 * c1[l] >= rot


def test_a_4_bit_tile_fits_its_stage_and_every_copy_is_aligned():
    """cache_attention.cu: offsets of a tile of 128 keys, the runs of each page size and
    the sixteen-byte copies of its scales."""
    row, tok = 64, 128
    off_v, off_ks = tok * row, 2 * tok * row
    off_vs = off_ks + 4 * tok
    off_kb = off_vs + 4 * tok
    off_vb = off_kb + 8 * tok
    size = off_vb + 8 * tok
    for page in (16, 32, 64, 128, 256):
        run, shift = min(tok, page), min(7, page.bit_length() - 1)
        runs = tok // run
        assert 2 * runs <= 32 and run * row % 16 == 0
        seen = set()
        for lane in range(2 * runs):
            o, part = (lane >> 1) * run, lane & 1
            seen |= set(range(part * off_v + o * row, part * off_v + (o + run) * row))
        assert seen == set(range(off_ks))
        for lane in range(32):
            for i in range(2):
                key = 64 * i + 2 * lane
                assert key + 1 < tok and (key >> shift) < runs and key // run == (key + 1) // run
                for base in (off_kb, off_vb):
                    assert (base + key * 8) % 16 == 0 and not seen & set(range(base + key * 8, base + key * 8 + 16))
                    seen |= set(range(base + key * 8, base + key * 8 + 16))
            key = 4 * lane
            assert key // run == (key + 3) // run
            for base in (off_ks, off_vs):
                seen |= set(range(base + key * 4, base + key * 4 + 16))
    assert seen == set(range(size))
    # three CTAs of two stages, or two of four, on an SM of 228 KB: merge 16 KB, queries, static memory, 1 KB each
    for nt, ctas, stages in ((1, 3, 2), (2, 2, 4)):
        assert ctas * (stages * size + 16384 + 2048 * nt + 4096 + 1024) <= 228 * 1024
