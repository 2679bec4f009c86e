"""What the KV cache's entry points refuse on the host, before any CUDA call."""
import ctypes

import pytest
import torch

import quantized_attention_diffusion_gb300 as qad
from quantized_attention_diffusion_gb300 import build as qbuild
from quantized_attention_diffusion_gb300.sage import _KVCache

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, NOMEM, TIMEOUT, WORKSPACE, BAD_PAGE = range(9)
FAKE = 0x10000          # a 256-byte aligned, never dereferenced address
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return qad.load_library()


def cache(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=4, H=2, page=16):
    return ctypes.byref(_KVCache(kc, ks, vc, vs, pages, H, page))


def write(lib, c=None, k=FAKE, v=FAKE, ksb=256, kss=256, vsb=256, vss=256, B=1, S=1, D=128, table=FAKE, width=1,
          stride=1, start=FAKE, count=None):
    return lib.sage_kv_cache_write(cache() if c is None else c, P(k), P(v), ksb, kss, vsb, vss, B, S, D, P(table),
                                   width, stride, P(start), P(count), None)


def read(lib, c=None, table=FAKE, width=1, stride=1, lens=FAKE, k=FAKE, v=FAKE, B=1, S=1, D=128):
    return lib.sage_kv_cache_read(cache() if c is None else c, P(table), width, stride, P(lens), P(k), P(v), B, S, D,
                                  None)


def attn(lib, q=FAKE, qsb=256, qss=256, c=None, table=FAKE, width=1, stride=1, lens=FAKE, out=FAKE, lse=None, B=1,
         Sq=1, Hq=4, D=128, scale=0.1, ws=None, ws_bytes=0, prefix=None):
    head = (P(q), qsb, qss, cache() if c is None else c)
    tail = (P(table), width, stride, P(lens), P(out), P(lse), B, Sq, Hq, D, scale, 1, P(ws), ws_bytes, None)
    if prefix is None:
        return lib.sage_attn_fwd_cache(*head, *tail)
    return lib.sage_attn_fwd_cache_prefix(*head, P(prefix[0]), prefix[1], *tail)


BAD_CACHES = [
    (dict(kc=0), INVALID, b"k_codes"), (dict(vs=0), INVALID, b"v_scale"), (dict(vc=FAKE + 8), MISALIGNED, b"v_codes"),
    (dict(ks=FAKE + 4), MISALIGNED, b"k_scale"), (dict(pages=0), INVALID, b"num_pages"), (dict(H=0), INVALID, b"H"),
    (dict(page=8), UNSUPPORTED, b"page_size"), (dict(page=48), UNSUPPORTED, b"page_size"),
    (dict(pages=1 << 26), INVALID, b"2^31-1"), (dict(page=512), UNSUPPORTED, b"page_size"), (dict(page=-16), UNSUPPORTED, b"page_size"),
]


@pytest.mark.parametrize("kw,want,text", BAD_CACHES)
def test_bad_caches(lib, kw, want, text):
    for call in (write, read, attn):
        assert call(lib, c=cache(**kw)) == want
        assert text in lib.sage_last_error()
    assert attn(lib, c=cache(**kw), prefix=(FAKE, 1)) == want


@pytest.mark.parametrize("call", [write, read, attn])
def test_what_all_refuse(lib, call):
    assert lib.sage_kv_cache_write(None, *[P(FAKE)] * 2, 8, 8, 8, 8, 1, 1, 128, P(FAKE), 1, 1, P(FAKE), None, None) == INVALID
    assert call(lib, D=64) == UNSUPPORTED
    assert call(lib, B=0) == INVALID and call(lib, B=-2) == INVALID
    assert call(lib, table=0) == INVALID and b"block_table" in lib.sage_last_error()
    assert call(lib, table=FAKE + 2) == MISALIGNED
    assert call(lib, width=0) == INVALID and call(lib, stride=-1) == INVALID


def test_write_refuses(lib):
    assert write(lib, S=0) == INVALID
    assert write(lib, k=0) == INVALID and write(lib, v=FAKE + 2) == MISALIGNED
    assert write(lib, kss=100) == MISALIGNED and b"k's strides" in lib.sage_last_error()
    assert write(lib, vsb=-8) == INVALID and b"v has a negative stride" in lib.sage_last_error()
    assert write(lib, start=0) == INVALID and write(lib, start=FAKE + 1) == MISALIGNED
    assert write(lib, count=FAKE + 2) == MISALIGNED
    assert write(lib, B=1 << 16, S=1 << 14) == INVALID and b"2^31-1" in lib.sage_last_error()


def test_read_refuses(lib):
    assert read(lib, S=0) == INVALID
    assert read(lib, k=0) == INVALID and read(lib, v=FAKE + 8) == MISALIGNED
    assert read(lib, k=FAKE + 16) == MISALIGNED and b"32-byte" in lib.sage_last_error()
    assert read(lib, lens=0) == INVALID and read(lib, lens=FAKE + 2) == MISALIGNED
    assert read(lib, B=1 << 16, S=1 << 14) == INVALID


@pytest.mark.parametrize("prefix", [None, (FAKE, 100)])
def test_attention_refuses(lib, prefix):
    assert attn(lib, Sq=0, prefix=prefix) == INVALID and attn(lib, Hq=0, prefix=prefix) == INVALID
    assert attn(lib, Hq=3, prefix=prefix) == INVALID and b"multiple" in lib.sage_last_error()
    assert attn(lib, B=1 << 15, Sq=1 << 14, prefix=prefix) == INVALID
    for scale in (float("nan"), float("inf"), 0.0, -1.0):
        assert attn(lib, scale=scale, prefix=prefix) == INVALID
    assert attn(lib, q=0, prefix=prefix) == INVALID and attn(lib, q=FAKE + 8, prefix=prefix) == MISALIGNED
    assert attn(lib, qss=12, prefix=prefix) == MISALIGNED and attn(lib, qsb=-8, prefix=prefix) == INVALID
    assert attn(lib, out=FAKE + 16, prefix=prefix) == MISALIGNED and attn(lib, lse=FAKE + 4, prefix=prefix) == MISALIGNED
    assert attn(lib, lens=0, prefix=prefix) == INVALID
    need = lib.sage_attn_fwd_cache_workspace_bytes(1, 1, 4, 2, 0 if prefix is None else prefix[1])
    assert attn(lib, ws=FAKE, ws_bytes=need - 1, prefix=prefix) == WORKSPACE
    assert attn(lib, ws=FAKE + 16, ws_bytes=need, prefix=prefix) == MISALIGNED


def test_prefix_refuses(lib):
    assert attn(lib, prefix=(0, 5)) == INVALID and b"prefix_table" in lib.sage_last_error()
    assert attn(lib, prefix=(FAKE + 2, 5)) == MISALIGNED
    for n in (0, -1, (1 << 30) + 1):
        assert attn(lib, prefix=(FAKE, n)) == INVALID and b"prefix_len" in lib.sage_last_error()


def test_workspace_bytes(lib):
    n = lib.sage_attn_fwd_cache_workspace_bytes
    assert n(1, 1, 8, 2, 0) > 0
    # the sequences' number does not enter without a prefix
    assert n(300, 1, 8, 2, 0) == n(1, 1, 8, 2, 0)
    assert n(8, 1, 8, 2, 100) > n(1, 1, 8, 2, 100) > n(1, 1, 8, 2, 0)
    for bad in ((0, 1, 8, 2, 0), (1, 0, 8, 2, 0), (1, 1, 8, 3, 0), (1, 1, 8, 0, 0), (1, 1, 8, 2, -1)):
        assert n(*bad) == 0
    assert lib.sage_status_string(BAD_PAGE) == b"SAGE_ERR_BAD_PAGE"


def test_binding_refuses():
    with pytest.raises(ValueError, match="page_size"):
        qad.kv_cache_alloc(4, 2, 20, device="cpu")
    with pytest.raises(ValueError, match="num_pages"):
        qad.kv_cache_alloc(0, 2, 16, device="cpu")
    c = qad.kv_cache_alloc(4, 2, 16, device="cpu")
    assert [t.dtype for t in c] == [torch.int8, torch.float32, torch.float8_e4m3fn, torch.float32]
    q = torch.zeros((1, 1, 4, 128), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 1), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        qad.attn_fwd_cache(q, c, table, lens)
    with pytest.raises(TypeError):
        qad.kv_cache_read(c[:3], table, lens, 1)
    with pytest.raises(ValueError, match="k_codes must be"):
        qad.kv_cache_read((c[0].float(),) + c[1:], table, lens, 1)


def test_attention_refuses_more_than_a_launch_counts(lib):
    # 2^23 units of 2^23 tiles of keys: no CTA's share fits 31 bits
    big = dict(c=cache(H=128), B=256, Sq=65535, Hq=128, width=(1 << 31) - 1)
    assert attn(lib, **big) == INVALID and b"too much for one call" in lib.sage_last_error()
    assert attn(lib, **dict(big, width=1), prefix=(FAKE, 1 << 30)) == INVALID
    assert b"too much for one call" in lib.sage_last_error()
