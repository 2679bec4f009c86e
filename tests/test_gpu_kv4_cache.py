"""The 4-bit KV cache on the GPU: writing (bit for bit against the stated
quantiser), reading back, and the attention over it against float64, within the
bounds of the 8-bit cache's tests (K's and V's values, code times block scale, are
exact in fp16 and take the codes' place)."""
import math

import pytest
import torch

from tests.cache_common import D, assert_within, ints, join, reference
from tests.gpu_common import ensure_library
from tests.kv4_common import Cache4, quantize4, values4

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)
NAMES = ("k_codes", "k_block", "k_scale", "v_codes", "v_block", "v_scale")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    import quantized_attention_diffusion_gb300 as qad
    yield
    assert qad.sync_status() == 0


def _marked(num_pages, H, page):
    import quantized_attention_diffusion_gb300 as qad
    cache = qad.kv_cache_alloc(num_pages, H, page, bits=4)
    for t in cache:
        t.view(torch.uint8).fill_(0xA5)
    return cache


def _expected(cache, table, start, count, k, v):
    want = [t.cpu().clone() for t in cache]
    page = want[0].shape[2]
    rows = quantize4(k) + quantize4(v)
    for b in range(k.shape[0]):
        for i in range(count[b]):
            p, o = int(table[b, (start[b] + i) // page]), (start[b] + i) % page
            for dst, src in zip(want, rows):
                if dst.dtype == torch.float32:
                    dst[p, :, o] = src[b, i]
                else:
                    dst.view(torch.uint8)[p, :, o] = src[b, i].view(torch.uint8)
    return want


def _assert_cache(cache, want):
    for name, got, ref in zip(NAMES, cache, want):
        got = got.cpu()
        if got.dtype == torch.float32:
            same = (got.view(torch.int32) == ref.view(torch.int32)) | (torch.isnan(got) & torch.isnan(ref))
            assert same.all(), name
        else:
            assert torch.equal(got.view(torch.uint8), ref.view(torch.uint8)), name


@pytest.mark.parametrize("B,S,H,page,start,count", [
    (1, 1, 1, 16, [0], None),
    (3, 1, 2, 16, [15, 16, 47], None),
    (2, 37, 3, 32, [0, 5], [37, 0]),
    (4, 70, 5, 64, [1, 63, 64, 0], [70, 1, 33, 99]),
    (2, 130, 7, 128, [200, 3], None),
    (1, 300, 16, 256, [100], None),
])
def test_write_is_bit_exact_and_touches_nothing_else(B, S, H, page, start, count):
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(B * 1000 + S)
    # channels of unlike size, so that blocks differ
    k = (torch.randn((B, S, H, D), generator=g) * torch.randn((B, S, H, 8, 1), generator=g).exp().expand(-1, -1, -1, -1, 16).flatten(-2)).to(torch.bfloat16)
    v = torch.randn((B, S, H, D), generator=g).to(torch.bfloat16)
    width = max(-(-(s + S) // page) for s in start) + 1
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width)
    cache = _marked(B * width, H, page)
    live = [S] * B if count is None else [min(S, c) for c in count]
    want = _expected(cache, table, start, live, k, v)
    got = qad.kv_cache_write(k.cuda(), v.cuda(), cache, table.cuda(), ints(start), None if count is None else ints(count))
    assert got is cache
    _assert_cache(cache, want)


def test_write_of_special_rows_and_reading_back():
    """Zeros of both signs, subnormals, the largest magnitudes, infinities, NaN, blocks
    that vanish beside the largest, and every border between two codes."""
    import quantized_attention_diffusion_gb300 as qad
    S, H = 64, 2
    g = torch.Generator().manual_seed(6)
    x = torch.randn((1, S, H, D), generator=g)
    for i, f in enumerate((0.0, -0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -120, 2.0 ** -115, 2.0 ** -113, 2.0 ** -100, 2.0 ** 100, 2.0 ** 125)):
        x[0, i] *= f
    x[0, 20, 0, 7] = math.inf
    x[0, 21, 1, 127] = -math.inf
    x[0, 22, 0, 64] = math.nan
    x[0, 23, :, :64] *= 2.0 ** -20
    x[0, 24, :, 1:] *= 2.0 ** -12
    x[0, 25, 0, 0] = 3.3895313892515355e38
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i in range(26, 42):               # the block's largest is 6 times an E4M3 value, the others on borders of it
        sb = 1 + (i % 8) / 8
        x[0, i] = (borders.repeat(16) * sb * torch.where(torch.rand(D, generator=g) < 0.5, -1.0, 1.0))[None]
    x[0, 42] = 2688.0                     # exactly the largest of its power of two
    x[0, 43] = 2704.0
    x = x.to(torch.bfloat16)
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32)
    cache = _marked(4, H, 16)
    y = x.flip(1)
    want = _expected(cache, table, [0], [S], x, y)
    qad.kv_cache_write(x.cuda(), y.cuda(), cache, table.cuda(), ints([0]))
    _assert_cache(cache, want)
    k, v = qad.kv_cache_read(cache, table.cuda(), ints([S]), S + 5)
    for got, src in ((k, x), (v, y)):
        c, b, s = quantize4(src[0])
        ref = (values4(c, b) * s.double()[..., None]).float().to(torch.bfloat16)
        got = got[0].cpu()
        assert ((got[:S] == ref) | (got[:S].isnan() & ref.isnan())).all()
        assert not got[S:].view(torch.int16).any()


def test_a_row_is_off_by_its_roundings_alone():
    """|x - value| of normal rows: codes are off by a quarter of |x| at most, or by half
    the smallest step of 0.5 times the block's scale (|x| behind 6, where that was rounded
    down, by a 16th)."""
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(9)
    x = torch.randn((1, 64, 3, D), generator=g).to(torch.bfloat16)
    cache = qad.kv_cache_alloc(4, 3, 16, bits=4)
    table = ints([3, 1, 0, 2]).view(1, 4)
    qad.kv_cache_write(x.cuda(), x.cuda(), cache, table, ints([0]))
    k, _ = qad.kv_cache_read(cache, table, ints([64]), 64)
    x, k = x.double(), k.double().cpu()
    block = x.abs().unflatten(-1, (8, 16)).amax(-1, keepdim=True).expand(*x.shape[:-1], 8, 16).flatten(-2) / 6 * (1 + 2.0 ** -4)
    assert ((x - k).abs() <= torch.maximum(0.25 * x.abs(), 0.25 * block)).all()


# ------------------------------------------------------------- attention --

def _attend(cache, q, causal, scale=SCALE, prefix=None):
    import quantized_attention_diffusion_gb300 as qad
    B = q.shape[0]
    t = cache.table.cuda()
    if prefix is None:
        return qad.attn_fwd_cache(q.cuda(), cache.gpu(), t[:B].contiguous(), ints(cache.lens), softmax_scale=scale, causal=causal, return_lse=True)
    return qad.attn_fwd_cache_prefix(q.cuda(), cache.gpu(), t[B, :-(-prefix // cache.page)].contiguous(), prefix, t[:B].contiguous(),
                                     ints(cache.lens), softmax_scale=scale, causal=causal, return_lse=True)


def _check(cache, q, causal, prefix=None, scale=SCALE):
    out, lse = _attend(cache, q, causal, scale, prefix)
    for b in range(q.shape[0]):
        rows = cache.dense(b) if prefix is None else join(cache.dense(q.shape[0]), cache.dense(b))
        ref, z, tol, ltol = reference(q[b], rows, causal, scale)
        assert_within(out[b], ref, tol, f"out of sequence {b}")
        assert_within(lse[b], z, ltol, f"lse of sequence {b}")


@pytest.mark.parametrize("lens,Sq,Hq,Hkv,page,causal,recipe", [
    ([1], 1, 1, 1, 16, True, "normal"),
    ([777], 1, 32, 8, 16, True, "offset"),                     # clusters
    ([0, 1, 63, 64, 65, 200], 1, 8, 2, 16, True, "normal"),
    ([5, 130, 257], 3, 6, 2, 32, True, "sharp"),
    ([300, 17], 2, 4, 4, 64, False, "offset"),
    ([1000, 3, 500], 1, 7, 1, 128, True, "sharp"),
    ([256, 255], 1, 2, 2, 256, True, "normal"),
    ([40, 12], 64, 2, 1, 16, True, "normal"),                  # longer chunks than sequences: rows that see nothing
    ([700, 650], 40, 8, 2, 64, True, "offset"),                # the wide kernel, or clusters
    ([513, 129], 300, 2, 2, 32, False, "normal"),
    ([900], 333, 3, 1, 16, True, "sharp"),
])
def test_attention(lens, Sq, Hq, Hkv, page, causal, recipe):
    g = torch.Generator().manual_seed(sum(lens) + Sq)
    cache = Cache4(lens, Hkv, page, seed=len(lens) * 7 + Sq, recipe=recipe)
    q = torch.randn((len(lens), Sq, Hq, D), generator=g).to(torch.bfloat16)
    _check(cache, q, causal)


@pytest.mark.parametrize("B,n,Sq,Hq,Hkv,page", [
    (2, 12000, 1, 8, 8, 64),        # 8 rows: CTAs share sequences
    (3, 5000, 1, 16, 1, 128),       # 16 rows
    (40, 500, 4, 8, 2, 16),         # 16 rows
    (2, 4000, 8, 4, 1, 32),         # 32 rows: the wide kernel, halves are key tiles
    (1, 3000, 200, 4, 2, 64),       # 400 rows: row tiles
])
def test_long_attention(B, n, Sq, Hq, Hkv, page):
    import random
    r = random.Random(n)
    lens = [r.randint(n // 2, n) for _ in range(B)]
    g = torch.Generator().manual_seed(n)
    cache = Cache4(lens, Hkv, page, seed=n, recipe="offset")
    q = torch.randn((B, Sq, Hq, D), generator=g).to(torch.bfloat16)
    _check(cache, q, True)


@pytest.mark.parametrize("B,prefix,lens,Sq,Hq,Hkv,page,causal", [
    (3, 100, [1, 5, 40], 1, 4, 2, 16, True),        # one launch
    (2, 1, [0, 1], 1, 2, 2, 32, True),
    (6, 5000, [1, 90, 33, 64, 65, 2], 1, 8, 2, 64, True),
    (24, 3000, [5 + i for i in range(24)], 5, 4, 1, 128, True),      # the wide kernel for the prefix
    (2, 777, [4, 3], 4, 4, 2, 16, False),
])
def test_prefix(B, prefix, lens, Sq, Hq, Hkv, page, causal):
    g = torch.Generator().manual_seed(prefix)
    cache = Cache4(lens, Hkv, page, seed=prefix + B, recipe="offset", extra=(prefix,))
    q = torch.randn((B, Sq, Hq, D), generator=g).to(torch.bfloat16)
    _check(cache, q, causal, prefix=prefix)


@pytest.mark.parametrize("Sq", [1, 40])
def test_scales_of_v_far_apart_and_rows_of_zeros(Sq):
    """V's scales over many powers of two, zeros among them: weights keep their bits."""
    def spread(n, g):
        s = torch.exp2(torch.randint(-40, 41, (n, 1, 1), generator=g).float())
        return torch.where(torch.rand((n, 1, 1), generator=g) < 0.1, torch.zeros(()), s)

    cache = Cache4([300, 1000], 2, 16, seed=5, v_scale=spread)
    q = torch.randn((2, Sq, 8, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    _check(cache, q, True)


def test_a_nan_row_reaches_those_that_see_it_alone():
    import quantized_attention_diffusion_gb300 as qad
    cache = Cache4([200, 200], 2, 16, seed=3)
    gpu = cache.gpu()
    page, at = int(cache.table[0, 100 // 16]), 100 % 16
    gpu[5][page, 1, at] = math.nan                     # V's scale of key 100, head 1, sequence 0
    q = torch.randn((2, 120, 4, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = qad.attn_fwd_cache(q.cuda(), gpu, cache.table.cuda(), ints([200, 200]))
    sees = torch.arange(120) >= 20                     # query i sees positions up to 80 + i
    assert out[0, sees][:, 2:].isnan().all()
    assert not out[0, ~sees].isnan().any() and not out[0, :, :2].isnan().any() and not out[1].isnan().any()
    for Sq in (1, 120):
        ref, _, tol, _ = reference(q[1, -Sq:], cache.dense(1), True, SCALE)
        got = qad.attn_fwd_cache(q[:, -Sq:].contiguous().cuda(), gpu, cache.table.cuda(), ints([200, 200]))
        assert_within(got[1], ref, tol)


def test_bad_pages_are_reported_and_stay_with_their_sequence():
    import quantized_attention_diffusion_gb300 as qad
    cache = Cache4([150, 90], 2, 16, seed=8)
    for bad in (-1, cache.num_pages, 2 ** 30):
        table = cache.table.clone()
        table[0, 4] = bad
        for Sq in (1, 100):
            q = torch.randn((2, Sq, 4, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
            out = qad.attn_fwd_cache(q.cuda(), cache.gpu(), table.cuda(), ints([150, 90]), causal=False)
            assert qad.sync_status() == 8
            ref, _, tol, _ = reference(q[1], cache.dense(1), False, SCALE)
            assert_within(out[1], ref, tol)
        k, _ = qad.kv_cache_read(cache.gpu(), table.cuda(), ints([150, 90]), 150)
        assert qad.sync_status() == 8
        assert not k[0, 64:80].any() and k[0, 63].any() and k[0, 80].any()


def test_offsets_behind_4_gb():
    """Rows whose codes begin behind 2^32 bytes of their tensor."""
    import quantized_attention_diffusion_gb300 as qad
    H, page = 16, 256
    pages = (1 << 32) // (H * page * 64) + 300
    cache = qad.kv_cache_alloc(pages, H, page, bits=4)
    n = 600
    x = torch.randn((1, n, H, D), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    table = ints([pages - 1, pages - 200, pages - 3]).view(1, 3)
    qad.kv_cache_write(x.cuda(), x.cuda(), cache, table, ints([0]))
    k, v = qad.kv_cache_read(cache, table, ints([n]), n)
    assert torch.equal(k, v)
    c, b, s = quantize4(x[0])
    assert torch.equal(k[0].cpu(), (values4(c, b) * s.double()[..., None]).to(torch.bfloat16))
    dense = (values4(c, b), s.double()) * 2
    for Sq in (1, 40):
        q = torch.randn((1, Sq, H, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        out = qad.attn_fwd_cache(q.cuda(), cache, table, ints([n]))
        ref, _, tol, _ = reference(q[0], dense, True, SCALE)
        assert_within(out[0], ref, tol)


def test_workspace_streams_and_graphs():
    """A caller's workspace, another stream, and a recorded call that follows the
    lengths: the same bits."""
    import quantized_attention_diffusion_gb300 as qad
    cache = Cache4([4000, 3500], 8, 64, seed=4)
    gpu, table = cache.gpu(), cache.table.cuda()
    q = torch.randn((2, 1, 32, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    lens = ints([4000, 3500])
    want = qad.attn_fwd_cache(q, gpu, table, lens)
    ws = torch.empty(qad.attn_fwd_cache_workspace_bytes(2, 1, 32, 8), dtype=torch.uint8, device="cuda")
    assert torch.equal(qad.attn_fwd_cache(q, gpu, table, lens, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = qad.attn_fwd_cache(q, gpu, table, lens)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(q)
    with torch.cuda.graph(graph):
        qad.attn_fwd_cache(q, gpu, table, lens, out=out)
    for n in ([4000, 3500], [1, 2000], [0, 3499]):
        lens.copy_(ints(n))
        graph.replay()
        assert torch.equal(out, qad.attn_fwd_cache(q, gpu, table, lens))


def test_refusals():
    import quantized_attention_diffusion_gb300 as qad
    c = qad.kv_cache_alloc(4, 2, 16, bits=4)
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), ints([1])
    q = torch.zeros((1, 1, 4, D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="k_codes must be"):
        qad.attn_fwd_cache(q, (c[0].view(torch.int8),) + c[1:], table, lens)
    with pytest.raises(ValueError, match="4 bits is codes"):
        qad.attn_fwd_cache(q, (c[0], c[1][..., :4].contiguous()) + c[2:], table, lens)
    with pytest.raises(ValueError, match="contiguous"):
        qad.attn_fwd_cache(q, (c[0][::2],) + c[1:], table, lens)
    with pytest.raises(ValueError, match="one device"):
        qad.attn_fwd_cache(q, c[:5] + (c[5].cpu(),), table, lens)
    with pytest.raises(TypeError):
        qad.attn_fwd_cache(q, c[:5], table, lens)
