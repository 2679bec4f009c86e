"""The attention over the KV cache where a key/value head has more than 32 query
rows (chunks, long prefixes' continuations), against float64 within bounds that
count its roundings: the sizes, masks, scales and page tables where it can go
wrong."""
import math

import pytest
import torch

from tests.cache_common import D, Cache, assert_within, ints, join, quantize_kv, reference
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


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


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


def _q(B, Sq, Hq, seed, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Sq, Hq, D), generator=g) * mul).to(torch.bfloat16)


def _roomy(c):
    """The cache's table with room for far more keys than clusters of CTAs take."""
    width = -(-20000 // c.page)
    return torch.nn.functional.pad(c.table, (0, max(0, width - c.table.shape[1])), value=-1)


def _check(out, lse, q, c, causal, scale=SCALE, prefix=None, what=""):
    for b in range(q.shape[0]):
        rows = c.dense(b) if prefix is None else join(c.dense(prefix), c.dense(b))
        ro, rl, to, tl = reference(q[b], rows, causal, scale)
        assert_within(out[b], ro, to, f"{what} out[{b}]")
        if lse is not None:
            assert_within(lse[b], rl, tl, f"{what} lse[{b}]")


SHAPES = [
    # lens, Sq, H, G, page: at most 128 rows (tiles of keys in turn), exactly 128,
    # 129 to 256 (tiles of rows), more; one key, one tile, odd and even numbers of tiles
    ([1, 128, 129, 256], 33, 1, 1, 16), ([400, 600], 16, 3, 8, 64), ([127, 385], 43, 2, 3, 128), ([640], 256, 1, 1, 256),
    ([1000, 0, 65], 65, 1, 2, 32),
    # fewer keys than queries: rows that see nothing
    ([40, 0, 300, 1], 100, 1, 3, 32), ([5], 300, 2, 1, 16),
    # many units of a single tile of keys behind full ones
    ([100] * 40, 70, 8, 4, 64), ([1] * 200, 34, 3, 1, 16), ([128] * 60, 65, 4, 4, 128),
]


@pytest.mark.parametrize("lens,Sq,H,G,page", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
def test_shapes(lens, Sq, H, G, page, causal):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=Sq + G, recipe="sharp")
    q = _q(len(lens), Sq, H * G, seed=Sq)
    for table in (c.table.cuda(), _roomy(c).cuda()):
        out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), table, ints(lens), causal=causal, return_lse=True)
        _check(out, lse, q, c, causal)
        again = qad.attn_fwd_cache(q.cuda(), c.gpu(), table, ints(lens), causal=causal)
        assert torch.equal(bits(again), bits(out))


@pytest.mark.parametrize("P,lens,Sq,H,G", [(1, [0, 3] * 20, 1, 2, 1), (128, [1] * 40, 1, 1, 1), (513, [9, 0] * 70, 1, 1, 1), (900, [7, 60, 5], 5, 2, 10)])
@pytest.mark.parametrize("causal", [True, False])
def test_prefixes(P, lens, Sq, H, G, causal):
    import quantized_attention_diffusion_gb300 as qad
    B = len(lens)
    c = Cache(lens, H, 32, seed=P, extra=[P], recipe="sharp")
    wide = _q(B, Sq + 2, H * G + 3, seed=P + 1).cuda()
    q = wide[:, 1:1 + Sq, 2:2 + H * G]                      # queries sliced out of something larger
    out, lse = qad.attn_fwd_cache_prefix(q, c.gpu(), c.table[B].cuda(), P, _roomy(c)[:B].cuda(), ints(lens), causal=causal,
                                         return_lse=True)
    _check(out, lse, q.cpu(), c, causal, prefix=B)


def _ramp(lens, H, Sq, G, span, seed):
    """Scores that rise along the sequence, by `span` in all: the softmax's reference moves again and again."""
    c = Cache(lens, H, 64, seed=seed)
    g = torch.Generator().manual_seed(seed)
    u = torch.where(torch.rand(D, generator=g) < 0.5, 1.0, -1.0)
    for b, n in enumerate(lens):
        t = torch.linspace(-0.5, 0.5, n)[:, None, None] if n > 1 else torch.zeros((n, 1, 1))
        k = u * (t * span / math.sqrt(D)) + 0.05 * torch.randn((n, H, D), generator=g)
        v = torch.randn((n, H, D), generator=g)
        codes = quantize_kv(k.to(torch.bfloat16), v.to(torch.bfloat16))
        c.put(b, codes)
        c.rows[b] = codes
    q = (u + 0.05 * torch.randn((len(lens), Sq, H * G, D), generator=g)).to(torch.bfloat16)
    return c, q


@pytest.mark.parametrize("Sq,G", [(20, 2), (50, 5)])
@pytest.mark.parametrize("span", [40.0, 400.0, -400.0, 20000.0])
def test_rising_and_falling_scores(Sq, G, span):
    import quantized_attention_diffusion_gb300 as qad
    lens = [1300, 77]
    c, q = _ramp(lens, 2, Sq, G, span, seed=int(abs(span)) + Sq)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints(lens), return_lse=True)
    _check(out, lse, q, c, True)


V_SCALES = [
    ("one far larger value row", lambda n, g: torch.where(torch.arange(n) == n // 2, 2.0 ** 30, 1.0)[:, None, None]),
    ("tiny values", lambda n, g: torch.full((n, 1, 1), 2.0 ** -100)),
    ("large values", lambda n, g: torch.full((n, 1, 1), 2.0 ** 100)),
    ("some rows of zeros", lambda n, g: (torch.rand((n, 1, 1), generator=g) < 0.3).float()),
    ("all zeros", lambda n, g: torch.zeros((n, 1, 1))),
    ("scales spread over 2^-40 .. 2^40", lambda n, g: 2.0 ** (80 * torch.rand((n, 1, 1), generator=g) - 40)),
]


@pytest.mark.parametrize("Sq", [40, 140])
@pytest.mark.parametrize("name,f", V_SCALES)
def test_scales_of_v_of_any_size(name, f, Sq):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([500, 150], 2, 32, seed=3, v_scale=f)
    q = _q(2, Sq, 2, seed=4)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints([500, 150]), return_lse=True)
    _check(out, lse, q, c, True, what=name)


@pytest.mark.parametrize("mul", [2.0 ** -120, 2.0 ** -60, 2.0 ** 40, 0.0])
def test_queries_of_any_size(mul):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([300], 1, 32, seed=8)
    q = _q(1, 37, 2, seed=9, mul=mul)
    scale = SCALE * (2.0 ** -40 if mul > 1 else 1.0)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints([300]), softmax_scale=scale, return_lse=True)
    _check(out, lse, q, c, True, scale=scale)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("Sq", [60, 200])
def test_a_row_that_is_not_finite_reaches_only_what_sees_it(Sq, value):
    import quantized_attention_diffusion_gb300 as qad
    lens, H = [350, 290], 2
    c = Cache(lens, H, 32, seed=10)
    q = _q(2, Sq, 4, seed=11)
    clean, clean_lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints(lens), return_lse=True)
    at = 350 - 20             # seen by the last twenty queries of sequence 0
    p, o = int(c.table[0, at // 32]), at % 32
    for which in ("k", "v", "both"):
        gpu = c.gpu()
        if which != "v":
            gpu[1][p, 1, o] = value
        if which != "k":
            gpu[3][p, 1, o] = value
            gpu[2].view(torch.uint8)[p, 1, o] = 0           # as the cache has such a row
        out, lse = qad.attn_fwd_cache(q.cuda(), gpu, _roomy(c).cuda(), ints(lens), return_lse=True)
        if which != "k" or math.isnan(value):
            assert torch.isnan(out[0, Sq - 20:, 2:]).all(), which
        assert torch.equal(bits(out[0, :Sq - 20]), bits(clean[0, :Sq - 20])), which
        assert torch.equal(bits(out[0, :, :2]), bits(clean[0, :, :2])) and torch.equal(bits(out[1]), bits(clean[1])), which
        assert torch.equal(bits(lse[0, :2]), bits(clean_lse[0, :2])) and torch.equal(bits(lse[1]), bits(clean_lse[1])), which


def test_scores_beyond_fp32_end_and_stay_in_their_rows():
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([400], 1, 32, seed=12)
    q = _q(1, 50, 1, seed=13)
    clean = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints([400]))
    q[0, 7] = q[0, 7] * 2.0 ** 126
    out = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints([400]))
    rest = [i for i in range(50) if i != 7]
    ro, _, to, _ = reference(q[0, rest].contiguous(), c.dense(0), False, SCALE)
    full = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c).cuda(), ints([400]), causal=False)
    assert_within(full[0, rest], ro, to)
    assert torch.allclose(out[0, rest].float(), clean[0, rest].float(), rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.parametrize("Sq", [40, 150])
def test_bad_pages_are_reported_and_reach_nothing_else(Sq):
    import quantized_attention_diffusion_gb300 as qad
    bad_page = 8
    lens = [200, 400, 300]
    c = Cache(lens, 2, 32, seed=20, extra=[170])
    q = _q(3, Sq, 2, seed=21)
    table = _roomy(c)
    table[1, 1] = c.num_pages
    table[1, 2] = -5
    table[1, 9] = -2 ** 31
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), table[:3].cuda(), ints(lens), return_lse=True)
    assert qad.sync_status() == bad_page and qad.sync_status() == 0
    for b in (0, 2):
        ro, rl, to, tl = reference(q[b], c.dense(b), True, SCALE)
        assert_within(out[b], ro, to)
        assert_within(lse[b], rl, tl)
    assert torch.isfinite(out).all()
    # A bad page of the prefix.
    pre = c.table[3].clone()
    pre[4] = 2 ** 31 - 1
    qad.attn_fwd_cache_prefix(q.cuda(), c.gpu(), pre.cuda(), 170, _roomy(c)[:3].cuda(), ints(lens))
    assert qad.sync_status() == bad_page
    qad.attn_fwd_cache_prefix(q.cuda(), c.gpu(), pre.cuda(), 128, _roomy(c)[:3].cuda(), ints(lens))   # not reached
    assert qad.sync_status() == 0


def test_the_workspace_ends_where_it_says_and_the_cache_is_only_read():
    import quantized_attention_diffusion_gb300 as qad
    lens, Sq, H, G = [700, 300, 0], 50, 2, 4
    c = Cache(lens, H, 64, seed=30, extra=[500])
    q = _q(3, Sq, H * G, seed=31).cuda()
    gpu = c.gpu()
    before = [bits(t) for t in gpu]
    for prefix in (0, 500):
        need = qad.attn_fwd_cache_workspace_bytes(3, Sq, H * G, H, prefix)
        buf = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        out = torch.full((4, Sq, H * G, D), -7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, H * G, Sq), -7.0, device="cuda")
        kw = dict(out=out[:3], lse=lse[:3], workspace=buf[:need])
        if prefix:
            qad.attn_fwd_cache_prefix(q, gpu, c.table[3].cuda(), prefix, _roomy(c)[:3].cuda(), ints(lens), **kw)
        else:
            qad.attn_fwd_cache(q, gpu, _roomy(c)[:3].cuda(), ints(lens), **kw)
        assert (buf[need:] == 0x5A).all() and (out[3] == -7).all() and (lse[3] == -7).all()
        _check(out[:3], lse[:3], q.cpu(), c, True, prefix=3 if prefix else None)
    for a, b in zip(before, gpu):
        assert torch.equal(a, bits(b))


def test_codes_of_v_as_bytes_and_pages_that_sequences_share():
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([320], 2, 64, seed=32)
    kc, ks, vc, vs = c.gpu()
    table = _roomy(c).cuda().expand(3, -1)                   # one table for three sequences
    lens = [320, 100, 64]
    for Sq in (1, 40):
        q = _q(3, Sq, 4, seed=33 + Sq).cuda()
        a = qad.attn_fwd_cache(q, (kc, ks, vc, vs), table, ints(lens))
        b = qad.attn_fwd_cache(q, (kc, ks, vc.view(torch.uint8), vs), table.contiguous(), ints(lens))
        assert torch.equal(bits(a), bits(b))
        for i, n in enumerate(lens):
            rows = tuple(t[:n] for t in c.dense(0))
            ro, _, to, _ = reference(q[i].cpu(), rows, True, SCALE)
            assert_within(a[i], ro, to)


def test_captured_and_replayed_on_another_stream():
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([900, 300], 2, 64, seed=34, extra=[400])
    q = _q(2, 80, 4, seed=35).cuda()
    gpu, table, pre = c.gpu(), _roomy(c)[:2].cuda(), c.table[2].cuda()
    first, second = ints([900, 300]), ints([80, 0])
    want = [(bits(qad.attn_fwd_cache(q, gpu, table, n)), bits(qad.attn_fwd_cache_prefix(q, gpu, pre, 400, table, n)))
            for n in (first, second)]
    n = first.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a = qad.attn_fwd_cache(q, gpu, table, n)
        b = qad.attn_fwd_cache_prefix(q, gpu, pre, 400, table, n)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        for i, lens in enumerate((second, first, second)):
            n.copy_(lens)
            g.replay()
            got = (bits(a), bits(b))
            k = 0 if lens is first else 1
            assert torch.equal(got[0], want[k][0]) and torch.equal(got[1], want[k][1])
