"""The quantised KV cache on the GPU: writing (bit for bit against the stated
quantiser), reading back, and the attention over it against float64 within
bounds that count its roundings."""
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
    qad.debug_inject_fault(qad.FAULT_NONE)
    assert qad.sync_status() == 0


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


# ----------------------------------------------------------------- write --

def _marked(num_pages, H, page):
    """A cache whose every byte is 0xA5."""
    import quantized_attention_diffusion_gb300 as qad
    cache = qad.kv_cache_alloc(num_pages, H, page)
    for t in cache:
        t.view(torch.uint8).fill_(0xA5)
    return cache


def _put(want, codes, p, o, b, i):
    for dst, src in zip(want, codes):
        if dst.dtype == torch.float32:
            dst[p, :, o] = src[b, i]
        else:
            dst.view(torch.uint8)[p, :, o] = src[b, i].view(torch.uint8)


def _expected(cache, table, start, count, k, v):
    want = [t.cpu().clone() for t in cache]
    page = want[0].shape[2]
    codes = quantize_kv(k, v)
    for b in range(k.shape[0]):
        for i in range(count[b]):
            p, o = int(table[b, (start[b] + i) // page]), (start[b] + i) % page
            _put(want, codes, p, o, b, i)
    return want


def _assert_cache(cache, want):
    for name, got, ref in zip(("k_codes", "k_scale", "v_codes", "v_scale"), cache, want):
        # a NaN scale may have any NaN's bits
        if got.dtype == torch.float32:
            got, ref = got.cpu(), ref
            same = (got.view(torch.int32) == ref.view(torch.int32)) | (torch.isnan(got) & torch.isnan(ref))
            assert same.all(), name
        else:
            assert torch.equal(bits(got), bits(ref)), name


@pytest.mark.parametrize("B,S,H,page,start,count", [
    (1, 1, 1, 16, [0], None),
    (3, 1, 2, 16, [15, 16, 47], None),
    (2, 37, 3, 32, [0, 5], [37, 0]),
    (4, 70, 5, 64, [1, 63, 64, 0], [70, 1, 33, 99]),
    (2, 300, 7, 128, [200, 3], None),
    (1, 700, 64, 256, [100], None),      # more rows than one per warp
])
def test_write_is_bit_exact_and_touches_nothing_else(B, S, H, page, start, count):
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(B * 1000 + S)
    k = (torch.randn((B, S, H, D), generator=g) * torch.randn((B, S, H, 1), generator=g).exp()).to(torch.bfloat16)
    v = torch.randn((B, S, H, D), generator=g).to(torch.bfloat16)
    width = max(-(-(s + S) // page) for s in start) + 1
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width)
    cache = _marked(B * width, H, page)
    live = [S] * B if count is None else [min(S, c) for c in count]
    want = _expected(cache, table, start, live, k, v)
    got = qad.kv_cache_write(k.cuda(), v.cuda(), cache, table.cuda(), ints(start), None if count is None else ints(count))
    assert got is cache
    _assert_cache(cache, want)


def test_write_takes_slices_of_a_projection():
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(5)
    B, S, H = 2, 19, 3
    qkv = torch.randn((B, S + 2, 3 * H, D), generator=g).to(torch.bfloat16).cuda()
    k, v = qkv[:, 1:S + 1, H:2 * H], qkv[:, 2:, 2 * H:]
    table = torch.tensor([[3, 0], [1, 2]], dtype=torch.int32)
    cache = _marked(4, H, 16)
    want = _expected(cache, table, [0, 7], [S, S], k.cpu(), v.cpu())
    qad.kv_cache_write(k, v, cache, table.cuda(), ints([0, 7]))
    _assert_cache(cache, want)


def test_write_of_special_rows():
    """Zeros (both signs), subnormals, the largest magnitudes, one infinity, one NaN."""
    import quantized_attention_diffusion_gb300 as qad
    S, H = 64, 2
    g = torch.Generator().manual_seed(6)
    x = torch.randn((1, S, H, D), generator=g)
    for i, f in enumerate((0.0, -0.0, 2.0 ** -133, 2.0 ** -126, 2.0 ** -120, 2.0 ** -100, 2.0 ** -92, 2.0 ** 100, 2.0 ** 125)):
        x[0, i] *= f
    x[0, 20, 0, 7] = math.inf
    x[0, 21, 1, 127] = -math.inf
    x[0, 22, 0, 0] = math.nan
    x[0, 23, 1] = math.nan
    x[0, 24, 0, 5] = 3.3895e38
    x[0, 25] = 1.0            # ties of the quotient
    x[0, 26] = (torch.arange(128) - 64.0) / 2
    x[0, 26, :, 0] = 63.5
    k = x.to(torch.bfloat16)
    v = x.flip(1).to(torch.bfloat16)
    table = torch.tensor([[1, 3, 2, 0]], dtype=torch.int32)
    cache = _marked(4, H, 16)
    want = _expected(cache, table, [0], [S], k, v)
    qad.kv_cache_write(k.cuda(), v.cuda(), cache, table.cuda(), ints([0]))
    _assert_cache(cache, want)
    kr, vr = qad.kv_cache_read(cache, table.cuda(), ints([S]), S)
    assert torch.isnan(kr[0, 20, 0]).all() and torch.isfinite(kr[0, 20, 1]).all()
    assert torch.isnan(vr[0, S - 1 - 22, 0]).all() and (kr[0, 0] == 0).all()


# ------------------------------------------------------------------ read --

@pytest.mark.parametrize("lens,H,page,S", [
    ([1], 1, 16, 1), ([0, 5, 16], 2, 16, 17), ([300, 64, 1, 0], 3, 64, 300), ([129, 500], 5, 128, 400), ([1100], 24, 256, 1100),
])
def test_read_is_the_codes_times_the_scales(lens, H, page, S):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=sum(lens) + H)
    out = tuple(torch.full((len(lens), S, H, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = qad.kv_cache_read(c.gpu(), c.table.cuda(), ints(lens), S, out=out)
    assert k is out[0]
    for b, n in enumerate(lens):
        kc, ks, vc, vs = c.rows[b]
        n = min(n, S)
        wk = (kc.float() * ks[..., None]).to(torch.bfloat16)[:n]
        wv = (vc.float() * vs[..., None]).to(torch.bfloat16)[:n]
        assert torch.equal(bits(k[b, :n]), bits(wk)) and torch.equal(bits(v[b, :n]), bits(wv))
        assert (k[b, n:] == 0).all() and (v[b, n:] == 0).all()


# ------------------------------------------------------------- attention --

def _q(B, Sq, Hq, seed, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, Sq, Hq, D), generator=g) * mul).to(torch.bfloat16)


def _roomy(table, page):
    """The table with room for far more keys: the work is cut up over all CTAs
    whatever the lengths, where a narrow table lets clusters of CTAs take a unit each."""
    width = -(-20000 // page)
    return torch.nn.functional.pad(table, (0, max(0, width - table.shape[1])), value=-1)


def _check(out, lse, q, c, causal, scale=SCALE, prefix=None, what=""):
    for b in range(q.shape[0]):
        rows = c.dense(b) if prefix is None else join(c.dense(prefix), c.dense(b))
        ro, rl, to, tl = reference(q[b], rows, causal, scale)
        assert_within(out[b], ro, to, f"{what} out[{b}]")
        if lse is not None:
            assert_within(lse[b], rl, tl, f"{what} lse[{b}]")


STEP = [
    # lens, H, G, page
    ([1], 1, 1, 16), ([16], 1, 4, 16), ([63, 64, 65], 2, 1, 16), ([0, 1, 2, 700], 3, 5, 32),
    ([129, 1000, 0], 2, 8, 64), ([777], 8, 4, 16), ([2000, 3, 513], 4, 16, 128), ([4099], 1, 3, 256), ([300] * 9, 2, 7, 64),
]


@pytest.mark.parametrize("lens,H,G,page", STEP)
@pytest.mark.parametrize("recipe", ["normal", "sharp"])
def test_one_token(lens, H, G, page, recipe):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=len(lens) * 7 + G, recipe=recipe)
    q = _q(len(lens), 1, H * G, seed=G)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints(lens), return_lse=True)
    _check(out, lse, q, c, True)
    plain = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints(lens), causal=False)
    assert torch.equal(bits(plain), bits(out))          # one token sees everything either way


CHUNK = [
    # lens, Sq, H, G, page
    ([5], 5, 1, 1, 16), ([70, 3, 0, 64], 5, 2, 1, 16), ([200, 17], 17, 1, 1, 32), ([100, 1000], 33, 2, 3, 64),
    ([70, 5], 8, 2, 4, 16), ([1300], 16, 1, 2, 64), ([300, 129], 129, 1, 1, 16), ([640, 257], 64, 2, 4, 32), ([1100], 257, 2, 1, 16),
    ([260], 130, 1, 4, 128), ([90, 512, 300], 70, 2, 2, 256), ([1500], 9, 4, 7, 64),
]


@pytest.mark.parametrize("lens,Sq,H,G,page", CHUNK)
@pytest.mark.parametrize("causal", [True, False])
def test_chunks(lens, Sq, H, G, page, causal):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=Sq, recipe="offset")
    q = _q(len(lens), Sq, H * G, seed=Sq + 1)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints(lens), causal=causal, return_lse=True)
    _check(out, lse, q, c, causal)


PREFIX = [
    # prefix, lens, Sq, H, G, page
    (1, [0], 1, 1, 1, 16), (16, [1, 0], 1, 2, 4, 16), (63, [5, 70, 0], 1, 2, 3, 16), (200, [1, 2, 90, 300], 5, 1, 2, 64),
    (1001, [33] * 7, 1, 4, 8, 32), (130, [0, 1, 2, 8], 6, 3, 1, 128), (700, [3, 600], 3, 2, 5, 256), (64, [1] * 40, 1, 1, 7, 64),
]


@pytest.mark.parametrize("P,lens,Sq,H,G,page", PREFIX)
@pytest.mark.parametrize("causal", [True, False])
def test_shared_prefix(P, lens, Sq, H, G, page, causal):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=P, extra=[P], recipe="offset")
    B = len(lens)
    q = _q(B, Sq, H * G, seed=P + 1)
    out, lse = qad.attn_fwd_cache_prefix(q.cuda(), c.gpu(), c.table[B].cuda(), P, c.table[:B].cuda(), ints(lens),
                                         causal=causal, return_lse=True)
    _check(out, lse, q, c, causal, prefix=B)


@pytest.mark.parametrize("lens,Sq,H,G,page", [(n, 1, H, G, page) for n, H, G, page in STEP] + CHUNK[:6])
def test_room_does_not_matter(lens, Sq, H, G, page):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=Sq + G, recipe="sharp")
    q = _q(len(lens), Sq, H * G, seed=G + 1)
    for table in (c.table, _roomy(c.table, page)):
        out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), table.cuda(), ints(lens), return_lse=True)
        _check(out, lse, q, c, True)


@pytest.mark.parametrize("P,lens,Sq,H,G,page", PREFIX + [(2000, [5], 4, 2, 8, 16), (65, [63, 64, 65, 0], 2, 2, 4, 128), (1999, [48], 1, 1, 1, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_room_does_not_matter_behind_a_prefix(P, lens, Sq, H, G, page, causal):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache(lens, H, page, seed=P, extra=[P], recipe="sharp")
    B = len(lens)
    q = _q(B, Sq, H * G, seed=P + 2)
    for table in (c.table, _roomy(c.table, page)):
        out, lse = qad.attn_fwd_cache_prefix(q.cuda(), c.gpu(), table[B, :-(-P // page)].cuda(), P, table[:B].cuda(), ints(lens),
                                             causal=causal, return_lse=True)
        _check(out, lse, q, c, causal, prefix=B)


LONG = [
    # prefix, lens, Sq, H, G, page: more of a prefix than clusters take, little room behind it
    (9000, [5, 0, 63], 1, 10, 1, 64), (9000, [64, 1], 1, 8, 8, 128), (9001, [3, 70, 0, 9] * 3, 1, 4, 4, 16), (8300, [7, 2, 20], 3, 8, 5, 32),
]


@pytest.mark.parametrize("P,lens,Sq,H,G,page", LONG)
@pytest.mark.parametrize("causal", [True, False])
def test_joined_behind_a_long_prefix(P, lens, Sq, H, G, page, causal):
    import quantized_attention_diffusion_gb300 as qad
    B = len(lens)
    c = Cache(lens, H, page, seed=P + Sq, extra=[P], recipe="sharp")
    q = _q(B, Sq, H * G, seed=P + 2).cuda()
    gpu, pre, own = c.gpu(), c.table[B].cuda(), c.table[:B, :-(-max(lens) // page)].contiguous().cuda()
    need = qad.attn_fwd_cache_workspace_bytes(B, Sq, H * G, H, P)
    buf = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    out, lse = qad.attn_fwd_cache_prefix(q, gpu, pre, P, own, ints(lens), causal=causal, return_lse=True, workspace=buf[:need])
    _check(out, lse, q.cpu(), c, causal, prefix=B)
    assert (buf[need:] == 0x5A).all()
    n, none = ints(lens), torch.zeros(B, dtype=torch.int32, device="cuda")
    want = bits(qad.attn_fwd_cache_prefix(q, gpu, pre, P, own, none, causal=causal))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = qad.attn_fwd_cache_prefix(q, gpu, pre, P, own, n, causal=causal)
    g.replay()
    assert torch.equal(bits(again), bits(out))
    n.zero_()
    g.replay()
    assert torch.equal(bits(again), want)


def test_softmax_scale_and_large_scores():
    """Scores of hundreds: weights of one key only, and the running maximum's path."""
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([1300], 2, 64, seed=1, recipe="sharp")
    q = _q(1, 2, 8, seed=2, mul=20.0)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints([1300]), softmax_scale=0.5, return_lse=True)
    _check(out, lse, q, c, True, scale=0.5)


@pytest.mark.parametrize("name,f", [
    ("one far larger value row", lambda n, g: torch.where(torch.arange(n) == n // 2, 2.0 ** 30, 1.0)[:, None, None]),
    ("tiny values", lambda n, g: torch.full((n, 1, 1), 2.0 ** -100)),
    ("large values", lambda n, g: torch.full((n, 1, 1), 2.0 ** 60)),
    ("some rows of zeros", lambda n, g: (torch.rand((n, 1, 1), generator=g) < 0.3).float()),
    ("all zeros", lambda n, g: torch.zeros((n, 1, 1))),
    ("scales spread over 2^-40 .. 2^40", lambda n, g: 2.0 ** (80 * torch.rand((n, 1, 1), generator=g) - 40)),
])
def test_scales_of_v_of_any_size(name, f):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([500, 77], 2, 32, seed=3, v_scale=f)
    q = _q(2, 1, 8, seed=4)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints([500, 77]), return_lse=True)
    _check(out, lse, q, c, True, what=name)


@pytest.mark.parametrize("mul", [2.0 ** -120, 2.0 ** -60, 2.0 ** 40, 0.0])
def test_queries_of_any_size(mul):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([300], 1, 32, seed=8)
    q = _q(1, 3, 2, seed=9, mul=mul)
    scale = SCALE * (2.0 ** -40 if mul > 1 else 1.0)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints([300]), softmax_scale=scale, return_lse=True)
    _check(out, lse, q, c, True, scale=scale)


def test_a_nan_row_reaches_only_what_sees_it():
    """A NaN token in a chunk: earlier queries of the same chunk, other heads and
    other sequences stay as they were; queries that see it are NaN."""
    import quantized_attention_diffusion_gb300 as qad
    lens, Sq, H = [150, 90], 12, 2
    c = Cache(lens, H, 32, seed=10)
    q = _q(2, Sq, 4, seed=11)
    clean, clean_lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints(lens), return_lse=True)
    at = 150 - 4              # seen by the last four queries of sequence 0
    p, o = int(c.table[0, at // 32]), at % 32
    for which in ("k", "v", "both"):
        gpu = c.gpu()
        if which != "v":
            gpu[1][p, 1, o] = math.nan
        if which != "k":
            gpu[3][p, 1, o] = math.nan
        out, lse = qad.attn_fwd_cache(q.cuda(), gpu, c.table.cuda(), ints(lens), return_lse=True)
        assert torch.isnan(out[0, Sq - 4:, 2:]).all(), which
        assert torch.equal(bits(out[0, :Sq - 4]), bits(clean[0, :Sq - 4])), which
        assert torch.equal(bits(out[0, :, :2]), bits(clean[0, :, :2])) and torch.equal(bits(out[1]), bits(clean[1])), which
        assert torch.equal(bits(lse[0, :2]), bits(clean_lse[0, :2])) and torch.equal(bits(lse[1]), bits(clean_lse[1])), which


def test_queries_may_be_slices_and_outputs_given():
    import quantized_attention_diffusion_gb300 as qad
    lens, H, G = [100, 900], 2, 4
    c = Cache(lens, H, 64, seed=12)
    wide = _q(2, 5, 16, seed=13).cuda()
    q = wide[:, 1:4, 4:12]
    out = torch.full((2, 3, 8, D), math.nan, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 8, 3), math.nan, device="cuda")
    ws = torch.full((qad.attn_fwd_cache_workspace_bytes(2, 3, 8, 2),), 0xFF, dtype=torch.uint8, device="cuda")
    table = torch.full((2, 40), -7, dtype=torch.int32, device="cuda")     # rows of a wider table
    table[:, 3:3 + c.table.shape[1]] = c.table.cuda()
    got = qad.attn_fwd_cache(q, c.gpu(), table[:, 3:3 + c.table.shape[1]], ints(lens), out=out, lse=lse, workspace=ws)
    assert got[0] is out and got[1] is lse
    _check(out, lse, q.cpu(), c, True)
    again = qad.attn_fwd_cache(q.contiguous(), c.gpu(), c.table.cuda(), ints(lens))
    assert torch.equal(bits(again), bits(out))


def test_results_do_not_depend_on_the_run():
    import quantized_attention_diffusion_gb300 as qad
    lens = [3000, 10, 1500]
    c = Cache(lens, 2, 64, seed=14)
    q = _q(3, 1, 8, seed=15).cuda()
    gpu, table, n = c.gpu(), c.table.cuda(), ints(lens)
    first = bits(qad.attn_fwd_cache(q, gpu, table, n))
    for _ in range(5):
        assert torch.equal(bits(qad.attn_fwd_cache(q, gpu, table, n)), first)


def test_more_sequences_than_one_launch_takes():
    import quantized_attention_diffusion_gb300 as qad
    B = 1100
    lens = [(i * 37) % 50 for i in range(B)]
    c = Cache(lens, 1, 16, seed=16, extra=[70])
    q = _q(B, 1, 2, seed=17)
    gpu = c.gpu()
    for table in (c.table[:B].cuda(), _roomy(c.table[:B], 16).cuda()):
        out, lse = qad.attn_fwd_cache(q.cuda(), gpu, table, ints(lens), return_lse=True)
        _check(out, lse, q, c, True)
        out, lse = qad.attn_fwd_cache_prefix(q.cuda(), gpu, c.table[B].cuda(), 70, table, ints(lens), return_lse=True)
        _check(out, lse, q, c, True, prefix=B)


def test_pages_behind_four_gigabytes():
    """Codes whose byte offsets pass 2^32 and rows whose numbers pass 2^25."""
    import quantized_attention_diffusion_gb300 as qad
    page, H, pages = 256, 2, 80000
    cache = qad.kv_cache_alloc(pages, H, page)       # 5.2 GB of codes each
    g = torch.Generator().manual_seed(18)
    n = 600
    k = torch.randn((1, n, H, D), generator=g).to(torch.bfloat16)
    v = torch.randn((1, n, H, D), generator=g).to(torch.bfloat16)
    table = ints([pages - 1, 70001, pages - 2]).view(1, 3)
    qad.kv_cache_write(k.cuda(), v.cuda(), cache, table, ints([0]))
    codes = quantize_kv(k, v)
    kr, vr = qad.kv_cache_read(cache, table, ints([n]), n)
    assert torch.equal(bits(kr), bits((codes[0].float() * codes[1][..., None]).to(torch.bfloat16)))
    assert torch.equal(bits(vr), bits((codes[2].float() * codes[3][..., None]).to(torch.bfloat16)))
    rows = (codes[0][0].double(), codes[1][0].double(), codes[2][0].float().double(), codes[3][0].double())
    for Sq in (1, 5, 40):
        q = _q(1, Sq, 4, seed=19 + Sq)
        ro, rl, to, tl = reference(q[0], rows, True, SCALE)
        for t in (table, _roomy(table, page)):
            out, lse = qad.attn_fwd_cache(q.cuda(), cache, t, ints([n]), return_lse=True)
            assert_within(out[0], ro, to)
            assert_within(lse[0], rl, tl)
        new = ints([70001]).view(1, 1)                      # the prefix's pages, and one behind
        codes_at = tuple(torch.cat([x, x[page:2 * page]]) for x in rows)
        ro, rl, to, tl = reference(q[0], codes_at, False, SCALE)
        for t in (new, _roomy(new, page)):
            out, lse = qad.attn_fwd_cache_prefix(q.cuda(), cache, table[0], n, t, ints([page]), causal=False, return_lse=True)
            assert_within(out[0], ro, to)
            assert_within(lse[0], rl, tl)


# ---------------------------------------------------- bad pages, streams --

def test_pages_outside_the_cache_are_reported_and_reach_nothing_else():
    import quantized_attention_diffusion_gb300 as qad
    bad_page = 8
    lens = [200, 100, 300]
    c = Cache(lens, 2, 32, seed=20)
    q = _q(3, 1, 8, seed=21)
    table = c.table.clone()
    table[1, 1] = c.num_pages
    table[1, 2] = -5
    for tab in (table, _roomy(table, 32)):
        out = qad.attn_fwd_cache(q.cuda(), c.gpu(), tab.cuda(), ints(lens))
        assert qad.sync_status() == bad_page and qad.sync_status() == 0
        for b in (0, 2):
            ro, _, to, _ = reference(q[b], c.dense(b), True, SCALE)
            assert_within(out[b], ro, to)
        pre = torch.tensor([c.num_pages + 5, int(c.table[2, 0])], dtype=torch.int32)
        qad.attn_fwd_cache_prefix(q.cuda(), c.gpu(), pre.cuda(), 40, _roomy(c.table, 32).cuda() if tab is not table else c.table.cuda(), ints(lens))
        assert qad.sync_status() == bad_page and qad.sync_status() == 0
    k, v = qad.kv_cache_read(c.gpu(), table.cuda(), ints(lens), 300)
    assert qad.sync_status() == bad_page
    assert (k[1, 32:96] == 0).all() and torch.isfinite(k).all() and torch.isfinite(v).all()
    assert (k[1, 96:100] != 0).any() and (k[1, :32] != 0).any()
    # A write behind the table, before its beginning and into bad pages.
    cache = _marked(c.num_pages, 2, 32)
    kv = [_q(3, 40, 2, seed=s) for s in (22, 23)]
    wide = torch.tensor([[0, 1, 2], [c.num_pages, 3, 4], [5, -1, 6]], dtype=torch.int32)
    start = [70, -3, 0]
    want = [t.cpu().clone() for t in cache]
    codes = quantize_kv(*kv)
    for b in range(3):
        for i in range(40):
            pos = start[b] + i
            if 0 <= pos < 96 and 0 <= wide[b, pos // 32] < c.num_pages:
                _put(want, codes, int(wide[b, pos // 32]), pos % 32, b, i)
    qad.kv_cache_write(kv[0].cuda(), kv[1].cuda(), cache, wide.cuda(), ints(start))
    assert qad.sync_status() == bad_page
    _assert_cache(cache, want)
    # Lengths behind the table are cut to it.
    out = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints([200, 100, 1 << 30]), causal=False)
    for b in (0, 1):
        ro, _, to, _ = reference(q[b], c.dense(b), False, SCALE)
        assert_within(out[b], ro, to)


def test_negative_lengths_are_empty():
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([40, 40], 1, 16, seed=24)
    q = _q(2, 3, 2, seed=25)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), c.table.cuda(), ints([-9, 40]), return_lse=True)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    ro, rl, to, tl = reference(q[1], c.dense(1), True, SCALE)
    assert_within(out[1], ro, to)
    k, _ = qad.kv_cache_read(c.gpu(), c.table.cuda(), ints([-9, 40]), 40)
    assert (k[0] == 0).all() and (k[1] != 0).any()


@pytest.mark.parametrize("room", ["little", "much"])
def test_two_streams_and_a_graph_that_follows_the_lengths(room):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([500, 900], 2, 64, seed=26, extra=[300])
    q = _q(2, 1, 8, seed=27).cuda()
    gpu, table, pre = c.gpu(), c.table[:2].cuda(), c.table[2].cuda()
    if room == "much":
        table = _roomy(table, 64)
    short, long = ints([100, 3]), ints([500, 900])
    want = [(bits(qad.attn_fwd_cache(q, gpu, table, n)), bits(qad.attn_fwd_cache_prefix(q, gpu, pre, 300, table, n)))
            for n in (short, long)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            n = (short, long)[i // 2 % 2]
            outs.append((i // 2 % 2, qad.attn_fwd_cache(q, gpu, table, n), qad.attn_fwd_cache_prefix(q, gpu, pre, 300, table, n)))
    torch.cuda.synchronize()
    for i, a, b in outs:
        assert torch.equal(bits(a), want[i][0]) and torch.equal(bits(b), want[i][1])
    n = short.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a = qad.attn_fwd_cache(q, gpu, table, n)
            b = qad.attn_fwd_cache_prefix(q, gpu, pre, 300, table, n)
        graphs.append((g, a, b))
    for i, lens in enumerate((long, short, long)):
        n.copy_(lens)
        for g, _, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, a, b in graphs:
            k = 1 if lens is long else 0
            assert torch.equal(bits(a), want[k][0]) and torch.equal(bits(b), want[k][1])


@pytest.mark.parametrize("site", ["FAULT_POOL_ALLOC", "FAULT_ATTN_LAUNCH"])
def test_injected_failures_leave_the_next_call_right(site):
    import quantized_attention_diffusion_gb300 as qad
    c = Cache([300], 1, 32, seed=28, width=1000)             # room for more than one launch of clusters takes
    q = _q(1, 1, 4, seed=29).cuda()
    args = (q, c.gpu(), c.table.cuda(), ints([300]))
    want = bits(qad.attn_fwd_cache(*args))
    torch.cuda.synchronize()
    _, used = qad.debug_pool_state()
    qad.debug_inject_fault(getattr(qad, site))
    with pytest.raises(qad.SageError, match="injected fault"):
        qad.attn_fwd_cache(*args)
    torch.cuda.synchronize()
    assert qad.debug_pool_state()[1] == used
    assert torch.equal(bits(qad.attn_fwd_cache(*args)), want)
    qad.debug_inject_fault(qad.FAULT_QUANT_LAUNCH)
    with pytest.raises(qad.SageError, match="injected fault"):
        qad.kv_cache_read(args[1], args[2], args[3], 300)


# ------------------------------------------------------- a run of all four --

def test_a_prompt_its_continuations_and_back():
    """A shared prompt is written once, four sequences continue it token by
    token; every step's attention is checked, then the cache is read back and
    attended to through attn_fwd_cross."""
    import quantized_attention_diffusion_gb300 as qad
    B, H, G, page, P, steps = 4, 2, 3, 16, 53, 20
    g = torch.Generator().manual_seed(30)

    def normal(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    cache = _marked(4 + 2 * B, H, page)
    prefix = ints([9, 2, 5, 7])
    table = torch.tensor([[0, 1], [3, 4], [6, 8], [10, 11]], dtype=torch.int32).cuda()
    kp, vp = normal(1, P, H, D), normal(1, P, H, D)
    qad.kv_cache_write(kp.cuda(), vp.cuda(), cache, prefix.view(1, 4), ints([0]))
    rows = [quantize_kv(kp[0], vp[0])] * B
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        q, k, v = normal(B, 1, H * G, D), normal(B, 1, H, D), normal(B, 1, H, D)
        qad.kv_cache_write(k.cuda(), v.cuda(), cache, table, lens)
        lens += 1
        out, lse = qad.attn_fwd_cache_prefix(q.cuda(), cache, prefix, P, table, lens, return_lse=True)
        joined = torch.cat([prefix[:3].expand(B, 3), table], 1).contiguous()
        for b in range(B):
            new = quantize_kv(k[b], v[b])
            rows[b] = tuple(torch.cat([x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x,
                                       y.view(torch.uint8) if y.dtype == torch.float8_e4m3fn else y]) for x, y in zip(rows[b], new))
            kc, ks, vc, vs = rows[b]
            dense = (kc.double(), ks.double(), vc.view(torch.float8_e4m3fn).float().double(), vs.double())
            ro, rl, to, tl = reference(q[b], dense, True, SCALE)
            assert_within(out[b], ro, to)
            assert_within(lse[b], rl, tl)
    assert joined.shape == (B, 5)
    kb, vb = qad.kv_cache_read(cache, table, lens, steps)
    alone, _ = qad.attn_fwd_cache(q.cuda(), cache, table, lens, return_lse=True)
    kg, vg = (t.repeat_interleave(G, dim=2).contiguous() for t in (kb, vb))
    cross = qad.attn_fwd_cross(q.cuda(), kg, vg)
    # both approximate the same attention: E4M3 weights and a second quantisation on the one side
    assert torch.nn.functional.cosine_similarity(cross.float().flatten(), alone.float().flatten(), dim=0) > 0.99
