"""Calls over a 4-bit cache and around it that the first tests do not make: many
sequences, slices, far scales, lengths behind the table, streams and graphs, large tensors."""
import math

import pytest
import torch

from tests.cache_common import D, assert_within, ints, reference
from tests.gpu_common import ensure_library
from tests.kv4_common import Cache4, quantize4, values4

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


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def check(cache, q, out, lse, causal, rows=None, lens=None):
    for b in range(q.shape[0]):
        ref, z, tol, ltol = reference(q[b].cpu(), (rows or cache.dense)(b), causal, SCALE)
        assert_within(out[b], ref, tol, f"out of sequence {b}")
        assert_within(lse[b], z, ltol, f"lse of sequence {b}")


@pytest.mark.parametrize("B,Sq,Hq,H,longest", [(300, 1, 4, 1, 400), (300, 9, 2, 1, 150), (257, 40, 1, 1, 90), (520, 2, 8, 2, 70)])
def test_more_sequences_than_a_launch_takes(B, Sq, Hq, H, longest):
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, longest + 1, (B,), generator=g).tolist()
    cache = Cache4(lens, H, 16, seed=B, width=64)          # room for 1024 keys: too much for clusters
    q = randn(B, B, Sq, Hq, D)
    out, lse = qad.attn_fwd_cache(q.cuda(), cache.gpu(), cache.table.cuda(), ints(lens), return_lse=True)
    check(cache, q, out, lse, True)


@pytest.mark.parametrize("Sq", [1, 50])
def test_slices_of_a_projection_and_of_a_table(Sq):
    import quantized_attention_diffusion_gb300 as qad
    lens = [333, 70]
    cache = Cache4(lens, 2, 32, seed=3)
    qkv = randn(4, 2, Sq + 3, 12, D).cuda()
    q = qkv[:, 2:Sq + 2, 3:11]
    wide = torch.full((2, cache.table.shape[1] + 5), 7777777, dtype=torch.int32)
    wide[:, :cache.table.shape[1]] = cache.table
    table = wide.cuda()[:, :cache.table.shape[1]]
    out, lse = qad.attn_fwd_cache(q, cache.gpu(), table, ints(lens), return_lse=True)
    check(cache, q, out, lse, True)


def far(n, g):
    return torch.exp2(torch.randint(-25, 26, (n, 1, 1), generator=g).float())


def near(n, g):       # within 2^14 of one another: the wide kernel moves the differences into the values
    s = torch.exp2(torch.randint(-6, 7, (n, 1, 1), generator=g).float())
    return torch.where(torch.rand((n, 1, 1), generator=g) < 0.1, torch.zeros(()), s)


@pytest.mark.parametrize("Sq", [1, 5, 70])
@pytest.mark.parametrize("k_scale,v_scale", [(None, near), (near, None), (near, near), (None, far)])
def test_rows_of_unlike_size(Sq, k_scale, v_scale):
    import quantized_attention_diffusion_gb300 as qad
    lens = [700, 129]
    cache = Cache4(lens, 2, 64, seed=Sq, k_scale=k_scale, v_scale=v_scale)
    q = (0.05 * torch.randn((2, Sq, 4, D), generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    out, lse = qad.attn_fwd_cache(q.cuda(), cache.gpu(), cache.table.cuda(), ints(lens), return_lse=True)
    check(cache, q, out, lse, True)


@pytest.mark.parametrize("Sq", [1, 70])
def test_scales_that_are_no_powers_of_two(Sq):
    """Not what the quantiser writes, but a cache that somebody else has filled."""
    import quantized_attention_diffusion_gb300 as qad
    lens = [500, 64]
    cache = Cache4(lens, 2, 64, seed=Sq)
    gpu = list(cache.gpu())
    gpu[2], gpu[5] = gpu[2] * 1.37, gpu[5] * 0.71

    def rows(b):
        kc, ks, vc, vs = cache.dense(b)
        return kc, (ks.float() * 1.37).double(), vc, (vs.float() * 0.71).double()

    q = randn(5, 2, Sq, 4, D)
    out, lse = qad.attn_fwd_cache(q.cuda(), tuple(gpu), cache.table.cuda(), ints(lens), return_lse=True)
    check(cache, q, out, lse, True, rows)


@pytest.mark.parametrize("Sq", [1, 60])
def test_lengths_behind_the_table(Sq):
    import quantized_attention_diffusion_gb300 as qad
    cache = Cache4([64, 100], 1, 16, seed=9, width=7)
    gpu, table = cache.gpu(), cache.table.cuda()
    table[0, 4:] = table[1, 4:]                      # 112 positions of pages that there are
    q = randn(6, 2, Sq, 2, D)
    got = qad.attn_fwd_cache(q.cuda(), gpu, table, ints([113, 100]))
    assert qad.sync_status() == 8
    ref, _, tol, _ = reference(q[1], cache.dense(1), True, SCALE)
    assert_within(got[1], ref, tol)
    full = qad.attn_fwd_cache(q.cuda()[:1], gpu, table[:1], ints([112]), causal=False)
    for n in (2 ** 30, 2 ** 31 - 1):
        assert torch.equal(qad.attn_fwd_cache(q.cuda()[:1], gpu, table[:1], ints([n]), causal=False).isnan(), full.isnan())
    assert qad.sync_status() == 0


def test_append_and_rotation_recorded_replayed_and_on_another_stream():
    import quantized_attention_diffusion_gb300 as qad
    T, Hq, H = 37, 6, 2
    rope = qad.Rope(96, interleaved=True)
    x = randn(7, 1, T, Hq + 2 * H, D).cuda()
    q, k, v = x.split([Hq, H, H], dim=2)
    cache, other = (qad.kv_cache_alloc(5, H, 16, bits=4) for _ in range(2))
    slots, pos = ints(range(T)), ints(range(T))
    out = torch.empty((1, T, Hq, D), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qad.kv_cache_append(q, k, v, cache, slots, rope, pos, eps=1e-6, out=out)
    side = torch.cuda.Stream()
    for step in range(3):
        x.copy_(randn(step, *x.shape))
        slots.copy_(torch.randperm(80, generator=torch.Generator().manual_seed(step))[:T].to(torch.int32))
        pos.add_(1000 * step)
        for c in cache + other:
            c.view(torch.uint8).zero_()
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = qad.kv_cache_append(q, k, v, other, slots, rope, pos, eps=1e-6)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)
        for a, b in zip(cache, other):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_tensors_of_more_than_2_31_elements():
    import quantized_attention_diffusion_gb300 as qad
    T, H = 180000, 96
    x = torch.empty((1, T, H, D), dtype=torch.bfloat16, device="cuda")
    tail = randn(8, 1, 64, H, D).cuda()
    x[:, -64:] = tail
    x[:, :64] = tail.flip(1)
    rope = qad.Rope(128)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    got = qad.qk_norm_rope(x, None, rope, pos, eps=1e-6, out=x)
    assert got is x
    assert torch.equal(got[:, -64:], qad.qk_norm_rope(tail, None, rope, pos[-64:].contiguous(), eps=1e-6))
    assert torch.equal(got[:, :64], qad.qk_norm_rope(tail.flip(1), None, rope, pos[:64].contiguous(), eps=1e-6))


def test_a_generation_step_of_two_requests_that_share_pages():
    """A forked request: the second reads the first's pages and goes on in its own."""
    import quantized_attention_diffusion_gb300 as qad
    H, page = 2, 16
    cache = qad.kv_cache_alloc(6, H, page, bits=4)
    x = randn(11, 1, 20, 2 * H, D).cuda()
    k, v = x.split([H, H], dim=2)
    table = ints([3, 1, 3, 5]).view(2, 2)
    qad.kv_cache_append(None, k[:, :18], v[:, :18], cache, ints([3 * page + i for i in range(16)] + [page, page + 1]))
    for i, s in enumerate((page + 2, 5 * page)):          # the first's token 18, the second's 16
        qad.kv_cache_append(None, k[:, 18 + i:19 + i], v[:, 18 + i:19 + i], cache, ints([s]))
    q = randn(12, 2, 1, 4, D)
    out = qad.attn_fwd_cache(q.cuda(), cache, table, ints([19, 17]))
    for b, rows in enumerate((list(range(19)), list(range(16)) + [19])):
        kk, vv = k[0, rows].cpu(), v[0, rows].cpu()
        kc, kb, ks = quantize4(kk)
        vc, vb, vs = quantize4(vv)
        ref, _, tol, _ = reference(q[b], (values4(kc, kb), ks.double(), values4(vc, vb), vs.double()), True, SCALE)
        assert_within(out[b], ref, tol)


@pytest.mark.parametrize("B,H,prefix", [(60, 8, 3000), (40, 8, 3000), (80, 8, 2500)])
def test_many_sequences_behind_a_prefix(B, H, prefix):
    """A unit for each sequence and head: more than fit an SM three at a time, fewer, and
    more than fit four at a time."""
    import quantized_attention_diffusion_gb300 as qad
    from tests.cache_common import join
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 90, (B,), generator=g).tolist()
    cache = Cache4(lens, H, 16, seed=B, extra=(prefix,))
    q = randn(B, B, 1, 2 * H, D)
    table = cache.table.cuda()
    width = max(1, -(-max(lens) // 16))
    out, lse = qad.attn_fwd_cache_prefix(q.cuda(), cache.gpu(), table[B, :-(-prefix // 16)].contiguous(), prefix,
                                         table[:B, :width].contiguous(), ints(lens), return_lse=True)
    check(cache, q, out, lse, True, lambda b: join(cache.dense(B), cache.dense(b)))
