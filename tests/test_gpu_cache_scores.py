"""Scores near the ends of fp32's range, on every path of the attention over the KV cache."""
import math

import pytest
import torch

from tests.cache_common import D, ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu


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


# Sq, G, positions that the table has room for, prefix
PATHS = [(1, 2, 320, 0), (1, 2, 20032, 0), (3, 4, 20032, 0), (40, 1, 20032, 0), (40, 5, 20032, 0), (1, 2, 320, 130),
         (1, 2, 20032, 130), (50, 1, 20032, 130), (1, 2, 320, 9000)]


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("power", [90, 110, 124])
@pytest.mark.parametrize("Sq,G,room,prefix", PATHS)
def test_equal_scores_of_any_size(Sq, G, room, prefix, power, sign):
    """Scores of sign 2^power: all equal, a row's output is the mean of V; one key half as
    far from zero (or the others), it is that key's V.  V is +-1 by channel and key, so that
    sums of n <= 9320 are exact and only the mean's reciprocal and bf16 round."""
    import quantized_attention_diffusion_gb300 as qad
    H, page, n = 2, 64, 300
    B, total = 2, prefix + n
    g = torch.Generator().manual_seed(power + Sq)
    k = torch.zeros((1, total, H, D))
    k[..., 0] = 2.0 ** 50
    v = torch.where(torch.rand((1, total, H, D), generator=g) < 0.25, 1.0, -1.0)
    q = torch.zeros((B, Sq, H * G, D), dtype=torch.bfloat16)
    q[..., 0] = sign * 2.0 ** (power - 50)
    pages = -(-prefix // page) + -(-n // page)
    cache = qad.kv_cache_alloc(pages, H, page)
    ids = torch.arange(pages, dtype=torch.int32)
    first = -(-prefix // page)
    own = torch.nn.functional.pad(ids[first:], (0, room // page - (pages - first)), value=-1).expand(B, -1).contiguous().cuda()
    lens = ints([n] * B)

    def attend(which):
        x = k.clone()
        if which is not None:                   # the largest score is that key's alone
            x[:, which, :, 0] *= 0.5 if sign < 0 else 2.0
        for at, rows in ((ids[:first], slice(0, prefix)), (ids[first:], slice(prefix, total))):
            if at.numel():
                qad.kv_cache_write(x[:, rows].to(torch.bfloat16).cuda(), v[:, rows].to(torch.bfloat16).cuda(), cache,
                                   at.view(1, -1).cuda(), ints([0]))
        kw = dict(softmax_scale=0.5, causal=False, return_lse=True)
        if prefix:
            return qad.attn_fwd_cache_prefix(q.cuda(), cache, ids[:first].cuda(), prefix, own, lens, **kw)
        return qad.attn_fwd_cache(q.cuda(), cache, own, lens, **kw)

    def each(x):                                # [H, D] for the query heads
        return x.repeat_interleave(G, dim=0)

    out, lse = attend(None)
    want = each(v[0].double().mean(0))
    assert float((out.double().cpu() - want).abs().max()) <= 2.0 ** -8      # 2^-9 of at most 1, and V's scale 1/448
    assert float((lse.double().cpu() / (sign * 2.0 ** (power - 1)) - 1).abs().max()) <= 2.0 ** -20
    for which in (total - 3, 1, prefix + 70):
        out, _ = attend(which)
        assert float((out.double().cpu() - each(v[0, which].double())).abs().max()) <= 2.0 ** -8, which


@pytest.mark.parametrize("Sq,G,room", [p[:3] for p in PATHS if p[3] == 0])
def test_a_sequence_without_keys_and_one_of_far_scores(Sq, G, room):
    """Next to scores of -2^124 a row that sees nothing stays a row of zeros and -inf."""
    import quantized_attention_diffusion_gb300 as qad
    H, page = 1, 64
    cache = qad.kv_cache_alloc(5, H, page)
    k = torch.zeros((1, 300, H, D), dtype=torch.bfloat16)
    k[..., 0] = 2.0 ** 60
    qad.kv_cache_write(k.cuda(), torch.ones_like(k).cuda(), cache, ints(range(5)).view(1, 5), ints([0]))
    q = torch.zeros((3, Sq, G, D), dtype=torch.bfloat16)
    q[..., 0] = -2.0 ** 65
    table = torch.nn.functional.pad(torch.arange(5, dtype=torch.int32), (0, room // page - 5), value=-1).expand(3, -1).contiguous()
    out, lse = qad.attn_fwd_cache(q.cuda(), cache, table.cuda(), ints([0, 300, 1]), softmax_scale=0.5, causal=False, return_lse=True)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all()
    assert (out[1:] - 1).abs().max() <= 2.0 ** -8 and torch.isfinite(lse[1:]).all()
