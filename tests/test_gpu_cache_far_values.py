"""Rows of V whose sizes lie as far apart as fp32's range in one sequence, under scores that
leave most of them without weight: 8 and 4 bits, against float64."""
import math

import pytest
import torch

from tests.cache_common import Cache, D, assert_within, ints, join, reference
from tests.gpu_common import ensure_library
from tests.kv4_common import Cache4

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


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("low,high", [(-125, 100), (-60, 100), (-125, -20)])
@pytest.mark.parametrize("scale", [1.0 / math.sqrt(D), 1.0, 40.0])
@pytest.mark.parametrize("lens,Sq,G,prefix", [([294], 33, 2, 0), ([130], 33, 5, 1500), ([0, 1503, 2422, 1], 60, 1, 0), ([20000], 33, 1, 0), ([40], 20, 1, 20000),
                                             ([1503, 20], 2, 2, 0), ([70], 1, 4, 300)])
def test_values_of_any_size_side_by_side(lens, Sq, G, prefix, scale, low, high, bits):
    import quantized_attention_diffusion_gb300 as qad
    B, H, page = len(lens), 2, 32

    def sizes(n, g):
        return torch.exp2(torch.randint(low, high, (n, 1, 1), generator=g).float())

    cache = (Cache if bits == 8 else Cache4)(lens, H, page, seed=Sq + high, v_scale=sizes, extra=(prefix,) if prefix else ())
    q = torch.randn((B, Sq, H * G, D), generator=torch.Generator().manual_seed(Sq)).to(torch.bfloat16)
    table = cache.table.cuda()
    kw = dict(softmax_scale=scale, causal=False, return_lse=True)
    if prefix:
        out, lse = qad.attn_fwd_cache_prefix(q.cuda(), cache.gpu(), table[B, :-(-prefix // page)].contiguous(), prefix, table[:B].contiguous(), ints(lens), **kw)
    else:
        out, lse = qad.attn_fwd_cache(q.cuda(), cache.gpu(), table, ints(lens), **kw)
    for b in range(B):
        rows = join(cache.dense(B), cache.dense(b)) if prefix else cache.dense(b)
        ref, z, tol, ltol = reference(q[b], rows, False, scale)
        # below 2^-126 bf16's steps are 2^-133 whatever the value: half of one
        assert_within(out[b], ref, tol + 2.0 ** -134, f"out of sequence {b}")
        assert_within(lse[b], z, ltol, f"lse of sequence {b}")
