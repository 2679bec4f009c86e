"""The longest prefix and the longest sequence behind it: 2^31 positions in all."""
import math

import pytest
import torch

from tests.cache_common import D, ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
LONGEST = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_library()


@pytest.mark.parametrize("Sq,G", [(2, 1), (20, 1)])
def test_the_longest_sequence_behind_the_longest_prefix(Sq, G):
    """One page of equal keys, again and again: out is V, and lse the number of keys, whose
    weights of 1 add up exactly.  The sums of V: with few rows 2^8 times a code, exact too;
    with many (over 16) a CTA of 152 adds 16 keys at a time, and the tensor core cuts each
    sum off at 24 bits, 2^-23 of it, so that its N additions are off by N 2^-23 at most."""
    import quantized_attention_diffusion_gb300 as qad
    cache = qad.kv_cache_alloc(1, 1, 256)
    v = torch.where(torch.arange(D) % 3 == 0, -1.0, 1.0).to(torch.bfloat16)
    qad.kv_cache_write(torch.zeros((1, 256, 1, D), dtype=torch.bfloat16, device="cuda"), v.cuda().expand(1, 256, 1, D).contiguous(),
                       cache, ints([0]).view(1, 1), ints([0]))
    q = torch.ones((1, Sq, G, D), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((1, LONGEST // 256), dtype=torch.int32, device="cuda")
    for prefix, length in ((LONGEST, LONGEST), (LONGEST, 0), (5, LONGEST), (LONGEST, 1)):
        out, lse = qad.attn_fwd_cache_prefix(q, cache, table[0], prefix, table, ints([length]), return_lse=True)
        assert qad.sync_status() == 0
        cut = 0.0 if Sq * G <= 16 else max(prefix, length) / (152 * 16) * 2.0 ** -23
        assert float((out.double().cpu() - v.double()).abs().max()) <= 2.0 ** -8 + cut
        seen = [math.log(prefix + length - Sq + 1 + i) for i in range(Sq)]
        assert float((lse.double().cpu() - torch.tensor(seen, dtype=torch.float64)).abs().max()) <= 2.0 ** -18   # 21.5: 2^-20 a rounding
