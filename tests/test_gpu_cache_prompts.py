"""A padded batch of prompts of unequal lengths, written and attended to together: the
write has a sequence's tokens at the front of its row, the attention its queries at the end."""
import math

import pytest
import torch

from tests.cache_common import D, assert_within, ints, quantize_kv, reference
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_library()


@pytest.mark.parametrize("room", [512, 20032])
@pytest.mark.parametrize("before,count", [([0, 0, 0, 0], [40, 1, 17, 0]), ([70, 0, 3, 129], [5, 33, 40, 1]), ([0, 9], [9, 9])])
def test_prompts_of_unequal_lengths(before, count, room):
    import quantized_attention_diffusion_gb300 as qad
    B, S, H, G, page = len(count), max(count), 2, 2, 64
    g = torch.Generator().manual_seed(sum(count) + B)

    def normal(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    cache = qad.kv_cache_alloc(4 * B, H, page)
    table = torch.randperm(4 * B, generator=g).to(torch.int32).view(B, 4)
    table = torch.nn.functional.pad(table, (0, room // page - 4), value=-1).cuda()
    old = max(before)
    if old:
        ko, vo = normal(B, old, H, D), normal(B, old, H, D)
        qad.kv_cache_write(ko.cuda(), vo.cuda(), cache, table, ints([0] * B), ints(before))
    k, v, q = normal(B, S, H, D), normal(B, S, H, D), normal(B, S, H * G, D)      # tokens at the front of each row
    qad.kv_cache_write(k.cuda(), v.cuda(), cache, table, ints(before), ints(count))
    # The queries at the end: row i of sequence b is its token i - (S - count[b]).
    at = torch.arange(S)[None, :] - (S - torch.tensor(count))[:, None]
    behind = torch.gather(q, 1, at.clamp(min=0)[:, :, None, None].expand(-1, -1, H * G, D))
    lens = [a + c for a, c in zip(before, count)]
    out, lse = qad.attn_fwd_cache(behind.cuda(), cache, table, ints(lens), return_lse=True)
    assert qad.sync_status() == 0
    for b, c in enumerate(count):
        if c == 0:
            continue
        kb, vb = (torch.cat([o[b, :before[b]], x[b, :c]]) if old else x[b, :c] for o, x in ((ko if old else None, k), (vo if old else None, v)))
        kc, ks, vc, vs = quantize_kv(kb, vb)
        ro, rl, to, tl = reference(q[b, :c], (kc.double(), ks.double(), vc.float().double(), vs.double()), True, SCALE)
        assert_within(out[b, S - c:], ro, to, f"out[{b}]")
        assert_within(lse[b, :, S - c:], rl, tl, f"lse[{b}]")
