"""Ragged batches of 17 to 128 query rows to a key/value head over roomy tables, whose
CTAs get short segments and long ones in turn, against float64; and the sizes on either
side of 16 rows, where one kernel hands over to the other."""
import math

import pytest
import torch

from tests.cache_common import D, Cache, assert_within, ints, reference
from tests.cache_split import RAGGED, ragged_lens
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


def _q(B, Sq, Hq, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((B, Sq, Hq, D), generator=g).to(torch.bfloat16)


def _roomy(c):
    """The cache's table with room for far more keys than clusters of CTAs take."""
    width = -(-20000 // c.page)
    return torch.nn.functional.pad(c.table, (0, max(0, width - c.table.shape[1])), value=-1).cuda()


def _spread(n, g):
    """V's scales over 2^-12 .. 2^12: weights with another tile's scales are far off."""
    return 2.0 ** (24 * torch.rand((n, 1, 1), generator=g) - 12)


@pytest.mark.parametrize("B,longest,Sq,H,G,seed", RAGGED)
def test_ragged_batches(B, longest, Sq, H, G, seed):
    import quantized_attention_diffusion_gb300 as qad
    lens = ragged_lens(B, longest, seed)
    c = Cache(lens, H, 64, seed=seed, v_scale=_spread)
    q = _q(B, Sq, H * G, seed=seed + 1)
    gpu, table, n, qd = c.gpu(), _roomy(c), ints(lens), q.cuda()
    out, lse = qad.attn_fwd_cache(qd, gpu, table, n, return_lse=True)
    first = bits(out)
    for b in range(B):
        ro, rl, to, tl = reference(q[b], c.dense(b), True, SCALE)
        assert_within(out[b], ro, to, f"out[{b}]")
        assert_within(lse[b], rl, tl, f"lse[{b}]")
    again = torch.empty_like(out)
    for _ in range(100):
        qad.attn_fwd_cache(qd, gpu, table, n, out=again)
        assert torch.equal(again, out)
    assert torch.equal(bits(again), first)


@pytest.mark.parametrize("Sq,G", [(8, 2), (16, 1), (17, 1), (4, 4), (6, 4), (31, 1), (32, 1), (4, 8), (33, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_either_side_of_sixteen_rows(Sq, G, causal):
    import quantized_attention_diffusion_gb300 as qad
    lens, H = [900, 1, 128, 0, 300, 129, 64], 3
    c = Cache(lens, H, 32, seed=Sq + G, recipe="sharp")
    q = _q(len(lens), Sq, H * G, seed=Sq)
    out, lse = qad.attn_fwd_cache(q.cuda(), c.gpu(), _roomy(c), ints(lens), causal=causal, return_lse=True)
    for b in range(len(lens)):
        ro, rl, to, tl = reference(q[b], c.dense(b), causal, SCALE)
        assert_within(out[b], ro, to, f"out[{b}]")
        assert_within(lse[b], rl, tl, f"lse[{b}]")
