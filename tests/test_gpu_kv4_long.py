"""Long tails behind a few heavy keys, and the longest sequences, over a 4-bit cache."""
import math

import pytest
import torch

from tests.cache_common import D, ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
PAGE, SINKS = 64, 64
LONGEST = 1 << 30


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


# B, Sq, H, G, keys, positions that the table has room for.  So many sequences and
# heads that a CTA has whole sequences: its own first keys are the largest.
PATHS = [
    ("clusters", 8, 1, 2, 4, 4096, 4096), ("few rows", 200, 1, 5, 4, 4096, 20480), ("sixteen rows", 160, 4, 5, 4, 4096, 20480),
    ("many rows", 100, 10, 4, 4, 8192, 20480), ("row tiles", 100, 50, 4, 4, 8192, 20480),
]


@pytest.mark.parametrize("below,bits", [(0, 10.0), (0, 18.7), (0, 22.0), (4, 10.0), (4, 18.7), (4, 22.0), (5, 26.0), (10, 20.6), (10, 32.0), (16, 38.0)])
@pytest.mark.parametrize("name,B,Sq,H,G,keys,room", PATHS)
def test_the_sum_of_a_long_tail(name, B, Sq, H, G, keys, room, below, bits):
    """All sequences read the same two pages again and again: SINKS keys whose scores
    are `bits` above the others', in units of log2, and whose V, in channel 0, is 2^-below of
    what the other keys have in the other channels.  There the output is n c / (n + SINKS 2^bits).

    Bound, relative: half a bf16 step, 2^-8; a weight's rounding to fp16, 2^-11, or
    2^-25 where it is subnormal, of a weight of at least 2^(5 - bits) while the two may count
    with one scale of V (up to 2^4 apart), 2^(5 + below - bits) otherwise; scores: 130
    roundings of 2^-23 of their size; sums in fp32: 16 products at a time, at most
    64 tiles and 16 parts, 2^-23 each; exponentials 2^-21."""
    import quantized_attention_diffusion_gb300 as qad
    k = torch.zeros((1, 2 * PAGE, H, D))
    v = torch.zeros((1, 2 * PAGE, H, D))
    k[:, :PAGE, :, 0] = 6.75                              # held exactly, as 0.75 and its powers of two
    k[:, PAGE:, :, 1] = 6.75
    v[:, :PAGE, :, 0] = 0.75 * 2.0 ** -below
    v[:, PAGE:, :, 1:] = 0.75
    cache = qad.kv_cache_alloc(2, H, PAGE, bits=4)
    pages = ints([0, 1]).view(1, 2)
    qad.kv_cache_write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, pages, ints([0]))
    back = qad.kv_cache_read(cache, pages, ints([2 * PAGE]), 2 * PAGE)
    assert torch.equal(back[0].float().cpu(), k) and torch.equal(back[1].float().cpu(), v)
    q = torch.zeros((B, Sq, H * G, D), dtype=torch.bfloat16)
    q[..., 0] = 2.0
    scale = torch.tensor(bits * math.log(2) / (2 * 6.75), dtype=torch.float32).item()
    table = torch.ones((B, room // PAGE), dtype=torch.int32)
    table[:, :SINKS // PAGE] = 0
    out, lse = qad.attn_fwd_cache(q.cuda(), cache, table.cuda(), ints([keys] * B), softmax_scale=scale, causal=False, return_lse=True)
    n, s = keys - SINKS, math.exp(2 * 6.75 * scale)
    got = out.double().cpu()
    least = bits - (below if below > 4 else 0)
    tol = 2.0 ** -8 + max(2.0 ** -11, 2.0 ** (-25 - 5 + least)) + 2 * 130 * 2.0 ** -23 * bits + (16 + 64 + 16) * 2.0 ** -23 + 2.0 ** -21
    worst = float((got[..., 1:] / (n * 0.75 / (n + SINKS * s)) - 1).abs().max())
    assert worst <= tol, f"{name}: the tail's sum is {worst:.5f} off, bound {tol:.5f}"
    sink = 0.75 * 2.0 ** -below * SINKS * s / (n + SINKS * s)
    assert float((got[..., 0] / sink - 1).abs().max()) <= tol
    assert float((lse.double().cpu() - math.log(n + SINKS * s)).abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("Sq,G", [(2, 1), (20, 1)])
def test_the_longest_sequence_behind_the_longest_prefix(Sq, G):
    """One page of equal keys, again and again: out is V, and lse the number of keys, whose
    weights of 1 add up exactly.  With many rows (over 16) a CTA of 152 adds 16 keys at a time,
    and the tensor core cuts each sum off at 24 bits, 2^-23 of it, so that its N additions are
    off by N 2^-23 at most."""
    import quantized_attention_diffusion_gb300 as qad
    cache = qad.kv_cache_alloc(1, 1, 256, bits=4)
    v = torch.where(torch.arange(D) % 3 == 0, -0.75, 0.75).to(torch.bfloat16)
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
