"""A long tail of keys behind a few that take nearly all the weight: the tail's sum has
to be right although each of its weights is far below the largest, on every path of the
attention over the KV cache."""
import math

import pytest
import torch

from tests.cache_common import D, ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
PAGE, SINKS = 256, 512


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


@pytest.mark.parametrize("bits", [10.0, 16.3, 18.7, 20.6, 22.0])
@pytest.mark.parametrize("name,B,Sq,H,G,keys,room", PATHS)
def test_the_sum_of_a_long_tail(name, B, Sq, H, G, keys, room, bits):
    """All sequences read the same two pages again and again: SINKS keys whose scores
    are `bits` above the others', in units of log2, with V in channel 0; then keys with
    the same V in the other channels.  There the output is n c / (n + SINKS 2^bits).

    Bound, relative: half a bf16 step, 2^-8; a weight's rounding to fp16, 2^-11, or
    2^-25 where it is subnormal, of a weight of at least 2^(5 - bits); scores: 130
    roundings of 2^-23 of their size; sums in fp32: 16 products at a time, at most
    64 tiles and 16 parts, 2^-23 each; exponentials 2^-21."""
    import quantized_attention_diffusion_gb300 as qad
    k = torch.zeros((1, 2 * PAGE, H, D))
    v = torch.zeros((1, 2 * PAGE, H, D))
    k[:, :PAGE, :, 0] = 4.0
    k[:, PAGE:, :, 1] = 4.0
    v[:, :PAGE, :, 0] = 1.0
    v[:, PAGE:, :, 1:] = 1.0
    cache = qad.kv_cache_alloc(2, H, PAGE)
    qad.kv_cache_write(k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda(), cache, ints([0, 1]).view(1, 2), ints([0]))
    kb, vb = (t.double().cpu() for t in qad.kv_cache_read(cache, ints([0, 1]).view(1, 2), ints([2 * PAGE]), 2 * PAGE))
    k0 = float(cache[0][0, 0, 0, 0]) * float(cache[1][0, 0, 0])      # the sinks' K in channel 0
    v0 = float(cache[2][1, 0, 0, 1].float()) * float(cache[3][1, 0, 0])
    assert abs(k0 / 4 - 1) < 2.0 ** -22 and abs(v0 - 1) < 2.0 ** -22 and kb[0, PAGE, 0, 0] == 0 and vb[0, 0, 0, 1] == 0
    q = torch.zeros((B, Sq, H * G, D), dtype=torch.bfloat16)
    q[..., 0] = 2.0
    scale = torch.tensor(bits * math.log(2) / (2 * k0), dtype=torch.float32).item()
    table = torch.ones((B, room // PAGE), dtype=torch.int32)
    table[:, :SINKS // PAGE] = 0
    out, lse = qad.attn_fwd_cache(q.cuda(), cache, table.cuda(), ints([keys] * B), softmax_scale=scale, causal=False, return_lse=True)
    n, s = keys - SINKS, math.exp(2 * k0 * scale)
    got = out.double().cpu()
    tol = (2.0 ** -8 + max(2.0 ** -11, 2.0 ** (-25 - 5 + bits)) + 2 * 130 * 2.0 ** -23 * bits + (16 + 64 + 16) * 2.0 ** -23 + 2.0 ** -21)
    want = n * v0 / (n + SINKS * s)
    worst = float((got[..., 1:] / want - 1).abs().max())
    assert worst <= tol, f"{name}: the tail's sum is {worst:.5f} off, bound {tol:.5f}"
    sink = SINKS * s / (n + SINKS * s)
    assert float((got[..., 0] / sink - 1).abs().max()) <= tol
    assert float((lse.double().cpu() - math.log(n + SINKS * s)).abs().max()) <= 2.0 ** -16
