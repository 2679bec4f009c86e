"""Lengths that the page table does not reach, for each path of the attention over the
KV cache: reported, and the other sequences right."""
import math

import pytest
import torch

from tests.cache_common import D, Cache, assert_within, ints, join, reference
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)
OK, BAD_PAGE = 0, 8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    import quantized_attention_diffusion_gb300 as qad
    yield
    assert qad.sync_status() == OK


def bits(t):
    return t.cpu().contiguous().view(torch.uint8)


# clusters of CTAs, few rows and many: Sq, G, positions that the table has room for
PATHS = [(1, 4, 512), (1, 4, 20032), (4, 4, 20032), (40, 2, 20032), (150, 1, 20032)]


def _setup(Sq, G, room, H=2, page=64, prefix=0):
    lens = [200, 300, 90]
    c = Cache(lens, H, page, seed=Sq + G, extra=[prefix] if prefix else [])
    table = c.table[:3].clone()
    # the last sequence's row leads to its first page again and again: all of it is in the cache
    width = room // page
    table = torch.nn.functional.pad(table, (0, width - table.shape[1]), value=-1)
    table[2] = int(table[2, 0])
    g = torch.Generator().manual_seed(Sq)
    q = torch.randn((3, Sq, H * G, D), generator=g).to(torch.bfloat16)
    return c, table, q, lens


@pytest.mark.parametrize("Sq,G,room", PATHS)
@pytest.mark.parametrize("prefix", [0, 150])
@pytest.mark.parametrize("causal", [True, False])
def test_a_length_behind_the_table_is_reported(Sq, G, room, prefix, causal):
    import quantized_attention_diffusion_gb300 as qad
    c, table, q, lens = _setup(Sq, G, room, prefix=prefix)

    def call(last):
        n = ints(lens[:2] + [last])
        if not prefix:
            return qad.attn_fwd_cache(q.cuda(), c.gpu(), table.cuda(), n, causal=causal, return_lse=True)
        return qad.attn_fwd_cache_prefix(q.cuda(), c.gpu(), c.table[3].cuda(), prefix, table.cuda(), n, causal=causal, return_lse=True)

    for last, status in ((room, OK), (room + 1, BAD_PAGE), (2 * room, BAD_PAGE), ((1 << 30) - 1, BAD_PAGE), (90, OK)):
        out, lse = call(last)
        assert qad.sync_status() == status, last
        for b in range(2):
            rows = join(c.dense(3), c.dense(b)) if prefix else c.dense(b)
            ro, rl, to, tl = reference(q[b], rows, causal, SCALE)
            assert_within(out[b], ro, to, f"{last} out[{b}]")
            assert_within(lse[b], rl, tl, f"{last} lse[{b}]")


@pytest.mark.parametrize("Sq,G,room", PATHS)
def test_the_largest_length_means_the_whole_table(Sq, G, room):
    import quantized_attention_diffusion_gb300 as qad
    c, table, q, lens = _setup(Sq, G, room)
    want = None
    for last in (room, 1 << 30, (1 << 31) - 1):
        got = qad.attn_fwd_cache(q.cuda(), c.gpu(), table.cuda(), ints(lens[:2] + [last]))
        assert qad.sync_status() == OK
        want = bits(got) if want is None else want
        assert torch.equal(bits(got), want)
