"""Scores of any size over a 4-bit cache, on every path of the attention."""
import math

import pytest
import torch

from tests.cache_common import D, assert_within, ints, join, reference
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


# B, Sq, G, H, own keys, positions that the table has room for, prefix.  Many rows, one key
# tile for a CTA and several, up to 128 rows and more; a prefix for itself; few rows.
WIDE = [(2, 40, 1, 2, 300, 20032, 0), (2, 40, 5, 2, 300, 20032, 0), (4, 40, 1, 4, 5000, 20032, 0), (4, 40, 5, 4, 5000, 20032, 0),
        (2, 50, 1, 2, 300, 20032, 130), (8, 6, 2, 2, 70, 320, 9000)]
PATHS = [(2, 1, 2, 2, 300, 320, 0), (2, 1, 2, 2, 300, 20032, 0), (2, 3, 4, 2, 300, 20032, 0), (2, 1, 2, 2, 300, 320, 130)] + WIDE
PAGE = 64
ODD = 6.75        # code 6 times the block scale 9/8: times any power of two, held exactly in 4 bits


class Keys:
    """B sequences with the same n own keys behind the same prefix, no key seen by some
    rows alone: k and v float64 [prefix + n, H, 128] that 4 bits hold exactly."""

    def __init__(self, path, k, v):
        import quantized_attention_diffusion_gb300 as qad
        B, _, _, H, n, room, prefix = path
        first, own = -(-prefix // PAGE), -(-n // PAGE)
        self.cache = qad.kv_cache_alloc(first + own, H, PAGE, bits=4)
        ids = torch.arange(first + own, dtype=torch.int32)
        self.prefix = ids[:first].cuda()
        self.table = torch.nn.functional.pad(ids[first:], (0, room // PAGE - own), value=-1).expand(B, -1).contiguous().cuda()
        self.lens, self.length = ints([n] * B), prefix
        for at, rows in ((ids[:first], slice(0, prefix)), (ids[first:], slice(prefix, prefix + n))):
            if at.numel():
                x, y = (t[None, rows].to(torch.bfloat16).cuda() for t in (k, v))
                table, start = at.view(1, -1).cuda(), ints([0])
                qad.kv_cache_write(x, y, self.cache, table, start)
                back = qad.kv_cache_read(self.cache, table, ints([x.shape[1]]), x.shape[1])
                assert torch.equal(back[0], x) and torch.equal(back[1], y)

    def attend(self, q):
        import quantized_attention_diffusion_gb300 as qad
        kw = dict(softmax_scale=0.5, causal=False, return_lse=True)
        if self.length:
            return qad.attn_fwd_cache_prefix(q, self.cache, self.prefix, self.length, self.table, self.lens, **kw)
        return qad.attn_fwd_cache(q, self.cache, self.table, self.lens, **kw)


def signs(path, seed, size):
    """V of +-size by key and channel."""
    B, Sq, G, H, n, room, prefix = path
    g = torch.Generator().manual_seed(seed)
    return torch.where(torch.rand((prefix + n, H, D), generator=g) < 0.25, size, -size).double()


def queries(path, channel, value):
    B, Sq, G, H = path[:4]
    q = torch.zeros((B, Sq, H * G, D), dtype=torch.bfloat16)
    q[..., channel] = value
    return q.cuda()


def assert_out(out, want, G, size, what):
    """bf16 is off by 2^-8 of the value at the most, a weight's fp16 by 2^-11 of V's size;
    two roundings of scores of less than 2^13 differ by 2^-12 (in log2), those of larger ones
    are the same for equal keys; the tensor cores cut the sums of n < 2^14 keys off at
    n / 16 2^-23 < 2^-13."""
    want = want.repeat_interleave(G, dim=0)
    tol = 2.0 ** -8 * want.abs() + size * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -13)
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"{what}: {float((err - tol).max())} above the bound"


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("power", [3, 11, 12, 14, 18, 22, 24, 26, 27, 28, 31, 40, 90, 120])
@pytest.mark.parametrize("size", [0.75, 1.5, 1.5 * 2.0 ** -16])
@pytest.mark.parametrize("path", PATHS)
def test_equal_scores_of_any_size(path, size, power, sign):
    """Scores of about sign 2^power, with odd significands on both sides: where all are
    equal, a row's output is the mean of V; with one key half as far from zero (or all others)
    it is that key's V.  (V's scales are 2^-11, 2^-10 and 2^-26: a reference stands that far and
    6 below the largest score, which fp32 has or has not room for.)"""
    G, H, n, prefix = path[2], path[3], path[4], path[6]
    total = prefix + n
    half = power // 2
    k = torch.zeros((total, H, D), dtype=torch.float64)
    k[..., 0] = ODD * 2.0 ** half
    v = signs(path, power, size)
    q = queries(path, 0, 1.0)
    row = torch.arange(q.shape[1] * q.shape[2]).view(q.shape[1:3]) % 64
    keys = Keys(path, k, v)
    # eight significant bits, unlike in each row, then the same in all rows of a warp
    for by in [129.0 + 2.0 * row.double()] + [torch.full_like(row.double(), m) for m in range(129, 257, 14)]:
        by = by / 128.0 * 2.0 ** (power - half - 2) * sign
        q[..., 0] = by.to(torch.bfloat16).cuda()
        score = (by * ODD * 2.0 ** half * 0.5).T
        out, lse = keys.attend(q)
        assert_out(out, v.mean(0), G, size, "all equal")
        err = (lse.double().cpu() - (score + math.log(total))).abs()
        assert bool((err <= 2.0 ** -20 * score.abs() + 2.0 ** -10).all())
    if power < 11:
        return                                                    # half of a score that still leaves weights
    for which in {total - 3, 1, prefix + 66} if total < 1000 or power in (12, 26, 31) else ():
        x = k.clone()
        x[which, :, 0] *= 0.5 if sign < 0 else 2.0                # the largest score is that key's alone
        out, _ = Keys(path, x, v).attend(q)
        assert_out(out, v[which], G, size, f"key {which}")


@pytest.mark.parametrize("power", [60, 76, 90, 100, 116])
@pytest.mark.parametrize("path", PATHS)
def test_rows_of_any_size_at_right_angles(path, power):
    """Rows of Q and K of about 2^power whose products are zero: the mean of V."""
    G, H, n, prefix = path[2], path[3], path[4], path[6]
    k = torch.zeros((prefix + n, H, D), dtype=torch.float64)
    k[..., 0] = ODD * 2.0 ** (power - 2)
    v = signs(path, power, 0.75)
    out, lse = Keys(path, k, v).attend(queries(path, 1, 2.0 ** power))
    assert_out(out, v.mean(0), G, 0.75, "all equal")
    assert float((lse.double().cpu() - math.log(prefix + n)).abs().max()) <= 2.0 ** -10


@pytest.mark.parametrize("near,far", [(4, -126), (4, -121), (20, -100), (0, -90), (-11, -126), (60, -40), (-60, -126), (100, -20)])
@pytest.mark.parametrize("path", PATHS)
def test_values_far_below_others_keep_their_probability(path, near, far):
    """The first 64 keys have scores of 0 and V of 1536 2^near, all others scores of -3.375
    (4.9 in log2) and V of 1536 2^far, which adds nothing to an output but to the sum of
    the probabilities that it is divided by."""
    G, H, n, prefix = path[2], path[3], path[4], path[6]
    total = prefix + n
    k = torch.zeros((total, H, D), dtype=torch.float64)
    k[64:, :, 0] = ODD
    v = torch.full((total, H, D), 1536.0 * 2.0 ** far, dtype=torch.float64)
    v[:64] = 1536.0 * 2.0 ** near
    out, lse = Keys(path, k, v).attend(queries(path, 0, -1.0))
    L = 64.0 + (total - 64) * math.exp(-0.5 * ODD)
    want = (64.0 * v[0] + (total - 64) * math.exp(-0.5 * ODD) * v[64]) / L
    # bf16, the weights' fp16, and sums as above
    assert float((out.double().cpu() / want.repeat_interleave(G, dim=0) - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12
    assert float((lse.double().cpu() - math.log(L)).abs().max()) <= 2.0 ** -10


def unlike(n, g):        # within 2^13 of one another
    return torch.exp2(torch.randint(-6, 8, (n, 1, 1), generator=g).float())


def some_zero(n, g):
    return torch.where(torch.rand((n, 1, 1), generator=g) < 0.1, torch.zeros(()), torch.ones(()))


def zero_or_unlike(n, g):
    return some_zero(n, g) * unlike(n, g)


@pytest.mark.parametrize("scale", [0.3, 1.0, 5.0])
@pytest.mark.parametrize("v_scale", [unlike, some_zero, zero_or_unlike])
@pytest.mark.parametrize("lens,Sq,G,prefix", [([700, 129], 17, 2, 0), ([1415, 343, 1, 2000], 60, 5, 128), ([130, 130], 60, 3, 0), ([7, 40], 129, 8, 0),
                                             ([300, 0, 64], 4, 2, 2500), ([5000], 33, 1, 0), ([700, 129], 2, 2, 0)])
def test_heavy_keys_of_small_values(lens, Sq, G, prefix, v_scale, scale):
    """Where the keys that have the scores have small values, or zeros, the others' are what the
    output is made of: weights count with their own scale of V in a row's reference."""
    import quantized_attention_diffusion_gb300 as qad
    B, H, page = len(lens), 2, 64
    cache = Cache4(lens, H, page, seed=Sq + prefix, v_scale=v_scale, extra=(prefix,) if prefix else ())
    q = torch.randn((B, Sq, H * G, D), generator=torch.Generator().manual_seed(Sq)).to(torch.bfloat16)
    table = cache.table.cuda()
    kw = dict(softmax_scale=scale, causal=True, return_lse=True)
    if prefix:
        out, lse = qad.attn_fwd_cache_prefix(q.cuda(), cache.gpu(), table[B, :-(-prefix // page)].contiguous(), prefix, table[:B].contiguous(), ints(lens), **kw)
    else:
        out, lse = qad.attn_fwd_cache(q.cuda(), cache.gpu(), table, ints(lens), **kw)
    for b in range(B):
        rows = join(cache.dense(B), cache.dense(b)) if prefix else cache.dense(b)
        ref, z, tol, ltol = reference(q[b], rows, True, scale)
        # below 2^-126 bf16's steps are 2^-133 whatever the value: half of one
        assert_within(out[b], ref, tol + 2.0 ** -134, f"out of sequence {b}")
        assert_within(lse[b], z, ltol, f"lse of sequence {b}")
