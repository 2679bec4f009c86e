"""Norms and rotary positions of Q and K, and the pass that puts K and V into the
cache behind them, on the GPU against float64.

Bound of |out error| (u = 2^-24), M = factor (|n_a| + |n_b|) with n the normed values of
the pair: the norm's factor has the sum of 128 squares (128 u, halved by the root),
rsqrt's 2 ulp (4 u) and eps (2 u); the angle enters sine and cosine with pi 2^-25 (1.6 u),
they have 2 ulp (2 u), their factor one rounding, the products two, the last product
one: below 80 u M; then one rounding to bf16, 2^-8 of |out|."""
import math

import pytest
import torch

from tests.cache_common import D, assert_within, ints
from tests.gpu_common import ensure_library

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    return ensure_library()


@pytest.fixture(autouse=True)
def no_device_error():
    import quantized_attention_diffusion_gb300 as qad
    yield
    qad.debug_inject_fault(qad.FAULT_NONE)
    assert qad.sync_status() == 0


def exact(x, rope, freqs, positions, weight, eps):
    """(out, bound) in float64; positions int64 [B, S, axes]."""
    x = x.double().cpu()
    if eps is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        if weight is not None:
            x = x * weight.double().cpu()
    mass = x.abs()
    y = x.clone()
    if rope is not None:
        R = rope.dim
        axis = [a for a, n in enumerate(rope.sections) for _ in range(n)]
        # the angle in revolutions, reduced exactly: positions are whole, frequencies
        # doubles
        from fractions import Fraction
        inv = Fraction(1) / (2 * Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62))
        turns = [Fraction(f) * inv for f in freqs]
        B, S = positions.shape[:2]
        ang = torch.tensor([[[float(int(positions[b, s, axis[i]]) * turns[i] % 1) for i in range(R // 2)] for s in range(S)] for b in range(B)],
                           dtype=torch.float64) * 2 * math.pi
        c, s = ang.cos()[:, :, None] * rope.factor, ang.sin()[:, :, None] * rope.factor
        if rope.interleaved:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            y[..., 0:R:2], y[..., 1:R:2] = a * c - b * s, a * s + b * c
            mass[..., 0:R:2] = mass[..., 1:R:2] = abs(rope.factor) * (a.abs() + b.abs())
        else:
            h = R // 2
            a, b = x[..., :h], x[..., h:R]
            y[..., :h], y[..., h:R] = a * c - b * s, a * s + b * c
            mass[..., :h] = mass[..., h:R] = abs(rope.factor) * (a.abs() + b.abs())
    return y, 80 * U * mass + 2.0 ** -8 * y.abs()


def plain_freqs(dim, base=10000.0):
    return [base ** (-2.0 * i / dim) for i in range(dim // 2)]


@pytest.mark.parametrize("B,S,Hq,Hk,dim,interleaved,sections,norm", [
    (1, 1, 1, 1, 128, False, None, True),
    (2, 5, 3, 1, 128, True, None, True),
    (1, 37, 8, 2, 64, False, None, True),
    (3, 7, 2, 2, 96, False, None, False),
    (1, 9, 4, 4, 32, False, None, True),
    (2, 4, 5, 5, 32, True, None, False),
    (2, 6, 5, 1, 96, True, (16, 16, 16), True),
    (1, 33, 2, 3, 128, False, (16, 24, 24), True),
    (1, 50, 2, 2, 128, True, (1, 20, 21, 22), True),
    (1, 11, 17, 16, 64, True, (8, 24), False),
])
def test_norm_and_rotation(B, S, Hq, Hk, dim, interleaved, sections, norm):
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(B * 100 + S)
    q = (3 * torch.randn((B, S, Hq, D), generator=g)).to(torch.bfloat16)
    k = torch.randn((B, S, Hk, D), generator=g).to(torch.bfloat16)
    wq, wk = (torch.randn(D, generator=g).to(torch.bfloat16) for _ in "qk")
    rope = qad.Rope(dim, interleaved=interleaved, sections=sections)
    axes = len(rope.sections)
    pos = torch.randint(0, 200000, (B, S, axes), generator=g, dtype=torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -(2 ** 31)
    freqs = sum((plain_freqs(2 * n) for n in rope.sections), [])
    kw = dict(q_weight=wq.cuda(), k_weight=wk.cuda(), eps=1e-5) if norm else {}
    qo, ko = qad.qk_norm_rope(q.cuda(), k.cuda(), rope, pos.cuda() if axes > 1 else pos[..., 0].contiguous().cuda(), **kw)
    for got, x, w, what in ((qo, q, wq, "q"), (ko, k, wk, "k")):
        ref, tol = exact(x, rope, freqs, pos.long(), w if norm else None, 1e-5 if norm else None)
        assert_within(got, ref, tol, what)


def test_norm_alone_rotation_alone_and_nothing():
    import quantized_attention_diffusion_gb300 as qad
    q = torch.randn((2, 9, 5, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    got = qad.qk_norm_rope(q.cuda(), eps=1e-6)
    ref, tol = exact(q, None, None, None, None, 1e-6)
    assert_within(got, ref, tol)
    assert torch.equal(qad.qk_norm_rope(q.cuda()).cpu(), q)
    # unrotated channels pass as they are, infinities and NaN too, whatever their partners' place holds
    q[0, 0, 0, 100], q[0, 0, 1, 127] = math.inf, math.nan
    rope = qad.Rope(64)
    got = qad.qk_norm_rope(q.cuda(), rope=rope, positions=ints(range(9))).cpu()
    assert torch.equal(got[..., 64:].view(torch.int16), q[..., 64:].view(torch.int16))
    assert not got[..., :64].isnan().any()


def test_positions_of_one_token_shared_ones_and_slices():
    """[S] and [S, axes] for all of the batch, [B, 1], a projection's slices, filled in place."""
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(3)
    B, S, H = 3, 7, 4
    rope = qad.Rope(128, interleaved=True)
    qkv = torch.randn((B, S + 2, 3 * H, D), generator=g).to(torch.bfloat16).cuda()
    q, k = qkv[:, 1:S + 1, :H], qkv[:, 2:, H:2 * H]
    pos = ints(range(50, 50 + S))
    qo, ko = qad.qk_norm_rope(q, k, rope, pos)
    full = pos.expand(B, S).contiguous()
    q2, k2 = qad.qk_norm_rope(q.contiguous(), k.contiguous(), rope, full)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    ref, tol = exact(q, rope, plain_freqs(128), full.cpu().long()[..., None], None, None)
    assert_within(qo, ref, tol)
    dense_q, dense_k = q.contiguous(), k.contiguous()
    got = qad.qk_norm_rope(dense_q, dense_k, rope, pos, out=(dense_q, dense_k))
    assert got[0] is dense_q and torch.equal(dense_q, qo) and torch.equal(dense_k, ko)
    one = qad.qk_norm_rope(q[:, :1], None, rope, full[:, :1])
    assert torch.equal(one, qo[:, :1])
    three = qad.Rope(128, sections=(16, 24, 24))
    p3 = torch.randint(0, 99, (S, 3), generator=g, dtype=torch.int32)
    a = qad.qk_norm_rope(q, None, three, p3.cuda())
    b = qad.qk_norm_rope(q, None, three, p3.expand(B, S, 3).contiguous().cuda())
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 80, 40), (5000, 3, 1), (700, 33, 17), (20000, 40, 1)])
def test_heads_split_over_warps_give_the_same_bits(T, Hq, Hk):
    """However many heads a warp takes: rows of a large call are those of one-token calls."""
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(T)
    q = torch.randn((1, T, Hq, D), generator=g).to(torch.bfloat16).cuda()
    k = torch.randn((1, T, Hk, D), generator=g).to(torch.bfloat16).cuda()
    rope = qad.Rope(128)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32).cuda()
    qo, ko = qad.qk_norm_rope(q, k, rope, pos, eps=1e-6)
    for t in {0, T // 2, T - 1}:
        a, b = qad.qk_norm_rope(q[:, t:t + 1], k[:, t:t + 1], rope, pos[t:t + 1], eps=1e-6)
        assert torch.equal(a[0, 0], qo[0, t]) and torch.equal(b[0, 0], ko[0, t])
    # the mean of the squares of normed rows is 1 within bf16's roundings: nothing is left unwritten
    assert (qo.float().square().mean(-1) - 1).abs().max() < 2.0 ** -6


# ---------------------------------------------------------------- append --

def _state(seed, B, S, Hq, H, page, pages, bits):
    import quantized_attention_diffusion_gb300 as qad
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn((B, S, Hq + 2 * H, D), generator=g).to(torch.bfloat16).cuda()
    caches = [qad.kv_cache_alloc(pages, H, page, bits=bits) for _ in range(2)]
    for c in caches:
        for t in c:
            t.view(torch.uint8).fill_(0x5A)
    return g, qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:], caches


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("B,S,Hq,H,page,dim,interleaved,norm", [
    (1, 1, 1, 1, 16, 128, False, True),
    (5, 1, 8, 2, 16, 64, False, True),
    (2, 37, 3, 3, 32, 96, True, True),
    (3, 20, 0, 2, 64, 32, False, True),            # no q
    (1, 300, 12, 5, 128, 128, True, False),
    (2, 150, 4, 1, 256, None, False, False),       # written as they are
])
def test_append_is_norm_rotation_and_write(bits, B, S, Hq, H, page, dim, interleaved, norm):
    import quantized_attention_diffusion_gb300 as qad
    width = -(-(S + 40) // page) + 1
    g, q, k, v, (one, two) = _state(S + bits, B, S, Hq, H, page, B * width + 2, bits)
    table = torch.randperm(B * width + 2, generator=g)[:B * width].to(torch.int32).view(B, width)
    start = torch.randint(0, 40, (B,), generator=g)
    at = start[:, None] + torch.arange(S)
    slots = (table.gather(1, at // page) * page + at % page).to(torch.int32)
    rope = None if dim is None else qad.Rope(dim, interleaved=interleaved, scaling=("yarn", 4.0, 8192))
    pos = None if dim is None else at.to(torch.int32).cuda()
    w = torch.randn((2, D), generator=g).to(torch.bfloat16).cuda()
    kw = dict(rope=rope, positions=pos, eps=1e-6 if norm else None, k_weight=w[1] if norm else None)
    kq = dict(kw, q_weight=w[0] if norm else None)
    got = qad.kv_cache_append(q if Hq else None, k, v, one, slots.cuda(), **(kq if Hq else kw))
    if Hq:
        want_q, want_k = qad.qk_norm_rope(q, k, **kq)
        assert torch.equal(got, want_q)
    else:
        assert got is None
        _, want_k = qad.qk_norm_rope(k, k, rope, pos, k_weight=w[1], eps=1e-6)
    qad.kv_cache_write(want_k, v, two, table.cuda(), start.to(torch.int32).cuda())
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [4, 8])
def test_append_skips_negative_slots_and_reports_those_behind_the_cache(bits):
    import quantized_attention_diffusion_gb300 as qad
    _, q, k, v, (one, two) = _state(7, 1, 9, 4, 2, 16, 3, bits)
    slots = ints([5, -1, 47, -(2 ** 31), 0, 17, 18, 19, 46])
    rope = qad.Rope()
    pos = ints(range(9))
    qad.kv_cache_append(q, k, v, one, slots, rope, pos)
    want_q, want_k = qad.qk_norm_rope(q, k, rope, pos)
    keep = [0, 2, 4, 5, 6, 7, 8]
    qad.kv_cache_write(want_k[:, keep].transpose(0, 1), v[:, keep].transpose(0, 1), two, ints([0, 1, 2]).expand(7, 3).contiguous(),
                       slots[keep].contiguous())
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert qad.sync_status() == 0
    bad = slots.clone()
    bad[1], bad[3] = 48, 2 ** 31 - 1
    got = qad.kv_cache_append(q, k, v, one, bad, rope, pos)
    assert qad.sync_status() == 8
    assert torch.equal(got, want_q)
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_injected_faults_and_refusals():
    import quantized_attention_diffusion_gb300 as qad
    _, q, k, v, (cache, _) = _state(7, 1, 3, 4, 2, 16, 3, 4)
    slots, pos, rope = ints([0, 1, 2]), ints([0, 1, 2]), qad.Rope()
    for call in (lambda: qad.qk_norm_rope(q, k, rope, pos), lambda: qad.kv_cache_append(q, k, v, cache, slots, rope, pos)):
        qad.debug_inject_fault(qad.FAULT_QUANT_LAUNCH)
        with pytest.raises(qad.SageError, match="injected"):
            call()
        call()
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    flat = torch.zeros((1, 8, 2, D), dtype=torch.bfloat16, device="cuda")
    dq = torch.zeros((1, 3, 2, D), dtype=torch.bfloat16, device="cuda")
    dk = torch.zeros_like(dq)
    refused = [
        (lambda: qad.qk_norm_rope(q, k, rope), TypeError), (lambda: qad.qk_norm_rope(q, k, None, pos), ValueError),
        (lambda: qad.qk_norm_rope(q, k, rope, pos.long()), ValueError), (lambda: qad.qk_norm_rope(q, k, rope, pos[:2]), ValueError),
        (lambda: qad.qk_norm_rope(q, k, rope, pos, q_weight=w), ValueError),
        (lambda: qad.qk_norm_rope(q, k, rope, pos, q_weight=w.float(), eps=0.0), ValueError),
        (lambda: qad.qk_norm_rope(q, k, rope, pos, eps=-1.0), ValueError), (lambda: qad.qk_norm_rope(q, k, rope, pos, eps=math.nan), ValueError),
        (lambda: qad.qk_norm_rope(q.float(), k, rope, pos), ValueError), (lambda: qad.qk_norm_rope(q, k[:, :2], rope, pos), ValueError),
        (lambda: qad.qk_norm_rope(q, k, rope, pos, out=(torch.empty_like(k.contiguous()),) * 2), ValueError),
        (lambda: qad.qk_norm_rope(dq, dk, rope, pos, out=(dk, dq)), qad.SageError),
        (lambda: qad.qk_norm_rope(flat[:1, 1:4], None, rope, pos, out=flat[:1, :3]), qad.SageError),
        (lambda: qad.kv_cache_append(dq[:, :, :2].contiguous(), dk, v, cache, slots, rope, pos, out=dk), qad.SageError),
        (lambda: qad.kv_cache_append(q, k, v, cache, slots[:2], rope, pos), ValueError),
        (lambda: qad.kv_cache_append(q, k, v, cache, slots.long(), rope, pos), ValueError),
        (lambda: qad.kv_cache_append(q, k, v[:, :, :1], cache, slots, rope, pos), ValueError),
        (lambda: qad.kv_cache_append(None, k, v, cache, slots, rope, pos, q_weight=w, eps=0.0), ValueError),
    ]
    for call, error in refused:
        with pytest.raises(error):
            call()
