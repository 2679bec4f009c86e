"""Pages of the KV cache given to new tokens and taken back on the GPU, against a plain
walk over the sequences, and the whole generation step: pages, append, attention."""
import math
import random

import pytest
import torch

from tests.cache_common import D, assert_within, ints, reference
from tests.gpu_common import ensure_library
from tests.kv4_common import quantize4, values4

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
    qad.debug_inject_fault(qad.FAULT_NONE)
    assert qad.sync_status() == 0


def walk(pool, free, lens, counts, table, page, tokens, layout):
    """What sage_kv_pages_reserve says it does."""
    B = len(lens)
    table = [list(r) for r in table]
    rows = tokens if layout == "packed" else B * tokens
    slots, positions = [-1] * rows, [0] * rows
    taken, first, asked, gone, at = [], [], 0, 0, 0
    for b, (n, c) in enumerate(zip(lens, counts)):
        held, want = -(-n // page), -(-(n + c) // page)
        ok = want == held or asked + want - held <= free
        if ok:
            for j in range(want - held):
                table[b][held + j] = pool[free - 1 - asked - j]
        asked += want - held
        if ok and want > held:
            gone = asked
        taken.append(c if ok else 0)
        row = at if layout == "packed" else b * tokens + (tokens - c if layout == "end" else 0)
        first.append(row)
        at += c
        for i in range(taken[-1]):
            p = n + i
            slots[row + i], positions[row + i] = table[b][p // page] * page + p % page, p
    return taken, first, free - gone, table, slots, positions


def _make(seed, B, page, most, new, free=None, tokens=None, layout="packed"):
    r = random.Random(seed)
    lens = [r.choice([0, r.randint(0, most), r.randint(0, most) // page * page]) for _ in range(B)]
    counts = [r.randint(0, new) for _ in range(B)]
    need = sum(-(-(n + c) // page) - -(-n // page) for n, c in zip(lens, counts))
    held = sum(-(-n // page) for n in lens)
    spare = need + 7
    pages = list(range(held + spare))
    r.shuffle(pages)
    width = max(1, max(-(-(n + c) // page) for n, c in zip(lens, counts))) + 1
    table, at = [], 0
    for n in lens:
        k = -(-n // page)
        table.append(pages[at:at + k] + [-1] * (width - k))
        at += k
    pool = pages[at:] + [-7] * held
    free = spare if free is None else free(need)
    if tokens is None:
        tokens = max(1, sum(counts)) + 5 if layout == "packed" else max(1, max(counts)) + 2
    return pool, free, lens, counts, table, tokens


@pytest.mark.parametrize("layout", ["packed", "front", "end"])
@pytest.mark.parametrize("B,page,most,new,short", [
    (1, 16, 0, 1, False), (1, 16, 40, 1, False), (48, 64, 16384, 1, False), (7, 16, 100, 50, False), (33, 32, 500, 200, True),
    (256, 16, 2000, 90, False), (1500, 16, 60, 12, False), (1500, 16, 60, 12, True), (3000, 64, 10, 1, True), (4, 256, 1000, 5000, False),
])
def test_reserve(B, page, most, new, short, layout):
    import quantized_attention_diffusion_gb300 as qad
    pool, free, lens, counts, table, tokens = _make(B + page, B, page, most, new, (lambda need: need // 2) if short else None, layout=layout)
    want = walk(pool, free, lens, counts, table, page, tokens, layout)
    t = torch.tensor(table, dtype=torch.int32, device="cuda")
    got = qad.kv_pages_reserve(ints(pool), ints([free]), ints(lens), ints(counts), t, page, tokens, layout)
    assert got.start.tolist() == lens
    assert got.taken.tolist() == want[0]
    assert got.lens.tolist() == [n + c for n, c in zip(lens, want[0])]
    assert got.first.tolist() == want[1]
    assert got.free_count.tolist() == [want[2]]
    assert t.tolist() == want[3]
    assert got.slots.flatten().tolist() == want[4]
    assert got.positions.flatten().tolist() == want[5]
    assert qad.sync_status() == (9 if want[0] != counts else 0)


def test_reserve_in_place_and_release_restore_the_stack():
    import quantized_attention_diffusion_gb300 as qad
    for B, layout in ((9, "packed"), (1400, "front")):
        pool, free, lens, counts, table, tokens = _make(B, B, 16, 90, 70, layout=layout)
        p, f, n = ints(pool), ints([free]), ints(lens)
        t = torch.tensor(table, dtype=torch.int32, device="cuda")
        fresh = qad.kv_pages_reserve(p, f, n, ints(counts), t.clone(), 16, tokens, layout)
        out = qad.PagePlan(fresh.start.clone(), fresh.taken.clone(), n, fresh.first.clone(), f, fresh.slots.clone(), fresh.positions.clone())
        got = qad.kv_pages_reserve(p, f, n, ints(counts), t, 16, tokens, layout, out=out)
        assert got is out and all(torch.equal(a, b) for a, b in zip(got, fresh))
        qad.kv_pages_release(p, f, n, ints([x + 1000 * (i % 2) for i, x in enumerate(n.tolist())]), t, 16)      # nothing to do
        assert torch.equal(f, fresh.free_count) and torch.equal(n, fresh.lens)
        qad.kv_pages_release(p, f, n, ints(lens), t, 16)
        assert n.tolist() == lens and f.tolist() == [free] and p.tolist() == pool and t.tolist() == table
        qad.kv_pages_release(p, f, n, ints([0] * B), t, 16)
        held = sum(-(-x // 16) for x in lens)
        assert f.tolist() == [free + held] and not n.any() and (t == -1).all()
        assert sorted(p.tolist()[:free + held]) == sorted(set(pool[:free]) | {x for r in table for x in r if x >= 0})


def test_release_of_some():
    import quantized_attention_diffusion_gb300 as qad
    table = torch.tensor([[3, 5, 7], [1, 0, -1], [2, -1, -1]], dtype=torch.int32, device="cuda")
    pool, free, lens = ints([4, 6, 9, 9, 9, 9, 9, 9]), ints([2]), ints([40, 17, 16])
    qad.kv_pages_release(pool, free, lens, ints([16, -3, 99]), table, 16)
    assert lens.tolist() == [16, 0, 16] and free.tolist() == [6]
    assert pool.tolist() == [4, 6, 0, 1, 7, 5, 9, 9]          # the last page given is the first back
    assert table.tolist() == [[3, -1, -1], [-1, -1, -1], [2, -1, -1]]


def test_what_is_wrong_on_the_device_is_reported():
    import quantized_attention_diffusion_gb300 as qad
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    pool = ints([0, 1, 2, 3])

    def call(lens=(0, 0, 0), counts=(1, 1, 1), free=4, tokens=3, pages=pool, layout="packed"):
        return qad.kv_pages_reserve(pages, ints([free]), ints(lens), ints(counts), table.fill_(-1), 16, tokens, layout)

    for lens, counts in (((0, -1, 0), (1, 1, 1)), ((0, 5, 0), (1, -1, 1)), ((0, 32, 0), (1, 1, 1)), ((0, 2 ** 31 - 1, 0), (1, 2 ** 31 - 1, 1))):
        got = call(lens, counts)
        assert qad.sync_status() == 8
        assert got.taken.tolist() == [1, 0, 1] and got.free_count.tolist() == [2] and got.lens.tolist()[1] == lens[1]
        assert table[0, 0] == 3 and table[2, 0] == 2 and table[1].tolist() == [-1, -1]
        assert got.slots[0] == 48
    got = call(tokens=2)                                       # fewer rows than tokens
    assert qad.sync_status() == 8 and got.slots.tolist() == [48, 32]
    got = call(counts=(1, 4, 1), layout="end", tokens=3)
    assert qad.sync_status() == 8 and got.taken.tolist() == [1, 0, 1]
    assert got.slots.tolist() == [[-1, -1, 48], [-1, -1, -1], [-1, -1, 32]]
    for free in (5, -1, 2 ** 31 - 1):
        got = call(free=free)
        assert qad.sync_status() in (8, 9)
    got = call(pages=ints([0, 1, 4, -1]))                      # no pages of this cache
    assert qad.sync_status() == 8 and got.slots.tolist() == [-1, -1, 16]
    # release: an entry that is no page, more pages than there are
    f, n = ints([0]), ints([20, 0, 0])
    t = torch.tensor([[1, 9], [-1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    qad.kv_pages_release(pool.clone(), f, n, ints([0, 0, 0]), t, 16)
    assert qad.sync_status() == 8
    f, n = ints([3]), ints([20, 0, 0])
    t = torch.tensor([[1, 2], [-1, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    guard = ints([0, 1, 2, 3, 77])
    qad.kv_pages_release(guard[:4], f, n, ints([0, 0, 0]), t, 16)
    assert qad.sync_status() == 8 and f.tolist() == [4] and guard[4] == 77


def test_refusals():
    import quantized_attention_diffusion_gb300 as qad
    pool, free, lens, t = ints([0, 1]), ints([2]), ints([0]), ints([-1]).view(1, 1)
    for kw in (dict(page_size=20), dict(layout="left"), dict(tokens=0), dict(counts=ints([1, 2])), dict(free_count=ints([1, 2])),
               dict(lens=lens.long()), dict(block_table=t.view(1)), dict(free_pages=pool.cpu())):
        args = dict(free_pages=pool, free_count=free, lens=lens, counts=ints([1]), block_table=t, page_size=16, tokens=1)
        with pytest.raises(ValueError):
            qad.kv_pages_reserve(**{**args, **kw})
    with pytest.raises(qad.SageError, match="overlap"):
        qad.kv_pages_reserve(pool, free, ints([0, 0]), ints([1, 1]), t.expand(2, 1), 16, 2)
    for call in (lambda: qad.kv_pages_reserve(pool, free, lens, ints([1]), t, 16, 1), lambda: qad.kv_pages_release(pool, free, lens, ints([0]), t, 16)):
        qad.debug_inject_fault(qad.FAULT_QUANT_LAUNCH)
        with pytest.raises(qad.SageError, match="injected"):
            call()


@pytest.mark.parametrize("bits", [8, 4])
def test_steps_recorded_and_replayed(bits):
    """Prompts of unequal lengths, padded at the end of their rows, then generation
    steps from one recorded graph: pages, norm, rotation, cache and attention, each step
    against float64 over what the cache should hold."""
    import quantized_attention_diffusion_gb300 as qad
    B, Hq, H, page, width, steps = 3, 8, 2, 16, 6, 20
    g = torch.Generator().manual_seed(bits)
    cache = qad.kv_cache_alloc(B * width + 1, H, page, bits=bits)
    rope = qad.Rope(128)
    w = (1 + 0.1 * torch.randn((2, D), generator=g)).to(torch.bfloat16).cuda()
    pool = torch.randperm(B * width + 1, generator=g).to(torch.int32).cuda()
    free, lens = ints([B * width + 1]), ints([0] * B)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    history = [[] for _ in range(B)]

    def remember(k, v, where):
        for b, rows in enumerate(where):
            for s in rows:
                history[b].append((k[b, s].cpu(), v[b, s].cpu()))

    def check(q, out, rows):
        for b in range(B):
            k, v = (torch.stack([x[i] for x in history[b]]) for i in (0, 1))
            if bits == 4:
                kc, kb, ks = quantize4(k)
                vc, vb, vs = quantize4(v)
                dense = values4(kc, kb), ks.double(), values4(vc, vb), vs.double()
            else:
                from tests.cache_common import quantize_kv
                kc, ks, vc, vs = quantize_kv(k, v)
                dense = kc.double(), ks.double(), vc.float().double(), vs.double()
            ref, _, tol, _ = reference(q[b, -rows[b]:].cpu(), dense, True, 1 / math.sqrt(D))
            assert_within(out[b, -rows[b]:], ref, tol, f"sequence {b}")

    counts = [37, 5, 21]
    S = 37
    qkv = torch.randn((B, S, Hq + 2 * H, D), generator=g).to(torch.bfloat16).cuda()
    plan = qad.kv_pages_reserve(pool, free, lens, ints(counts), table, page, S, "end")
    lens.copy_(plan.lens)
    free.copy_(plan.free_count)
    kw = dict(q_weight=w[0], k_weight=w[1], eps=1e-6)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    q_out = qad.kv_cache_append(q, k, v, cache, plan.slots, rope, plan.positions, **kw)
    out = qad.attn_fwd_cache(q_out, cache, table, lens)
    turned = qad.qk_norm_rope(q, k, rope, plan.positions, **kw)[1]
    remember(turned, v, [range(S - c, S) for c in counts])
    check(q_out, out, counts)

    # one token a step
    x = torch.empty((B, 1, Hq + 2 * H, D), dtype=torch.bfloat16, device="cuda")
    one = ints([1] * B)
    out = torch.empty((B, 1, Hq, D), dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty_like(out)
    rows = qad.PagePlan(*(torch.empty(n, dtype=torch.int32, device="cuda") for n in (B, B)), lens, torch.empty_like(lens), free,
                        *(torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2)))

    def step():
        qad.kv_pages_reserve(pool, free, lens, one, table, page, B, out=rows)
        qad.kv_cache_append(x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:], cache, rows.slots, rope, rows.positions, out=q_out, **kw)
        qad.attn_fwd_cache(q_out, cache, table, lens, out=out)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        x.copy_(torch.randn(x.shape, generator=g))
        graph.replay()
        assert rows.positions.tolist() == [c + i for c in counts] and lens.tolist() == [c + i + 1 for c in counts]
        turned = qad.qk_norm_rope(x[:, :, :Hq], x[:, :, Hq:Hq + H], rope, rows.positions, **kw)[1]
        remember(turned, x[:, :, Hq + H:], [[0]] * B)
        if i in (0, 10, steps - 1):
            check(q_out, out, [1] * B)
    used = sum(-(-(c + steps) // page) for c in counts)
    assert free.tolist() == [B * width + 1 - used]
    assert len({p for p in table.flatten().tolist() if p >= 0} | set(pool.tolist()[:free.item()])) == B * width + 1
