"""Timed cases of the quantised KV cache and of the attention that reads it.

The cache holds K as INT8 and V as E4M3 codes, one fp32 scale for each token of
each key/value head, in pages of ``page`` tokens:

    k_codes int8 [pages, Hkv, page, 128]      k_scale fp32 [pages, Hkv, page]
    v_codes e4m3 [pages, Hkv, page, 128]      v_scale fp32 [pages, Hkv, page]

Position i of sequence b is token ``i % page`` of page ``table[b, i // page]``.

    write    k, v bf16 -> codes and scales at start[b] .. start[b] + count[b] - 1
    read     codes and scales -> k, v bf16, zeros behind a sequence's end
    attn     the last Sq positions of each sequence attend to all of it
    prefix   the same where all sequences begin with the same cached tokens

With ``own`` false ``run`` computes them by elementary torch operations in 32
bits (the quantiser's quotients in 64, rounded once to 32), with ``own`` true
it calls the library.
"""
import math
import random

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


def listed():
    return [
        # one new token for each of eight running sequences: a generation step's write
        dict(name="write_step", op="write", B=8, S=1, H=8, page=16, len_min=100, len_max=4000, lens=1, ragged=False, fused=False),
        # a padded batch of prompts of unequal lengths, K and V sliced out of one projection's output
        dict(name="write_prompts", op="write", B=5, S=1531, H=4, page=32, len_min=0, len_max=700, lens=2, ragged=True, fused=True),
        # a video's tokens, all at once
        dict(name="write_video", op="write", B=2, S=32760, H=16, page=128, len_min=0, len_max=0, lens=3, ragged=False, fused=False),
        # a few short contexts read back, as for attention in full precision
        dict(name="read_short", op="read", B=3, S=333, H=2, page=16, len_min=1, len_max=333, lens=4),
        # long contexts read back
        dict(name="read_long", op="read", B=4, S=16384, H=8, page=64, len_min=12000, len_max=16384, lens=5),
        # one sequence, one token, a short context: latency
        dict(name="attn_step_one", op="attn", B=1, Sq=1, Hq=32, Hkv=8, page=16, len_min=777, len_max=777, lens=6, causal=True),
        # a generation step of a ragged batch with grouped heads
        dict(name="attn_step_batch", op="attn", B=48, Sq=1, Hq=32, Hkv=8, page=64, len_min=64, len_max=16384, lens=7, causal=True),
        # one long video context, a head of keys for each head of queries
        dict(name="attn_step_long", op="attn", B=1, Sq=1, Hq=24, Hkv=24, page=128, len_min=65536, len_max=65536, lens=8, causal=True),
        # a chunk of new tokens against what came before it
        dict(name="attn_chunk", op="attn", B=2, Sq=1000, Hq=16, Hkv=4, page=64, len_min=7000, len_max=9000, lens=9, causal=True),
        # a few continuations of one short prompt
        dict(name="prefix_few", op="prefix", B=6, Sq=1, Hq=8, Hkv=2, page=16, prefix=1001, len_min=1, len_max=90, lens=10, causal=True),
        # many continuations of one long context
        dict(name="prefix_many", op="prefix", B=64, Sq=1, Hq=32, Hkv=8, page=64, prefix=16384, len_min=1, len_max=512, lens=11, causal=True),
        # blocks of five drafted tokens behind a video's context, ungrouped heads
        dict(name="prefix_drafts", op="prefix", B=24, Sq=5, Hq=16, Hkv=16, page=128, prefix=32760, len_min=5, len_max=64, lens=12, causal=True),
    ]


def draw(rng):
    def over(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["write", "read", "attn", "attn", "prefix", "prefix"])
    case = dict(op=op, page=rng.choice([16, 32, 64, 128, 256]), lens=rng.randrange(1 << 30))
    if op == "write":
        B, S, H = over(1, 64), over(1, 32760), over(1, 24)
        S = max(1, min(S, (1 << 20) // (B * H)))
        case.update(B=B, S=S, H=H, len_min=0, len_max=over(1, 1000), ragged=rng.random() < 0.5, fused=rng.random() < 0.5)
    elif op == "read":
        B, S, H = over(1, 32), over(1, 16384), over(1, 16)
        S = max(1, min(S, (1 << 19) // (B * H)))
        case.update(B=B, S=S, H=H, len_min=0, len_max=S)
    elif op == "attn":
        Hkv, G = over(1, 16), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        Sq = 1 if rng.random() < 0.5 else over(1, 1000)
        B, longest = over(1, 48), over(1, 65536)
        longest = max(Sq, min(longest, (1 << 21) // (B * Hkv), (1 << 27) // (B * Hkv * G * Sq)))
        B = max(1, min(B, (1 << 27) // (longest * Hkv * G * Sq)))
        case.update(B=B, Sq=Sq, Hq=Hkv * G, Hkv=Hkv, len_min=rng.choice([0, Sq]), len_max=longest, causal=rng.random() < 0.7)
    else:
        Hkv, G = over(1, 16), rng.choice([1, 2, 4, 5, 8])
        Sq, B, prefix = rng.choice([1, 1, 1, 2, 5, 8]), over(2, 64), over(50, 32760)
        prefix = max(1, min(prefix, (1 << 26) // (B * Hkv * G * Sq)))
        case.update(B=B, Sq=Sq, Hq=Hkv * G, Hkv=Hkv, prefix=prefix, len_min=rng.choice([0, Sq]), len_max=over(Sq, 512), causal=rng.random() < 0.7)
    return case


def _lens(case):
    """Lengths of the sequences in the cache (for a write: before it)."""
    r = random.Random(case["lens"])
    return [r.randint(case["len_min"], case["len_max"]) for _ in range(case["B"])]


def _counts(case):
    """New tokens of each sequence of a write."""
    r = random.Random(case["lens"] + 1)
    S = case["S"]
    return [r.randint(0, S) for _ in range(case["B"])] if case["ragged"] else [S] * case["B"]


def _quantize(x, levels):
    """Scales of rows of 128 and the quotients x / scale, both fp32 rounded to nearest."""
    x = x.double()
    scale = (x.abs().amax(-1) / levels).float()
    y = (x / scale.double().unsqueeze(-1)).float()
    return scale, torch.where(scale.unsqueeze(-1) == 0, torch.zeros_like(y), y)


def _codes_k(y):
    return y.round().clamp(-127, 127).to(torch.int8)


def _codes_v(y):
    return y.clamp(-448, 448).to(torch.float8_e4m3fn)


def _tables(gen, need, page, width, spare):
    """A table of distinct pages in no order, -1 behind what a sequence needs."""
    pages = [-(-n // page) for n in need]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(1, width)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _filled(gen, total, H, page):
    """A cache of `total` pages as it stands after the writes of normal K and V,
    K with channel offsets as diffusion models have them."""
    shape = (total, H, page, D)
    offset = torch.randn((1, H, 1, D), generator=gen, device="cuda") * 2
    k_codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    v_codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    k_scale = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
    v_scale = torch.empty_like(k_scale)
    step = max(1, (1 << 27) // (H * page * D))
    for i in range(0, total, step):
        n = min(step, total - i)
        for codes, scale, levels, to in ((k_codes, k_scale, 127.0, _codes_k), (v_codes, v_scale, 448.0, _codes_v)):
            x = torch.randn((n,) + shape[1:], generator=gen, device="cuda")
            if codes is k_codes:
                x = x + offset
            x = x.to(torch.bfloat16).float()
            s = x.abs().amax(-1) / levels
            codes[i:i + n] = to(x / s.unsqueeze(-1))
            scale[i:i + n] = s
    return k_codes, k_scale, v_codes, v_scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    B, page = case["B"], case["page"]
    lens = _lens(case)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    s = dict(case=dict(case))
    if case["op"] == "write":
        S, H = case["S"], case["H"]
        counts = _counts(case)
        need = [a + c for a, c in zip(lens, counts)]
        width = -(-max(a + S for a in lens) // page)
        s["table"], total = _tables(gen, need, page, width, 3)
        if case["fused"]:   # q, k and v heads of one projection: H each
            qkv = normal(B, S, 3 * H, D)
            s["k"], s["v"] = qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
        else:
            s["k"], s["v"] = normal(B, S, H, D), normal(B, S, H, D)
        s["cache"] = (torch.zeros((total, H, page, D), dtype=torch.int8, device="cuda"),
                      torch.zeros((total, H, page), device="cuda"),
                      torch.zeros((total, H, page, D), device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn),
                      torch.zeros((total, H, page), device="cuda"))
        s["start"] = ints(lens)
        s["count"] = ints(counts) if case["ragged"] else None
        return s
    s["lens"], s["longest"] = ints(lens), max([1] + lens)
    if case["op"] == "read":
        s["table"], total = _tables(gen, lens, page, -(-case["S"] // page), 3)
        s["cache"] = _filled(gen, total, case["H"], page)
        return s
    s["q"] = normal(B, case["Sq"], case["Hq"], D)
    width = -(-max(lens) // page)
    if case["op"] == "prefix":
        both, total = _tables(gen, lens + [case["prefix"]], page, max(width, -(-case["prefix"] // page)), 3)
        s["table"] = both[:B, :max(1, width)].contiguous()
        s["prefix_table"] = both[B, :-(-case["prefix"] // page)].contiguous()
    else:
        s["table"], total = _tables(gen, lens, page, width, 3)
    s["cache"] = _filled(gen, total, case["Hkv"], page)
    return s


# --------------------------------------------------------------- plain form --

def _gather(codes, scale, table, L):
    """fp32 [B, H, L, 128] of the first L positions of each row of the table."""
    page = codes.shape[2]
    pages = table[:, :-(-L // page)].clamp(min=0).long()
    c = codes[pages].float()                                  # [B, n, H, page, D]
    x = c * scale[pages].unsqueeze(-1)
    x = x.transpose(1, 2).reshape(table.shape[0], codes.shape[1], -1, D)
    return x[:, :, :L]


def _write(s):
    k, v, cache, table, start, count = s["k"], s["v"], s["cache"], s["table"], s["start"], s["count"]
    page = cache[0].shape[2]
    B, S = k.shape[:2]
    i = torch.arange(S, device="cuda")
    pos = start.long()[:, None] + i
    where = table.long().gather(1, pos // page)
    for x, codes, scale, levels, to in ((k, cache[0], cache[1], 127.0, _codes_k), (v, cache[2], cache[3], 448.0, _codes_v)):
        sc, y = _quantize(x, levels)
        p, o, c = where, pos % page, to(y)
        if count is not None:
            live = i < count[:, None]
            p, o, c, sc = p[live], o[live], c[live], sc[live]
        codes.view(torch.uint8)[p, :, o] = c.view(torch.uint8)
        scale[p, :, o] = sc
    return cache


def _read(s):
    case, cache = s["case"], s["cache"]
    dead = torch.arange(case["S"], device="cuda") >= s["lens"][:, None]
    out = []
    for codes, scale in (cache[:2], cache[2:]):
        x = _gather(codes, scale, s["table"], case["S"]).transpose(1, 2).to(torch.bfloat16)
        out.append(x.masked_fill(dead[:, :, None, None], 0))
    return tuple(out)


def _limits(case, lens, before):
    """Keys that each query of each sequence sees, [B, Sq]: `before` + its own."""
    Sq = case["Sq"]
    lens = lens.long()[:, None] + before
    if not case["causal"]:
        return lens.expand(-1, Sq)
    return (lens - Sq + 1 + torch.arange(Sq, device="cuda")).clamp(min=0)


def _attn(s):
    case, cache, q = s["case"], s["cache"], s["q"]
    B, Sq, Hq, Hkv = case["B"], case["Sq"], case["Hq"], case["Hkv"]
    G, P = Hq // Hkv, case.get("prefix", 0)
    L = s["longest"]
    rows = q.float().view(B, Sq, Hkv, G, D).permute(0, 2, 1, 3, 4)            # [B, Hkv, Sq, G, D]
    k, v = (_gather(cache[i], cache[i + 1], s["table"], L) for i in (0, 2))
    x = rows.reshape(B, Hkv, Sq * G, D) @ k.transpose(2, 3)
    if P:
        pk, pv = (_gather(cache[i], cache[i + 1], s["prefix_table"][None], P)[0] for i in (0, 2))
        px = rows.permute(1, 0, 2, 3, 4).reshape(Hkv, B * Sq * G, D) @ pk.transpose(1, 2)
        x = torch.cat([px.view(Hkv, B, Sq * G, P).transpose(0, 1), x], dim=-1)
    sees = torch.arange(P + L, device="cuda") < _limits(case, s["lens"], P)[:, :, None]   # [B, Sq, P + L]
    x = (x * SCALE).view(B, Hkv, Sq, G, P + L).masked_fill(~sees[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - torch.where(m == -math.inf, torch.zeros_like(m), m)).exp().view(B, Hkv, Sq * G, P + L)
    total = p.sum(-1, keepdim=True)
    o = p[..., P:] @ v
    if P:
        o = o + (p[..., :P].transpose(0, 1).reshape(Hkv, -1, P) @ pv).view(Hkv, B, Sq * G, D).transpose(0, 1)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = m.view(B, Hkv, Sq, G) + total.view(B, Hkv, Sq, G).log()
    o = o.view(B, Hkv, Sq, G, D).permute(0, 2, 1, 3, 4).reshape(B, Sq, Hq, D)
    return o.to(torch.bfloat16), lse.permute(0, 1, 3, 2).reshape(B, Hq, Sq).contiguous()


def run(state):
    case = state["case"]
    if own:
        import quantized_attention_diffusion_gb300 as qad
        if case["op"] == "write":
            return qad.kv_cache_write(state["k"], state["v"], state["cache"], state["table"], state["start"], state["count"])
        if case["op"] == "read":
            return qad.kv_cache_read(state["cache"], state["table"], state["lens"], case["S"])
        if case["op"] == "attn":
            return qad.attn_fwd_cache(state["q"], state["cache"], state["table"], state["lens"], causal=case["causal"], return_lse=True)
        return qad.attn_fwd_cache_prefix(state["q"], state["cache"], state["prefix_table"], case["prefix"], state["table"],
                                         state["lens"], causal=case["causal"], return_lse=True)
    if case["op"] == "write":
        return _write(state)
    if case["op"] == "read":
        return _read(state)
    return _attn(state)


# --------------------------------------------------------- work and 64 bits --

def work(case):
    B, lens = case["B"], _lens(case)
    if case["op"] == "write":   # K and V in bf16, codes and scales out, the table's entries
        rows = sum(_counts(case)) * case["H"]
        return {"bytes": rows * (4 * D + 2 * D + 8) + 8 * B, "flops": rows * 4 * D}
    if case["op"] == "read":    # codes and scales in, bf16 out, zeros behind the end
        rows = sum(lens) * case["H"]
        return {"bytes": rows * (2 * D + 8) + B * case["S"] * case["H"] * 4 * D + 4 * B, "flops": rows * 2 * D}
    P, Sq, Hq, Hkv = case.get("prefix", 0), case["Sq"], case["Hq"], case["Hkv"]
    seen = 0
    for n in lens:
        seen += sum(max(0, P + n - Sq + 1 + i) for i in range(Sq)) if case["causal"] else Sq * (P + n)
    moved = (P + sum(lens)) * Hkv * (2 * D + 8) + B * Sq * Hq * (4 * D + 4) + 4 * B
    return {"bytes": moved, "flops": 4 * D * Hq * seen}


def exact(case, seed):
    s = prepare(case, seed)
    cache, table, lens = s["cache"], s["table"].tolist(), _lens(case)
    page = cache[0].shape[2]
    if case["op"] == "write":
        counts = _counts(case)
        for b in range(case["B"]):
            if counts[b] == 0:
                continue
            at = torch.arange(lens[b], lens[b] + counts[b], device="cuda")
            pg, off = s["table"][b].long()[at // page], at % page
            for x, codes, scale, top in ((s["k"], cache[0], cache[1], 127), (s["v"], cache[2], cache[3], 448)):
                x = x[b, :counts[b]].to(torch.float64)
                sc = (x.abs().max(dim=-1).values / top).to(torch.float32)
                quot = torch.nan_to_num(x / sc.to(torch.float64)[..., None]).to(torch.float32)   # the quotient is rounded to 32 bits
                scale[pg, :, off] = sc
                if top == 127:
                    codes[pg, :, off] = torch.round(quot).clamp(-127, 127).to(torch.int8)
                else:   # e4m3: steps of 2^-3 of the value's power of two, 2^-9 at the least
                    q = quot.to(torch.float64)
                    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
                    val = (torch.round(q / step) * step).clamp(-448, 448)
                    codes.view(torch.uint8)[pg, :, off] = val.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
        return cache

    def row(codes, scale, pages, n):
        pages = torch.tensor(pages[:-(-n // page)], dtype=torch.long, device="cuda")
        x = codes[pages].to(torch.float64) * scale[pages].to(torch.float64)[..., None]
        return x.permute(1, 0, 2, 3).reshape(codes.shape[1], -1, D)[:, :n]     # [H, n, D]

    B = case["B"]
    if case["op"] == "read":
        out = [torch.zeros((B, case["S"], case["H"], D), dtype=torch.float64, device="cuda") for _ in range(2)]
        for b in range(B):
            for o, (codes, scale) in zip(out, (cache[:2], cache[2:])):
                if lens[b]:
                    o[b, :lens[b]] = row(codes, scale, table[b], lens[b]).transpose(0, 1)
        return tuple(out)
    Sq, Hq, Hkv, P = case["Sq"], case["Hq"], case["Hkv"], case.get("prefix", 0)
    G = Hq // Hkv
    out = torch.zeros((B, Sq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    pre = [row(cache[i], cache[i + 1], s["prefix_table"].tolist(), P) for i in (0, 2)] if P else None
    for b in range(B):
        n = P + lens[b]
        if n == 0:
            continue
        k, v = (row(cache[i], cache[i + 1], table[b], lens[b]) for i in (0, 2)) if lens[b] else (None, None)
        if P:
            k, v = (pre[j] if t is None else torch.cat([pre[j], t], 1) for j, t in ((0, k), (1, v)))
        for h in range(Hq):
            x = (s["q"][b, :, h].to(torch.float64) @ k[h // G].T) * SCALE
            if case["causal"]:
                last = n - Sq + torch.arange(Sq, device="cuda")
                x = x.masked_fill(torch.arange(n, device="cuda") > last[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h] = z
            p = torch.where(torch.isinf(z)[:, None], torch.zeros_like(x), torch.exp(x - z[:, None]))
            out[b, :, h] = p @ v[h // G]
    return out, lse
