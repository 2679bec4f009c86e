"""Timed cases of the operators around the paged KV cache: pages given to new
tokens, norms and rotary positions of Q and K, tokens put into the cache behind
them in the same pass, and a cache held in 4 bits with the attention over it.

A row of the 4-bit cache is one token of one key/value head: 128 E2M1 codes, two
to a byte (the even channel in the low half), an E4M3 scale for each 16 channels
and one power of two for the row:

    codes uint8 [pages, H, page, 64]   block e4m3 [pages, H, page, 8]   scale fp32 [pages, H, page]
    value = e2m1(code) * block * scale

    pages    request lengths -> pages off a free list, block tables, slots, positions
    rope     RMS norm of each head, then the rotation, of q and k: bf16 out
    append   the same, and k and v quantised and written to their slots; what was
             written is read back as bf16
    cache4   k and v written to a 4-bit cache and read back
    attn4    the newest Sq tokens attend to their sequences in a 4-bit cache,
             with prefix > 0 behind cached tokens that all of them share

With ``own`` false ``run`` computes them by elementary torch operations, with
``own`` true it calls the library.
"""
import math
import random

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6


def listed():
    return [
        # one new token for each running sequence: a generation step's bookkeeping
        dict(name="pages_step", op="pages", B=48, page=64, len_min=64, len_max=16384, new_min=1, new_max=1, lens=1, layout="packed", short=False),
        # prompts and chunks of unequal lengths side by side
        dict(name="pages_prompts", op="pages", B=256, page=16, len_min=0, len_max=2000, new_min=0, new_max=1531, lens=2, layout="packed", short=False),
        # a text encoder's tokens: half layout, one axis
        dict(name="rope_text", op="rope", B=2, S=333, Hq=24, Hk=24, R=128, interleaved=False, axes=1, scaling="none", norm=True, fused=False, lens=3),
        # a video's tokens, sliced out of one projection: time, height and width
        dict(name="rope_video", op="rope", B=1, S=32760, Hq=40, Hk=40, R=128, interleaved=True, axes=3, scaling="none", norm=True, fused=True, lens=4),
        # a generation step of a ragged batch, grouped heads, into 4 bits
        dict(name="append_step", op="append", bits=4, B=48, Hq=32, Hk=8, R=128, interleaved=False, scaling="none", norm=True, page=64,
             len_min=64, len_max=16384, new_min=1, new_max=1, lens=5),
        # packed prompts of unequal lengths, part of the head rotated, positions scaled, into 8 bits
        dict(name="append_prompts", op="append", bits=8, B=8, Hq=32, Hk=8, R=64, interleaved=False, scaling="yarn", norm=True, page=64,
             len_min=0, len_max=0, new_min=333, new_max=4096, lens=6),
        # a few short contexts
        dict(name="cache4_short", op="cache4", B=3, S=333, H=2, page=16, lens=7),
        # long contexts
        dict(name="cache4_long", op="cache4", B=4, S=16384, H=8, page=64, lens=8),
        # one sequence, one token, a short context: latency
        dict(name="attn4_step_one", op="attn4", B=1, Sq=1, Hq=32, Hkv=8, page=16, prefix=0, len_min=777, len_max=777, lens=9, causal=True),
        # a generation step of a ragged batch with grouped heads
        dict(name="attn4_step_batch", op="attn4", B=48, Sq=1, Hq=32, Hkv=8, page=64, prefix=0, len_min=64, len_max=16384, lens=10, causal=True),
        # a chunk of new tokens against what came before it
        dict(name="attn4_chunk", op="attn4", B=2, Sq=1000, Hq=16, Hkv=4, page=64, prefix=0, len_min=7000, len_max=9000, lens=11, causal=True),
        # many continuations of one long context
        dict(name="attn4_prefix", op="attn4", B=64, Sq=1, Hq=32, Hkv=8, page=64, prefix=16384, len_min=1, len_max=512, lens=12, causal=True),
    ]


def draw(rng):
    def over(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["pages", "rope", "append", "cache4", "attn4", "attn4"])
    case = dict(op=op, lens=rng.randrange(1 << 30))
    page = rng.choice([16, 32, 64, 128, 256])
    rope = dict(R=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                norm=rng.random() < 0.7)
    if op == "pages":
        B = over(1, 256)
        new = over(1, 1531)
        case.update(B=B, page=page, len_min=0, len_max=over(1, 16384), new_min=rng.choice([0, 1]), new_max=new,
                    layout=rng.choice(["packed", "front", "end"]), short=rng.random() < 0.2)
    elif op == "rope":
        Hq = over(1, 40)
        Hk = rng.choice([Hq, max(1, Hq // 4), 1])
        B, S = over(1, 8), over(1, 32760)
        S = max(1, min(S, (1 << 20) // (B * (Hq + Hk))))
        case.update(B=B, S=S, Hq=Hq, Hk=Hk, axes=rng.choice([1, 1, 2, 3]), fused=rng.random() < 0.5, **rope)
    elif op == "append":
        Hk, G = over(1, 16), rng.choice([1, 2, 4, 5, 8])
        bits = rng.choice([4, 8])
        B, new = over(1, 48), 1 if rng.random() < 0.5 else over(1, 4096)
        new = max(1, min(new, ((1 << 18) if bits == 8 else (1 << 10)) // (B * Hk * (G + 2) if bits == 8 else B * Hk)))
        case.update(bits=bits, B=B, Hq=Hk * G, Hk=Hk, page=page, len_min=0, len_max=over(1, 100000), new_min=rng.choice([0, 1, new]), new_max=new, **rope)
    elif op == "cache4":
        B, S, H = over(1, 32), over(1, 16384), over(1, 16)
        S = max(1, min(S, (1 << 19) // (B * H)))
        case.update(B=B, S=S, H=H, page=page)
    elif rng.random() < 0.6:
        Hkv, G = over(1, 16), rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        Sq = 1 if rng.random() < 0.5 else over(1, 1000)
        B, longest = over(1, 48), over(1, 65536)
        longest = max(Sq, min(longest, (1 << 21) // (B * Hkv), (1 << 27) // (B * Hkv * G * Sq)))
        B = max(1, min(B, (1 << 27) // (longest * Hkv * G * Sq)))
        case.update(B=B, Sq=Sq, Hq=Hkv * G, Hkv=Hkv, page=page, prefix=0, len_min=rng.choice([0, Sq]), len_max=longest, causal=rng.random() < 0.7)
    else:
        Hkv, G = over(1, 16), rng.choice([1, 2, 4, 5, 8])
        Sq, B, prefix = rng.choice([1, 1, 1, 2, 5, 8]), over(2, 64), over(50, 32760)
        prefix = max(1, min(prefix, (1 << 26) // (B * Hkv * G * Sq)))
        case.update(B=B, Sq=Sq, Hq=Hkv * G, Hkv=Hkv, page=page, prefix=prefix, len_min=rng.choice([0, Sq]), len_max=over(Sq, 512),
                    causal=rng.random() < 0.7)
    return case


def _lens(case):
    """Lengths of the sequences in the cache (for pages and append: before the new tokens)."""
    r = random.Random(case["lens"])
    if case["op"] == "cache4":
        return [r.randint(0, case["S"]) for _ in range(case["B"])]
    return [r.randint(case["len_min"], case["len_max"]) for _ in range(case["B"])]


def _counts(case):
    """New tokens of each sequence."""
    r = random.Random(case["lens"] + 1)
    return [r.randint(case["new_min"], case["new_max"]) for _ in range(case["B"])]


def _sections(case):
    """Pairs of channels of each axis."""
    n, axes = case["R"] // 2, case.get("axes", 1)
    if axes == 1:
        return [n]
    if axes == 2:
        return [n // 2, n - n // 2]
    return [n - 2 * (3 * n // 8), 3 * n // 8, 3 * n // 8]


def _scaling(case):
    return {"none": None, "linear": ("linear", 4.0), "ntk": ("ntk", 8.0), "yarn": ("yarn", 4.0, 32768), "bands": ("bands", 8.0, 8192)}[case["scaling"]]


def _frequencies(dim, base, scaling):
    """Radians a position of each pair of `dim` rotated channels, and the factor of sine and cosine."""
    kind = scaling[0] if scaling else "none"
    factor = scaling[1] if scaling else 1.0
    if kind == "ntk" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if kind == "linear":
        return [x / factor for x in f], 1.0
    if kind == "yarn":       # pairs that turn often in the original length stay, slow ones are stretched
        turns = [dim * math.log(scaling[2] / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        lo, hi = max(0, math.floor(turns[0])), min(dim - 1, math.ceil(turns[1]))
        ramp = [min(1.0, max(0.0, (i - lo) / max(1e-3, hi - lo))) for i in range(dim // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    if kind == "bands":      # by the wavelengths in the original length: below 1 stretched, above 4 kept
        keep = [min(1.0, max(0.0, (scaling[2] * x / (2 * math.pi) - 1.0) / 3.0)) for x in f]
        return [x / factor * (1 - k) + x * k for x, k in zip(f, keep)], 1.0
    return f, 1.0


def _all_frequencies(case):
    freqs, factor = [], 1.0
    for n in _sections(case):
        f, factor = _frequencies(2 * n, 10000.0, _scaling(case))
        freqs += f
    return freqs, factor


def _quantize4(x):
    """Codes (two to a byte), block scales and row scales of rows of 128."""
    x = x.double()
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    k = (e - 12 + (m > 0.65625)).clamp(min=-126)
    scale = torch.where(top == 0, torch.zeros_like(top), torch.exp2(k.double()))
    x = (x * torch.exp2(-k.double()).unsqueeze(-1)).view(x.shape[:-1] + (8, 16))
    block = (x.abs().amax(-1) / 6).float().to(torch.float8_e4m3fn)
    sb = block.double().unsqueeze(-1)
    y = torch.where(sb == 0, torch.zeros_like(x), x / sb).float()
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(y).byte()).view(x.shape[:-2] + (64, 2))
    return code[..., 0] | (code[..., 1] << 4), block, scale.float()


def _values4(codes, block, scale):
    """fp32 values of rows."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    pairs = torch.stack([codes & 15, codes >> 4], -1)
    y = grid[pairs.int()].view(codes.shape[:-1] + (8, 16)) * block.float().unsqueeze(-1)
    return y.view(codes.shape[:-1] + (D,)) * scale.unsqueeze(-1)


def _quantize8(x, levels):
    """Scales of rows of 128 and the quotients x / scale, both rounded once to 32 bits."""
    x = x.double()
    scale = (x.abs().amax(-1) / levels).float()
    y = (x / scale.double().unsqueeze(-1)).float()
    return scale, torch.where(scale.unsqueeze(-1) == 0, torch.zeros_like(y), y)


def _rows(x, bits, is_v):
    """What a cache of `bits` holds of rows x: the tensors of K or V."""
    if bits == 4:
        return _quantize4(x)
    scale, y = _quantize8(x, 448.0 if is_v else 127.0)
    return (y.clamp(-448, 448).to(torch.float8_e4m3fn) if is_v else y.round().clamp(-127, 127).to(torch.int8)), scale


def _put(cache, at, rows):
    for t, x in zip(cache, rows):
        t.view(torch.uint8 if t.element_size() == 1 else t.dtype)[at] = x.view(torch.uint8 if x.element_size() == 1 else x.dtype)


def _empty(pages, H, page, bits):
    shape = (pages, H, page)

    def zeros(n, dtype):
        return torch.zeros(shape + (n,), dtype=torch.uint8, device="cuda").view(dtype)

    out = []
    for dtype in (torch.int8, torch.float8_e4m3fn):
        out += [zeros(64, torch.uint8), zeros(8, torch.float8_e4m3fn)] if bits == 4 else [zeros(D, dtype)]
        out.append(torch.zeros(shape, device="cuda"))
    return tuple(out)


def _filled(gen, total, H, page, bits):
    """A cache as it stands after the writes of normal K and V, K with channel offsets as diffusion models have them."""
    cache = _empty(total, H, page, bits)
    offset = torch.randn((1, H, 1, D), generator=gen, device="cuda") * 2
    step = max(1, (1 << 24) // (H * page * D))
    for i in range(0, total, step):
        n = min(step, total - i)
        for is_v in (False, True):
            x = torch.randn((n, H, page, D), generator=gen, device="cuda")
            x = (x if is_v else x + offset).to(torch.bfloat16)
            half = len(cache) // 2
            _put(cache[half:] if is_v else cache[:half], slice(i, i + n), _rows(x, bits, is_v))
    return cache


def _tables(gen, need, page, width, spare):
    """A table of distinct pages in no order, -1 behind what a sequence needs, and the pages left over."""
    pages = torch.tensor([-(-n // page) for n in need], device="cuda")
    total = int(pages.sum()) + spare
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(1, width)
    live = torch.arange(width, device="cuda") < pages[:, None]
    table = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    table[live] = order[:total - spare]
    return table, total, order[total - spare:]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, B = case["op"], case["B"]
    lens = [] if op == "rope" else _lens(case)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    s = dict(case=dict(case))
    if op in ("rope", "append"):
        s["freqs"], s["factor"] = _all_frequencies(case)
        s["freq"] = torch.tensor(s["freqs"], dtype=torch.float64, device="cuda")
        s["q_weight"] = (1 + 0.2 * normal(D)).to(torch.bfloat16) if case["norm"] else None
        s["k_weight"] = (1 + 0.2 * normal(D)).to(torch.bfloat16) if case["norm"] else None
        if own:
            import quantized_attention_diffusion_gb300 as qad
            s["rope"] = qad.Rope(case["R"], 10000.0, interleaved=case["interleaved"], sections=_sections(case) if case.get("axes", 1) > 1 else None,
                                 scaling=_scaling(case))
    if op == "pages":
        page, counts = case["page"], _counts(case)
        need = [-(-(a + c) // page) - -(-a // page) for a, c in zip(lens, counts)]
        free = sum(need) // 2 if case["short"] else sum(need) + 40
        width = max(1, max(-(-(a + c) // page) for a, c in zip(lens, counts)))
        s["table"], s["num_pages"], left = _tables(gen, lens, page, width, max(1, free))
        s["free_pages"] = torch.full((s["num_pages"],), -1, dtype=torch.int32, device="cuda")
        s["free_pages"][:left.numel()] = left
        s["free_count"] = ints([free])
        s["lens"], s["counts"] = ints(lens), ints(counts)
        s["tokens"] = max(1, sum(counts)) if case["layout"] == "packed" else max(1, max(counts))
        return s
    if op == "rope":
        S, Hq, Hk = case["S"], case["Hq"], case["Hk"]
        if case["fused"]:      # q, k and v heads of one projection
            qkv = normal(B, S, Hq + 2 * Hk, D)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
        else:
            s["q"], s["k"] = normal(B, S, Hq, D), normal(B, S, Hk, D)
        r = random.Random(case["lens"])
        i = torch.arange(S, device="cuda", dtype=torch.int32)
        if case["axes"] == 1:
            pos = (ints([r.randint(0, 100000) for _ in range(B)])[:, None] + i).unsqueeze(-1)
        else:                  # frames of rows of tokens, the same for each of the batch
            w = max(1, int(math.sqrt(S / 13)))
            axes = [i // w, i % w] if case["axes"] == 2 else [i // (w * w), i // w % w, i % w]
            pos = torch.stack(axes, -1).expand(B, -1, -1)
        s["positions"] = pos.contiguous()
        return s
    page = case["page"]
    if op == "append":
        counts = _counts(case)
        first = [a % page for a in lens]                       # tokens that the first page holds already
        need = [f + c for f, c in zip(first, counts)]
        width = -(-max(need + [1]) // page)
        s["table"], total, _ = _tables(gen, need, page, width, 3)
        s["cache"] = _filled(gen, total, case["Hk"], page, case["bits"])
        s["read_lens"], s["read"] = ints(need), max(need + [1])
        seq = [b for b, c in enumerate(counts) for _ in range(c)] or [0]
        i = [j for c in counts for j in range(c)] or [0]
        seq, i = ints(seq).long(), ints(i)
        at = ints(first)[seq] + i
        s["slots"] = s["table"][seq, (at // page).long()] * page + at % page if sum(counts) else ints([-1])
        s["positions"] = ints(lens)[seq] + i
        T = len(seq)
        qkv = normal(1, T, case["Hq"] + 2 * case["Hk"], D)
        s["q"], s["k"], s["v"] = qkv.split([case["Hq"], case["Hk"], case["Hk"]], dim=2)
        return s
    if op == "cache4":
        S, H = case["S"], case["H"]
        s["table"], total, _ = _tables(gen, lens, page, -(-S // page), 3)
        s["cache"] = _empty(total, H, page, 4)
        s["k"], s["v"] = normal(B, S, H, D), normal(B, S, H, D)
        s["start"], s["lens"] = ints([0] * B), ints(lens)
        return s
    s["lens"], s["longest"] = ints(lens), max([1] + lens)
    s["q"] = normal(B, case["Sq"], case["Hq"], D)
    width, P = -(-max(lens) // page), case["prefix"]
    if P:
        both, total, _ = _tables(gen, lens + [P], page, max(width, -(-P // page)), 3)
        s["table"] = both[:B, :max(1, width)].contiguous()
        s["prefix_table"] = both[B, :-(-P // page)].contiguous()
    else:
        s["table"], total, _ = _tables(gen, lens, page, width, 3)
    s["cache"] = _filled(gen, total, case["Hkv"], page, 4)
    return s


# --------------------------------------------------------------- plain form --

def _pages(s):
    case = s["case"]
    page, layout, T = case["page"], case["layout"], s["tokens"]
    B, width = s["table"].shape
    lens, counts, free = s["lens"].long(), s["counts"].long(), s["free_count"].long()
    held = (lens + page - 1) // page
    need = (lens + counts + page - 1) // page - held
    upto = need.cumsum(0)
    served = (need == 0) | (upto <= free)
    taken = torch.where(served, counts, 0)
    gone = torch.where(served & (need > 0), upto, 0).amax()
    j = torch.arange(width, device="cuda") - held[:, None]
    new = served[:, None] & (j >= 0) & (j < need[:, None])
    at = (free - 1 - (upto - need)[:, None] - j).clamp(min=0, max=s["free_pages"].numel() - 1)
    table = torch.where(new, s["free_pages"][at], s["table"])
    s["table"].copy_(table)
    if layout == "packed":
        r = torch.arange(T, device="cuda")
        ends = counts.cumsum(0)
        b = torch.searchsorted(ends, r, right=True)
        live = b < B
        b = b.clamp(max=B - 1)
        i = r - (ends - counts)[b]
    else:
        b = torch.arange(B, device="cuda")[:, None].expand(B, T).reshape(-1)
        i = torch.arange(T, device="cuda").repeat(B)
        if layout == "end":
            i = i - (T - counts[b])
        live = (i >= 0) & (i < counts[b])
    live &= served[b]
    pos = torch.where(live, lens[b] + i, 0)
    slots = torch.where(live, table[b, (pos // page).clamp(max=width - 1)].long() * page + pos % page, -1)
    return dict(start=s["lens"], taken=taken.int(), lens=(lens + taken).int(), free_count=(free - gone).int(), table=s["table"],
                slots=slots.int(), positions=pos.int())


def _turned(s, x, weight, dtype):
    """Norm and rotation of x [B, S, H, 128], computed in `dtype`."""
    case = s["case"]
    R = case["R"]
    x = x.to(dtype)
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(dtype)
    axis = torch.tensor([a for a, n in enumerate(_sections(case)) for _ in range(n)], device="cuda")
    pos = s["positions"].view(x.shape[:2] + (-1,))[..., axis]
    angle = pos.double() * s["freq"]
    cos, sin = ((f(angle) * s["factor"]).to(dtype).unsqueeze(2) for f in (torch.cos, torch.sin))
    y = x[..., :R]
    if case["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :R // 2], y[..., R // 2:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., R:]], -1).to(torch.bfloat16)


def _gather(cache, table, L):
    """fp32 [B, H, L, 128] of the first L positions of each row of the table, of K's or V's tensors."""
    H, page = cache[0].shape[1:3]
    pages = table[:, :-(-L // page)].clamp(min=0).long()
    t = [x[pages] for x in cache]
    x = _values4(*t) if len(t) == 3 else t[0].float() * t[1].unsqueeze(-1)
    return x.transpose(1, 2).reshape(table.shape[0], H, -1, D)[:, :, :L]


def _read(cache, table, lens, S):
    """bf16 [B, S, H, 128] of K and V, zeros behind a sequence's end."""
    dead = torch.arange(S, device="cuda") >= lens[:, None]
    half = len(cache) // 2
    return [_gather(c, table, S).transpose(1, 2).to(torch.bfloat16).masked_fill(dead[:, :, None, None], 0) for c in (cache[:half], cache[half:])]


def _append(s):
    case, cache, slots = s["case"], s["cache"], s["slots"].long()
    page, half = case["page"], len(s["cache"]) // 2
    q = _turned(s, s["q"], s["q_weight"], torch.float32)
    k = _turned(s, s["k"], s["k_weight"], torch.float64)         # near a border of its codes
    live = slots >= 0
    at = (slots[live] // page, slice(None), slots[live] % page)
    for x, c, is_v in ((k, cache[:half], False), (s["v"], cache[half:], True)):
        _put(c, at, _rows(x[0][live], case["bits"], is_v))
    return [q] + _read(cache, s["table"], s["read_lens"], s["read"])


def _cache4(s):
    case, cache = s["case"], s["cache"]
    page, S = case["page"], case["S"]
    i = torch.arange(S, device="cuda")
    live = i < s["lens"][:, None]
    pages = s["table"].long()[:, i // page]
    at = (pages[live], slice(None), (i % page).expand(case["B"], -1)[live])
    for x, c in ((s["k"], cache[:3]), (s["v"], cache[3:])):
        _put(c, at, _quantize4(x[live]))
    return _read(cache, s["table"], s["lens"], S)


def _attn(s):
    case, cache, q = s["case"], s["cache"], s["q"]
    B, Sq, Hq, Hkv, P, L = case["B"], case["Sq"], case["Hq"], case["Hkv"], case["prefix"], s["longest"]
    G = Hq // Hkv
    rows = q.float().view(B, Sq, Hkv, G, D).permute(0, 2, 1, 3, 4)            # [B, Hkv, Sq, G, D]
    k, v = (_gather(c, s["table"], L) for c in (cache[:3], cache[3:]))
    x = rows.reshape(B, Hkv, Sq * G, D) @ k.transpose(2, 3)
    if P:
        pk, pv = (_gather(c, s["prefix_table"][None], P)[0] for c in (cache[:3], cache[3:]))
        px = rows.permute(1, 0, 2, 3, 4).reshape(Hkv, B * Sq * G, D) @ pk.transpose(1, 2)
        x = torch.cat([px.view(Hkv, B, Sq * G, P).transpose(0, 1), x], dim=-1)
    last = s["lens"].long()[:, None] + P
    last = (last - Sq + 1 + torch.arange(Sq, device="cuda")).clamp(min=0) if case["causal"] else last.expand(-1, Sq)
    sees = torch.arange(P + L, device="cuda") < last[:, :, None]                # [B, Sq, P + L]
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


def _run_own(s):
    import quantized_attention_diffusion_gb300 as qad

    case, op = s["case"], s["case"]["op"]
    if op == "pages":
        r = qad.kv_pages_reserve(s["free_pages"], s["free_count"], s["lens"], s["counts"], s["table"], case["page"], s["tokens"], case["layout"])
        slots, positions = (r.slots, r.positions) if case["layout"] == "packed" else (r.slots.view(-1), r.positions.view(-1))
        return dict(start=r.start, taken=r.taken, lens=r.lens, free_count=r.free_count, table=s["table"], slots=slots, positions=positions)
    if op == "rope":
        return qad.qk_norm_rope(s["q"], s["k"], s["rope"], s["positions"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                eps=EPS if case["norm"] else None)
    if op == "append":
        q = qad.kv_cache_append(s["q"], s["k"], s["v"], s["cache"], s["slots"], rope=s["rope"], positions=s["positions"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS if case["norm"] else None)
        return [q, *qad.kv_cache_read(s["cache"], s["table"], s["read_lens"], s["read"])]
    if op == "cache4":
        qad.kv_cache_write(s["k"], s["v"], s["cache"], s["table"], s["start"], s["lens"])
        return qad.kv_cache_read(s["cache"], s["table"], s["lens"], case["S"])
    if case["prefix"]:
        return qad.attn_fwd_cache_prefix(s["q"], s["cache"], s["prefix_table"], case["prefix"], s["table"], s["lens"], causal=case["causal"],
                                         return_lse=True)
    return qad.attn_fwd_cache(s["q"], s["cache"], s["table"], s["lens"], causal=case["causal"], return_lse=True)


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state)
    if op == "pages":
        return _pages(state)
    if op == "rope":
        return [_turned(state, state[x], state[x + "_weight"], torch.float32) for x in ("q", "k")]
    if op == "append":
        return _append(state)
    if op == "cache4":
        return _cache4(state)
    return _attn(state)


# --------------------------------------------------------- work and 64 bits --

def work(case):
    op, B = case["op"], case["B"]
    lens = [] if op == "rope" else _lens(case)
    if op == "pages":        # lengths, counts; start, taken, new lengths; the new pages; a slot and a position a token
        counts, page = _counts(case), case["page"]
        need = sum(-(-(a + c) // page) - -(-a // page) for a, c in zip(lens, counts))
        rows = sum(counts) if case["layout"] == "packed" else B * max(1, max(counts))
        return {"bytes": 20 * B + 8 * need + 8 * max(1, rows) + 8, "flops": 4 * max(1, rows)}
    if op == "rope":         # bf16 in and out, positions
        rows = B * case["S"] * (case["Hq"] + case["Hk"])
        return {"bytes": rows * 4 * D + 4 * B * case["S"] * case["axes"], "flops": rows * (4 * D + 3 * case["R"])}
    row8, row4 = 2 * D + 8, 2 * (64 + 8 + 4)
    if op == "append":       # q in and out, k and v in, their rows out; those of the pages read back
        counts, row = _counts(case), row8 if case["bits"] == 8 else row4
        need = [a % case["page"] + c for a, c in zip(lens, counts)]
        T, Hq, Hk = max(1, sum(counts)), case["Hq"], case["Hk"]
        back = sum(need) * Hk * row + B * max(need + [1]) * Hk * 4 * D
        return {"bytes": T * (Hq * 4 * D + Hk * (4 * D + row) + 8) + back, "flops": T * (Hq + Hk) * (4 * D + 3 * case["R"])}
    if op == "cache4":       # bf16 in, rows out, rows in, bf16 and zeros out
        rows = sum(lens) * case["H"]
        return {"bytes": rows * (4 * D + 2 * row4) + B * case["S"] * case["H"] * 4 * D + 4 * B, "flops": rows * 6 * D}
    P, Sq, Hq, Hkv = case["prefix"], case["Sq"], case["Hq"], case["Hkv"]
    seen = 0
    for n in lens:
        seen += sum(max(0, P + n - Sq + 1 + i) for i in range(Sq)) if case["causal"] else Sq * (P + n)
    return {"bytes": (P + sum(lens)) * Hkv * row4 + B * Sq * Hq * (4 * D + 4) + 4 * B, "flops": 4 * D * Hq * max(1, seen)}


def _decoded(parts, f64=torch.float64):
    """Values in 64 bits of a row's tensors."""
    if len(parts) == 2:
        return parts[0].to(f64) * parts[1].to(f64)[..., None]
    codes, block, scale = parts
    two = torch.stack((codes % 16, codes // 16), dim=-1).flatten(-2).to(f64)
    sign, mag = 1 - 2 * torch.floor(two / 8), two % 8
    e, m = torch.floor(mag / 2), mag % 2
    val = sign * torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e - 1))
    return val * block.to(f64).repeat_interleave(16, dim=-1) * scale.to(f64)[..., None]


def _held(x, bits, is_v):
    """What rows x (64 bits) read back as, by the cache's definition."""
    top = x.abs().max(dim=-1, keepdim=True).values
    one = torch.ones_like(top)
    if bits == 8:
        sc = (top / (448 if is_v else 127)).float().double()
        y = torch.where(sc == 0, 0 * x, x / torch.where(sc == 0, one, sc)).float().double()
        if not is_v:
            return torch.round(y).clamp(-127, 127) * sc
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        return (torch.round(y / step) * step).clamp(-448, 448) * sc
    k = torch.ceil(torch.log2(torch.where(top == 0, one, top) / 2688))
    k = torch.where(top > 2688 * torch.exp2(k), k + 1, torch.where(top <= 2688 * torch.exp2(k - 1), k - 1, k)).clamp(min=-126)
    x = (x * torch.exp2(-k)).unflatten(-1, (8, 16))
    t = (x.abs().amax(-1, keepdim=True) / 6).float().double()
    step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    sb = torch.round(t / step) * step
    y = torch.where(sb == 0, 0 * x, x / torch.where(sb == 0, torch.ones_like(sb), sb)).float().double()
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=1.0))) - 1)          # 1/2 up to 2, 1 up to 4, 2 up to 6
    y = (torch.round(y / step) * step).clamp(-6, 6)
    return (y * sb).flatten(-2) * torch.exp2(k)


def _spun(s, x, weight):
    """Norm and rotation in 64 bits, a complex product for each pair."""
    case, R = s["case"], s["case"]["R"]
    x = x.to(torch.float64)
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.to(torch.float64)
    B, S, H = x.shape[:3]
    pos = s["positions"].reshape(B, S, -1).to(torch.float64)
    angles = torch.cat([pos[..., a:a + 1] * s["freq"][sum(_sections(case)[:a]):sum(_sections(case)[:a + 1])] for a in range(len(_sections(case)))], -1)
    turn = torch.polar(torch.full_like(angles, s["factor"]), angles)[:, :, None]
    y = x[..., :R]
    pairs = y.unflatten(-1, (R // 2, 2)) if case["interleaved"] else y.unflatten(-1, (2, R // 2)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _exact_pages(case, s):
    page, free = case["page"], int(s["free_count"][0])
    pool, table = s["free_pages"].tolist(), s["table"].tolist()
    lens, counts = _lens(case), _counts(case)
    asked = gone = 0
    start, taken, slots, positions = [], [], [], []
    T = s["tokens"]
    for b, (a, c) in enumerate(zip(lens, counts)):
        have, want = -(-a // page), -(-(a + c) // page)
        asked += want - have
        ok = want == have or asked <= free
        if ok and want > have:
            for j in range(want - have):
                table[b][have + j] = pool[free - 1 - (asked - (want - have) + j)]
            gone = asked
        start.append(a)
        taken.append(c if ok else 0)
        mine = [table[b][p // page] * page + p % page if ok else -1 for p in range(a, a + c)]
        where = [p if ok else 0 for p in range(a, a + c)]
        pad = 0 if case["layout"] == "packed" else T - c
        front = case["layout"] == "end"
        slots += [-1] * (pad * front) + mine + [-1] * (pad * (not front))
        positions += [0] * (pad * front) + where + [0] * (pad * (not front))
    if case["layout"] == "packed":
        slots += [-1] * (T - len(slots))
        positions += [0] * (T - len(positions))
    as_ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(start=as_ints(start), taken=as_ints(taken), lens=as_ints([a + t for a, t in zip(start, taken)]), free_count=as_ints([free - gone]),
                table=as_ints(table), slots=as_ints(slots), positions=as_ints(positions))


def exact(case, seed):
    s = prepare(case, seed)
    op, B, f64 = case["op"], case["B"], torch.float64
    if op == "pages":
        return _exact_pages(case, s)
    if op == "rope":
        return [_spun(s, s["q"], s["q_weight"]), _spun(s, s["k"], s["k_weight"])]
    page, cache = case["page"], s["cache"]
    half = len(cache) // 2
    if op == "append":
        q = _spun(s, s["q"], s["q_weight"])
        k = _spun(s, s["k"], s["k_weight"]).to(torch.bfloat16).to(f64)            # K enters its codes as bf16
        out = []
        for x, parts, is_v in ((k, cache[:half], False), (s["v"].to(f64), cache[half:], True)):
            held = _decoded(parts)
            for t, slot in enumerate(s["slots"].tolist()) if len(s["slots"]) <= 64 else ():
                if slot >= 0:
                    held[slot // page, :, slot % page] = _held(x[0, t], case["bits"], is_v)
            if len(s["slots"]) > 64:
                held[torch.div(s["slots"], page, rounding_mode="floor").long(), :, (s["slots"] % page).long()] = _held(x[0], case["bits"], is_v)
            back = torch.zeros((B, s["read"]) + (case["Hk"], D), dtype=f64, device="cuda")
            for b, n in enumerate(s["read_lens"].tolist()):
                rows = held[s["table"][b, :-(-n // page)].long()].permute(0, 2, 1, 3).flatten(0, 1)
                back[b, :n] = rows[:n]
            out.append(back)
        return [q] + out
    lens = _lens(case)
    if op == "cache4":
        out = []
        for x in (s["k"], s["v"]):
            y = _held(x.to(f64), 4, False)
            for b, n in enumerate(lens):
                y[b, n:] = 0
            out.append(y)
        return out
    Sq, Hq, Hkv, P = case["Sq"], case["Hq"], case["Hkv"], case["prefix"]
    G = Hq // Hkv

    def rows(parts, pages, n):
        pages = pages[:-(-n // page)].long()
        return _decoded([t[pages] for t in parts]).permute(1, 0, 2, 3).flatten(1, 2)[:, :n]

    out = torch.zeros((B, Sq, Hq, D), dtype=f64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=f64, device="cuda")
    before = [rows(c, s["prefix_table"], P) for c in (cache[:3], cache[3:])] if P else None
    for b in range(B):
        n = P + lens[b]
        if n == 0:
            continue
        k, v = (rows(c, s["table"][b], lens[b]) for c in (cache[:3], cache[3:])) if lens[b] else (None, None)
        if P:
            k, v = (before[j] if t is None else torch.cat([before[j], t], 1) for j, t in ((0, k), (1, v)))
        for h in range(Hq):
            x = (s["q"][b, :, h].to(f64) @ k[h // G].T) * SCALE
            if case["causal"]:
                x = x.masked_fill(torch.arange(n, device="cuda") > (n - Sq + torch.arange(Sq, device="cuda"))[:, None], -math.inf)
            z = torch.logsumexp(x, -1)
            lse[b, h] = z
            out[b, :, h] = torch.where(torch.isinf(z)[:, None], torch.zeros_like(x), torch.exp(x - z[:, None])) @ v[h // G]
    return out, lse
