"""Helpers of the 4-bit cache's tests: a plain statement of its rows in float64
(no test functions here)."""
import math

import torch

from tests.cache_common import D

GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def nearest_code(y):
    """E2M1 magnitudes' codes of |y|: the nearest, ties to the even code, at most 7."""
    a = y.abs().clamp(max=6.0)
    dist = (a[..., None] - GRID).abs()
    best = dist.amin(-1, keepdim=True)
    tied = dist == best                                   # one, or two neighbours
    first = tied.float().argmax(-1)
    return torch.where((tied.sum(-1) == 2) & (first % 2 == 1), first + 1, first)


def e4m3(x):
    """fp32 values -> E4M3 bytes (round to nearest even; none is above 448)."""
    return x.to(torch.float8_e4m3fn)


def quantize4(x):
    """(codes uint8 [.., 64], blocks e4m3 [.., 8], scale fp32) of bf16 rows [.., 128]."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, torch.zeros_like(x))
    top = x.abs().amax(-1)
    k = torch.zeros_like(top)
    for i, t in enumerate(top.flatten().tolist()):
        e = -126
        while t > 2688.0 * 2.0 ** e:
            e += 1 if t <= 2688.0 * 2.0 ** (e + 8) else 8
        k.view(-1)[i] = e
    scale = torch.where(top == 0, torch.zeros_like(top), torch.exp2(k)).float()
    x = (x * torch.exp2(-k)[..., None]).unflatten(-1, (8, 16))
    blocks = e4m3((x.abs().amax(-1) / 6.0).float())
    sb = blocks.double()[..., None]
    y = torch.where(sb == 0, torch.zeros_like(x), x / sb).float().double()
    code = nearest_code(y) + 8 * torch.signbit(y).long()
    code = code.flatten(-2).unflatten(-1, (64, 2))
    scale = torch.where(finite, scale, torch.full_like(scale, math.nan))
    return (code[..., 0] | code[..., 1] << 4).to(torch.uint8), blocks, scale


def values4(codes, blocks):
    """float64 code * block of rows, without the rows' scales."""
    two = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = GRID[two & 7] * torch.where(two >= 8, -1.0, 1.0).double()
    return v * blocks.double().repeat_interleave(16, dim=-1)


class Cache4:
    """A CPU model of a paged 4-bit cache of normal data; NaN scales and blocks and odd
    codes where nothing is written."""

    def __init__(self, lens, H, page, seed, width=None, spare=2, recipe="normal", v_scale=None, k_scale=None, extra=()):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.page = list(lens), H, page
        need = [-(-n // page) for n in list(lens) + list(extra)]
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        width = max([1] + need) if width is None else width
        self.table = torch.full((len(need), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, H, page)
        self.t = [torch.full(shape + (64,), 0xF7, dtype=torch.uint8), torch.full(shape + (8,), 0x7F, dtype=torch.uint8),
                  torch.full(shape, math.nan)]
        self.t += [t.clone() for t in self.t]
        self.rows = []
        for b, n in enumerate(list(lens) + list(extra)):
            k = torch.randn((n, H, D), generator=g)
            v = torch.randn((n, H, D), generator=g)
            if recipe == "offset":
                k = k + 2 * torch.randn((1, H, D), generator=g)
            elif recipe == "sharp":        # a few keys take nearly all the weight
                k = k * torch.where(torch.rand((n, H, 1), generator=g) < 0.02, 12.0, 1.0)
            if v_scale is not None:
                v = v * v_scale(n, g)
            if k_scale is not None:
                k = k * k_scale(n, g)
            rows = quantize4(k.to(torch.bfloat16)) + quantize4(v.to(torch.bfloat16)) if n else None
            if n:
                p = self.table[b].long()[torch.arange(n) // page]
                for dst, src in zip(self.t, rows):
                    dst[p, :, torch.arange(n) % page] = src.view(torch.uint8) if src.element_size() == 1 else src
            self.rows.append(rows)

    def gpu(self, dev="cuda"):
        out = [t.to(dev) for t in self.t]
        out[1], out[4] = out[1].view(torch.float8_e4m3fn), out[4].view(torch.float8_e4m3fn)
        return tuple(out)

    def dense(self, b):
        """float64 (k codes * blocks, k scale, v codes * blocks, v scale) of a sequence."""
        if self.rows[b] is None:
            z = torch.zeros((0, self.H, D), dtype=torch.float64)
            return z, z[..., 0], z, z[..., 0]
        kc, kb, ks, vc, vb, vs = self.rows[b]
        return values4(kc, kb), ks.double(), values4(vc, vb), vs.double()
