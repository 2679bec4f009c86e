"""Helpers of the KV cache tests: a plain statement of the cache and of the
attention over it in float64, and the bounds that the GPU's results are held to
(no test functions here)."""
import math

import torch

D = 128


def quantize_rows(x, top):
    """(scale fp32, fp32 quotients) of bf16 rows [..., 128]: scale = fl(amax / top),
    quotient fl(x / scale); a double quotient rounded to fp32 is the fp32
    quotient.  Non-finite rows: NaN and zeros."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    amax = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(-1)
    scale = (amax / top).float()
    y = (torch.where(finite[..., None], x, torch.zeros_like(x)) / scale.double()[..., None]).float()
    y = torch.where((scale == 0)[..., None], torch.zeros_like(y), y)
    scale = torch.where(finite, scale, torch.full_like(scale, math.nan))
    return scale, y


def quantize_kv(k, v):
    """(k_codes int8, k_scale, v_codes e4m3, v_scale) of rows [..., 128]."""
    ks, ky = quantize_rows(k, 127.0)
    vs, vy = quantize_rows(v, 448.0)
    return ky.round().clamp(-127, 127).to(torch.int8), ks, vy.clamp(-448, 448).to(torch.float8_e4m3fn), vs


class Cache:
    """A CPU model of a paged cache whose contents are random codes of normal
    data; ``fill`` puts NaN and the E4M3 NaN code where nothing is written."""

    def __init__(self, lens, H, page, seed, width=None, spare=2, recipe="normal", v_scale=None, extra=()):
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
        shape = (self.num_pages, H, page, D)
        self.k_codes = torch.full(shape, -128, dtype=torch.int8)
        self.v_codes = torch.full(shape, 0x7F, dtype=torch.uint8)
        self.k_scale = torch.full(shape[:3], math.nan)
        self.v_scale = torch.full(shape[:3], math.nan)
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
            codes = quantize_kv(k.to(torch.bfloat16), v.to(torch.bfloat16))
            self.put(b, codes)
            self.rows.append(codes)

    def put(self, b, codes):
        kc, ks, vc, vs = codes
        for i in range(kc.shape[0]):
            p, o = int(self.table[b, i // self.page]), i % self.page
            self.k_codes[p, :, o] = kc[i]
            self.k_scale[p, :, o] = ks[i]
            self.v_codes[p, :, o] = vc[i].view(torch.uint8)
            self.v_scale[p, :, o] = vs[i]

    def gpu(self, dev="cuda"):
        return (self.k_codes.to(dev), self.k_scale.to(dev), self.v_codes.to(dev).view(torch.float8_e4m3fn),
                self.v_scale.to(dev))

    def dense(self, b):
        """float64 (k codes, k scale, v codes, v scale) of a sequence, [n, H, 128] and [n, H]."""
        kc, ks, vc, vs = self.rows[b]
        return kc.double(), ks.double(), vc.float().double(), vs.double()


def join(a, b):
    return tuple(torch.cat([x, y]) for x, y in zip(a, b))


def reference(q, rows, causal, scale):
    """q bf16 [Sq, Hq, 128] over dense rows (codes and scales, n keys): (out,
    lse, bound of |out error|, bound of |lse error|) in float64.

    The bounds, term by term (u = 2^-24):
      scores   x = fp32 sum of 128 exact products, two products by scales: at
               most (128 + 4) u relative to the sum of magnitudes X (the tensor
               core may truncate its partial sums, hence 2u each), so
               dx <= 264 u X, and a running maximum near x costs one rounding
               more of |x|: 2 u X
      weights  ex2.approx: 2^-22 relative; a rounding of 2^-11 to fp16, or
               2^-25 of the largest weight times scale if smaller; log2 of the
               scale: 2^-22 absolute and a rounding of |x| + |log2 sv|
      sums     fp32, n keys: n 2u of the sum of magnitudes at the most
      out      one rounding to bf16: 2^-8 of |out|
    """
    u = 2.0 ** -24
    kc, ks, vc, vs = rows
    Sq, Hq, _ = q.shape
    n, H = kc.shape[0], kc.shape[1]
    G = Hq // H
    out = torch.zeros((Sq, Hq, D), dtype=torch.float64)
    lse = torch.full((Hq, Sq), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(out)
    ltol = torch.zeros_like(lse)
    if n == 0:
        return out, lse, tol, ltol
    qd = q.double()
    seen = torch.arange(n)[None, :] <= (n - Sq + torch.arange(Sq))[:, None] if causal else torch.ones((Sq, n), dtype=torch.bool)
    for h in range(Hq):
        g = h // G
        k = kc[:, g] * ks[:, g, None]
        v = vc[:, g] * vs[:, g, None]
        x = (qd[:, h] @ k.T * scale).masked_fill(~seen, -math.inf)
        mag = qd[:, h].abs() @ k.abs().T * scale
        z = torch.logsumexp(x, -1)
        lse[h] = z
        live = torch.isfinite(z)
        p = torch.where(seen & live[:, None], torch.exp(x - torch.where(live, z, torch.zeros_like(z))[:, None]), torch.zeros_like(x))
        pv = torch.where((p > 0)[:, :, None], v[None], torch.zeros_like(v)[None]) if not torch.isfinite(v).all() else None
        out[:, h] = torch.einsum("sn,snd->sd", p, pv) if pv is not None else p @ v
        vabs = torch.nan_to_num(v.abs(), nan=0.0)
        mass = p @ vabs
        dx = 266 * u * torch.where(seen, mag, torch.zeros_like(mag)).amax(-1)
        dlog = (torch.log2(torch.nan_to_num(vs[:, g], nan=1.0).clamp(min=2.0 ** -140)).abs().amax() + 64) * 2 * u
        rel = 2 * dx + 2.0 ** -21 + 2.0 ** -11 + 2 * n * u + dlog
        largest = (p * torch.nan_to_num(vs[:, g], nan=0.0)[None]).amax(-1)
        tol[:, h] = 2.0 ** -8 * out[:, h].abs() + rel[:, None] * mass + 2.0 ** -25 * largest[:, None] * vc[:, g].abs().sum(0)[None]
        ltol[h] = 2 * dx + 2.0 ** -20 + 2 * n * u + torch.where(live, z, torch.zeros_like(z)).abs() * 4 * u
    return out, lse, tol, ltol


def assert_within(got, ref, tol, what=""):
    got = got.double().cpu()
    same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    err = torch.where(same, torch.zeros_like(ref), (got - ref).abs())
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(int(t) for t in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound; first at {i}: "
                             f"{got[i].item()} for {ref[i].item()}, bound {tol[i].item():.3g}")


def ints(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")
