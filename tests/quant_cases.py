"""Helpers for the tests of 4-bit caches: the format in plain 64-bit torch, and batches over a
cache in it, whose attention the CPU oracle computes on the values that the cache stands for.

Tolerances on top of cache_cases': a weight is rounded to fp16: off by 2^-11 of it, and a weight below
fp16's normal numbers by half of their step of 2^-24: weights are held times 2^6 relative to a maximum that is
at most the row's true one, so its largest is 2^6 or more, and a small one is off by 2^-25 / 2^6 = 2^-31 of that.
A sum over n keys is off by n 2^-31 max|v| more (tiny(), which shows only where the keys of large
weights hold zeros).  Queries are taken to fp16 with 2^-39 of the row's largest element
lost at most.  Keys and values are exact in the products.
"""
import numpy as np
import torch

from cache_cases import LSE_TOL, SLACK, Case, np64

BF, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
CODES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def nearest(x, grid):
    """Index of the ascending grid's entry nearest to x >= 0, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    below, at = torch.searchsorted(mid, x.contiguous()), torch.searchsorted(mid, x.contiguous(), right=True)
    return torch.where(below == at, below, torch.where(below % 2 == 0, below, at))


def quantise(x, factor):
    """Codes [.., D / 2] and scale bytes [.., D / 16] of 64-bit rows x [.., D]."""
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(E4M3).double()
    e2m1 = torch.tensor(CODES, dtype=F64, device=x.device)
    y = x.unflatten(-1, (-1, 16))
    byte = nearest(y.abs().amax(-1) / (6 * factor), grid)
    step = (grid[byte] * factor)[..., None]
    code = torch.where(step > 0, nearest(y.abs() / torch.where(step > 0, step, 1.0), e2m1), 0)
    code = (code + 8 * ((y < 0) & (code > 0))).flatten(-2)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).to(torch.uint8), byte.to(torch.uint8)


def values(codes, scales, factor):
    """64-bit rows [.., D]; a zero of either sign is +0."""
    table = torch.tensor(CODES + [-x for x in CODES], dtype=F64, device=codes.device)
    x = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    return (x.unflatten(-1, (-1, 16)) * scales.view(E4M3).double()[..., None]).flatten(-2) * factor + 0.0


def arrays(n_pages, page, Hkv, D, layout, device="cuda"):
    """Codes [n_pages, page, Hkv, D / 2] and scales [n_pages, Hkv, page, D / 16], uint8."""
    u8 = dict(dtype=torch.uint8, device=device)
    if layout == "tokens":
        return torch.zeros(n_pages, page, Hkv, D // 2, **u8), torch.zeros(n_pages, Hkv, page, D // 16, **u8)
    if layout == "heads":
        return torch.zeros(n_pages, Hkv, page, D // 2, **u8).transpose(1, 2), torch.zeros(n_pages, Hkv, page, D // 16, **u8)
    # one array of pages: a head's codes, then its scales, then 16 bytes of something else
    both = torch.zeros(n_pages, Hkv, page * (D // 2 + D // 16) + 16, **u8)
    n = page * D // 2
    return both[:, :, :n].unflatten(2, (page, D // 2)).transpose(1, 2), both[:, :, n:-16].unflatten(2, (page, D // 16))


class QCase(Case):
    """A Case whose cache is held in 4 bits; self.Kc and self.Vc are the values it stands for."""

    def __init__(self, *a, factors=(1.0, 1.0), layout="heads", **kw):
        super().__init__(*a, dtype=BF, **kw)
        self.factors, self.held = factors, []
        g = torch.Generator(device=self.device).manual_seed(kw.get("seed", 0))
        for name, f in zip(("Kc", "Vc"), factors):
            x = getattr(self, name).double() * f
            undefined = torch.isnan(x[..., 0])                       # [n_pages, page, Hkv]
            codes, scales = arrays(self.n_pages, self.page, self.Hkv, self.D, layout, self.device)
            c, s = quantise(torch.nan_to_num(x), f)
            noise = torch.randint(0, 256, c.shape, generator=g, device=self.device, dtype=torch.uint8)
            codes.copy_(torch.where(undefined[..., None], noise, c))
            scales.copy_(torch.where(undefined[..., None], torch.tensor(0x7F, dtype=torch.uint8, device=self.device), s).transpose(1, 2))
            self.held.append((codes, scales))
            setattr(self, name, values(codes, scales.transpose(1, 2).contiguous(), f))

    def cache(self, jfa):
        (k, ks), (v, vs) = self.held
        return jfa.jfa_cache_create_quantized(k, v, ks, vs, *self.factors)

    def run(self, jfa, cache=None, **kw):
        return super().run(jfa, cache or self.cache(jfa), **kw)

    def tiny(self):
        return self.kv.max(initial=0) * 2.0 ** -31 * np.abs(np.nan_to_num(np64(self.Vc))).max()

    def check(self, O, lse, ref=None, slack=SLACK):
        ro, rl, A = ref or self.reference()
        o, l = np64(O)[:self.T], np64(lse)[:self.T]
        tol = slack * A + 2.0 ** -11 * A + self.tiny() + 1e-30
        if O.dtype == BF:
            tol = tol + 2.0 ** -8 * np.abs(ro)
        assert np.all(np.isfinite(o)), "non-finite output"
        assert (np.abs(o - ro) - tol).max(initial=-1.0) <= 0.0, f"O off by {(np.abs(o - ro) - tol).max()} more than the tolerance"
        fin = np.isfinite(rl)
        assert np.array_equal(fin, np.isfinite(l)) and np.all(l[~fin] == -np.inf)
        assert np.abs(l[fin] - rl[fin]).max(initial=0.0) <= LSE_TOL
