"""Helpers for the paged-cache tests: random batches with their pages dealt out in random
order, and the same attention by the CPU oracle (64 bits) on the gathered rows.

Tolerances.  A rounding to a type is off by at most half a step, relative to the value:
2^-8 for bf16, 2^-24 for fp32.  With A = sum_j p_j |v_j| (the oracle's output on |V|):
  bf16 cache, fp32 output:  2^-8 A from rounding each p_j to bf16 before P V, plus SLACK A;
  bf16 output:              2^-8 |o| more;
  fp32 cache:               SLACK A, and in rows of moderate scores FP32_SLACK A.
SLACK = 1e-4 covers what fp32 arithmetic adds.  A score of D <= 128 products sums with an
error of at most D 2^-24 sum|q k| scale, for N(0,1) inputs about 128 * 6e-8 * 128 * 0.64 /
11.3 = 5.5e-5 in the worst order (bf16 products are exact in fp32, their sum is not); the
exponential turns an error e of the score into a relative error e of p_j, and sums over n
keys in any tree of fp32 additions stay well inside the rest.  The lse is off by at most the
scores' error: LSE_TOL = 1e-4.
FP32_SLACK = 2e-5 for N(0,1) inputs and D <= 64: a score's terms sum to 64 * 0.64 / 8 = 5.1 in
magnitude; a plain fp32 sum of 64 products, or the tensor core's (products of split operands
exact to 2^-24, so 3e-7 in all, and at most 8 roundings of a full-size accumulator, each below
2^-23 of it), is off by less than 3e-7 + 8 * 2^-23 * 5.1 = 5.2e-6 natural units, so p by 5.2e-6
and its normalised weight by twice that; the exponential (2^-22), the products of split P and V
(2^-24), 8 roundings of 2^-23 in a tile's output and 2^-24 for each of the tiles added add less
than 4e-6.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle

FP32_SLACK = 2e-5
SLACK = 1e-4
LSE_TOL = 1e-4


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Case:
    """A batch over a paged cache.  layout: "tokens" [n_pages, page, Hkv, D], "heads"
    [n_pages, Hkv, page, D] or "both" (K and V interleaved in one array, page by page)."""

    def __init__(self, q_lens, kv_lens, *, H, Hkv, D, page, dtype=torch.bfloat16, causal=True, window=None,
                 bias=False, seed=0, layout="tokens", pad_rows=0, unset=True, device="cuda", std=1.0):
        g = torch.Generator(device=device).manual_seed(seed + 77)
        q, kv = np.asarray(q_lens, np.int64), np.asarray(kv_lens, np.int64)
        self.q, self.kv, self.H, self.Hkv, self.D, self.page = q, kv, H, Hkv, D, page
        self.dtype, self.causal, self.window, self.device = dtype, causal, window, device
        B = q.size
        need = -(-kv // page)
        n_pages = int(need.sum()) + 2
        self.n_pages = n_pages

        def normal(*s):
            return (torch.randn(*s, generator=g, device=device, dtype=torch.float32) * std).to(dtype)

        if layout == "tokens":
            self.Kc, self.Vc = normal(n_pages, page, Hkv, D), normal(n_pages, page, Hkv, D)
        elif layout == "heads":
            self.Kc = normal(n_pages, Hkv, page, D).permute(0, 2, 1, 3)
            self.Vc = normal(n_pages, Hkv, page, D).permute(0, 2, 1, 3)
        else:
            both = normal(n_pages, 2, page, Hkv, D)
            self.Kc, self.Vc = both[:, 0], both[:, 1]
        order = torch.randperm(n_pages, generator=g, device=device).cpu().numpy()
        width = max(1, int(need.max()) if B else 1) + 1
        table = np.full((B, width), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        if unset:  # what no row may see is undefined: NaN slots, unset pages
            seen = np.zeros((n_pages, page), bool)
            for b in range(B):
                lo = 0
                if window is not None and q[b] > 0:
                    lo = max(0, int(kv[b] - q[b]) - window)
                p = np.arange(lo, kv[b])
                seen[table[b, p // page], p % page] = True
            hidden = torch.from_numpy(~seen).to(device)
            self.Kc[hidden] = float("nan")
            self.Vc[hidden] = float("nan")
            if window is not None:
                for b in range(B):
                    lo = max(0, int(kv[b] - q[b]) - window) if q[b] > 0 else 0
                    table[b, :lo // page] = -1
        T = int(q.sum())
        self.T = T
        self.Q = normal(T + pad_rows, H, D)
        self.bias = torch.randn(H, 32, generator=g, device=device, dtype=torch.float32) * 0.5 if bias else None
        self.q_off = torch.tensor(np.concatenate([[0], np.cumsum(q)]), dtype=torch.int32, device=device)
        self.kv_lens = torch.tensor(kv, dtype=torch.int32, device=device)
        self.table = torch.from_numpy(table).to(device)
        self.host_table = table

    def gathered(self, which):
        """[sum kv, Hkv, D] in 64 bits, unseen positions 0."""
        c = np64(which)
        rows = []
        for b in range(self.q.size):
            p = np.arange(self.kv[b])
            pages = self.host_table[b, p // self.page]
            r = c[np.maximum(pages, 0), p % self.page]
            r[pages < 0] = 0.0
            rows.append(np.nan_to_num(r, nan=0.0))
        return np.concatenate(rows) if rows else np.zeros((0, self.Hkv, self.D))

    def reference(self):
        """(O, lse, A) of the oracle; A = sum_j p_j |v_j|."""
        g = self.H // self.Hkv
        kv_off = np.concatenate([[0], np.cumsum(self.kv)]).astype(np.int32)
        q_off = np.concatenate([[0], np.cumsum(self.q)]).astype(np.int32)
        K, V = np.repeat(self.gathered(self.Kc), g, 1), np.repeat(self.gathered(self.Vc), g, 1)
        Q = np64(self.Q)[:self.T]
        kw = dict(causal=self.causal, bias=None if self.bias is None else np64(self.bias), window=self.window)
        O, lse = oracle.fwd(q_off, kv_off, Q, K, V, **kw)
        A, _ = oracle.fwd(q_off, kv_off, Q, K, np.abs(V), **kw)
        return O, lse, A

    def run(self, jfa, cache=None, **kw):
        cache = cache or jfa.jfa_cache_create(self.Kc, self.Vc)
        O, lse = jfa.jfa_cache_fwd(cache, kw.pop("Q", self.Q), self.q_off, self.kv_lens, self.table, bias=self.bias,
                                   causal=self.causal, window=self.window,
                                   max_q_len=kw.pop("max_q_len", int(self.q.max()) if self.q.size else 0), **kw)
        torch.cuda.synchronize()
        status = jfa.jfa_cache_device_status(cache)
        assert status == jfa.JFA_OK, jfa.jfa_status_string(status)
        return O, lse

    def check(self, O, lse, ref=None, slack=SLACK):
        ro, rl, A = ref or self.reference()
        o, l = np64(O)[:self.T], np64(lse)[:self.T]
        tol = slack * A + 1e-30
        if self.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * A
        if O.dtype == torch.bfloat16:
            tol = tol + 2.0 ** -8 * np.abs(ro)
        over = np.abs(o - ro) - tol
        assert np.all(np.isfinite(o)), "non-finite output"
        assert over.max(initial=-1.0) <= 0.0, f"O off by {over.max()} more than the tolerance"
        fin = np.isfinite(rl)
        assert np.array_equal(fin, np.isfinite(l)) and np.all(l[~fin] == -np.inf)
        assert np.abs(l[fin] - rl[fin]).max(initial=0.0) <= LSE_TOL
