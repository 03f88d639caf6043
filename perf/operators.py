"""Measured cases of the paged-cache operators: appending new keys and values to a paged
cache with the position rotation applied on the way, and attention of ragged new tokens
over that cache.

`run` computes them in plain torch operations, or, with `own` set, by the framework's
calls on the same inputs.  A batch holds B sequences; sequence b has q_len[b] new tokens,
the last of its kv_len[b] positions.  Position p of sequence b lies in page
page_table[b, p // page], slot p % page, of caches [n_pages, page, Hkv, D].
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases

def listed():
    base = {"dtype": "bf16", "H": 32, "Hkv": 8, "D": 128, "page": 16, "prompts": 1.0, "lens": 1}
    append = dict(base, op="append", rot=128, kind="half")
    attend = dict(base, op="attend", causal=True, window=-1, bias=False)
    return [
        # one user's next token: the latency of a single small call
        dict(append, name="append_one_token", B=1, q_lo=1, q_hi=1, past_lo=1000, past_hi=1000),
        # a decode step of a full serving batch
        dict(append, name="append_decode_256", B=256, q_lo=1, q_hi=1, past_lo=100, past_hi=4000, page=32, lens=2),
        # prompts of very different lengths entering the cache together
        dict(append, name="append_prompts", B=24, q_lo=1, q_hi=2048, past_lo=0, past_hi=1500, lens=3),
        # fp32 reference serving, partial rotation of neighbouring pairs
        dict(append, name="append_f32_pairs", dtype="f32", B=7, H=8, Hkv=8, D=64, page=64, rot=32, kind="pairs",
             q_lo=100, q_hi=1300, past_lo=0, past_hi=77, lens=4),
        # one user's next token over a short history
        dict(attend, name="decode_one_user", B=1, q_lo=1, q_hi=1, past_lo=1000, past_hi=1000),
        # a decode step of a full batch, ragged histories
        dict(attend, name="decode_batch", B=64, q_lo=1, q_hi=1, past_lo=200, past_hi=16000, page=64, lens=5),
        # one very long history: the key axis has to be split
        dict(attend, name="decode_long", B=1, q_lo=1, q_hi=1, past_lo=131000, past_hi=131000, page=128),
        # ungrouped heads with the relative-position table: this framework's causal model, served
        dict(attend, name="decode_bias_heads8", B=200, H=8, Hkv=8, q_lo=1, q_hi=1, past_lo=31, past_hi=2047,
             page=32, bias=True, lens=6),
        # prompt chunks over long cached prefixes
        dict(attend, name="chunk_prefill", B=8, q_lo=700, q_hi=1024, past_lo=2000, past_hi=15000, page=64, lens=7),
        # a scheduler's mixed step: a few prompt chunks among single tokens, window and table
        dict(attend, name="mixed_window", B=48, H=8, Hkv=2, q_lo=200, q_hi=800, past_lo=0, past_hi=9000, page=16,
             prompts=0.2, window=2048, bias=True, lens=8),
        # query sets over cached user histories, not causal (1-64 rows, head_dim 64)
        dict(attend, name="cross_sets", B=256, H=8, Hkv=8, D=64, q_lo=1, q_hi=64, past_lo=100, past_hi=8000,
             page=128, causal=False, lens=9),
        # fp32 reference serving: chunks and single tokens together
        dict(attend, name="f32_mixed", dtype="f32", B=20, H=8, Hkv=4, D=64, q_lo=100, q_hi=700, past_lo=200,
             past_hi=6000, page=16, prompts=0.5, lens=10),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        c = {"op": rng.choice(["append", "attend", "attend"]), "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"])}
        c["D"] = rng.choice([64, 128] if c["dtype"] == "bf16" else [32, 64])
        c["Hkv"] = rng.choice([1, 2, 4, 8])
        c["H"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
        c["page"] = rng.choice([8, 16, 32, 64, 128, 256])
        c["prompts"] = rng.choice([0.0, 0.25, 1.0])
        c["B"] = _log(rng, 1, 256)
        c["q_lo"] = _log(rng, 1, 1024)
        c["q_hi"] = _log(rng, c["q_lo"], 2048)
        c["past_lo"] = _log(rng, 1, 16000) - 1
        c["past_hi"] = _log(rng, c["past_lo"] + 1, 131000) - 1
        c["lens"] = rng.randrange(1 << 30)
        if c["op"] == "append":
            c["rot"] = rng.choice([0, 16, c["D"] // 2, c["D"], c["D"]])
            c["kind"] = rng.choice(["half", "pairs"])
        else:
            c["causal"] = rng.random() < 0.8
            c["window"] = _log(rng, 1, 4096) if c["causal"] and rng.random() < 0.4 else -1
            c["bias"] = rng.random() < 0.4
        w, q, kv = work(c), *lengths(c)
        cells = c["B"] * c["H"] * int(q.max()) * int(kv.max())  # what the plain form holds of the scores
        rows = c["B"] * int(kv.max()) * c["Hkv"] * c["D"]
        if c["op"] == "append":
            if w["bytes"] < 6e8 and int(kv.sum()) * c["Hkv"] * c["D"] < 5e8:
                return c
        elif w["flops"] < (8e11 if c["dtype"] == "bf16" else 2e10) and w["bytes"] < 6e8 and cells < 3e9 and rows < 4e9:
            return c


def lengths(c):
    """(q_len, kv_len) of the case: prompts of q_lo..q_hi tokens, the other sequences one
    token, after past_lo..past_hi tokens spread over their logarithm."""
    rs = np.random.RandomState(c["lens"] % (1 << 32))
    B = c["B"]
    q = rs.randint(c["q_lo"], c["q_hi"] + 1, B)
    q = np.where(rs.random_sample(B) < c["prompts"], q, 1)
    past = np.exp(rs.uniform(math.log(c["past_lo"] + 1), math.log(c["past_hi"] + 1.0001), B)).astype(np.int64) - 1
    return q.astype(np.int64), q + np.clip(past, c["past_lo"], c["past_hi"])


def _pairs(c):
    """Allowed (query, key) pairs of each sequence and the keys that any of its rows may see."""
    q, kv = lengths(c)
    if not c["causal"]:
        return q * kv, kv
    i = np.arange(int(q.max()))[None, :]
    last = kv[:, None] - q[:, None] + i                    # the last key of each row
    first = np.maximum(last - c["window"], 0) if c["window"] >= 0 else np.zeros_like(last)
    n = np.where(i < q[:, None], last - first + 1, 0).sum(1)
    return n, kv - first[:, 0]


def work(c):
    q, kv = lengths(c)
    T, es = int(q.sum()), 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        moved = (4 * c["Hkv"] + (2 * c["H"] if c["rot"] else 0)) * c["D"] * es
        return {"bytes": T * (moved + 4 * c["rot"]), "flops": 3 * T * (c["H"] + c["Hkv"]) * c["rot"]}
    pairs, keys = _pairs(c)
    moved = int(keys.sum()) * 2 * c["Hkv"] * c["D"] * es + T * c["H"] * (2 * c["D"] * es + 4)
    return {"bytes": moved, "flops": 4 * c["D"] * c["H"] * int(pairs.sum())}


# ------------------------------------------------------------------------------ inputs

def prepare(c, seed):
    """The batch on the GPU: pages dealt out in random order, slots that no position uses
    undefined (NaN: a fresh page holds anything)."""
    dev, dt = torch.device("cuda"), TYPES[c["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    q, kv = lengths(c)
    B, T, page, Hkv, D = c["B"], int(q.sum()), c["page"], c["Hkv"], c["D"]
    need = -(-kv // page)
    n_pages, width = int(need.sum()) + 3, int(need.max())
    order = torch.randperm(n_pages, generator=g, device=dev).int()
    first = torch.from_numpy(np.cumsum(need) - need).to(dev)
    col = torch.arange(width, device=dev)
    used = col[None, :] < torch.from_numpy(need).to(dev)[:, None]
    table = torch.where(used, order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).int().contiguous()
    kv_len = torch.from_numpy(kv).to(dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    s = {"c": c, "table": table, "kv_len": kv_len.int(), "q_max": int(q.max()), "kv_max": int(kv.max()),
         "q_off": torch.from_numpy(np.concatenate([[0], np.cumsum(q)])).to(dev).int(),
         "Q": normal(T, c["H"], D), "kc": normal(n_pages, page, Hkv, D), "vc": normal(n_pages, page, Hkv, D)}
    if c["op"] == "append":
        s["K"], s["V"] = normal(T, Hkv, D), normal(T, Hkv, D)
        s["Q_out"] = torch.empty_like(s["Q"])
        s["rot"] = None
        if c["rot"]:
            half = c["rot"] // 2
            f = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
            a = torch.arange(s["kv_max"], device=dev, dtype=torch.float64)[:, None] * f
            s["rot"] = torch.cat([a.cos(), a.sin()], 1).float()
    else:
        slot = col[:, None] * page + torch.arange(page, device=dev)  # [width, page] positions
        spare = torch.ones(n_pages, page, dtype=torch.bool, device=dev)
        spare[table[used].long()] = (slot[None] >= kv_len[:, None, None])[used]
        s["kc"][spare], s["vc"][spare] = float("nan"), float("nan")
        s["bias"] = torch.randn(c["H"], 32, generator=g, device=dev) * 0.1 if c["bias"] else None
        s["O"] = torch.empty_like(s["Q"])
        s["lse"] = torch.empty(T, c["H"], device=dev)
    if own:
        from jagged_sequence_attention_gb300 import jfa
        s["jfa"] = jfa
        s["cache"] = jfa.jfa_cache_create(s["kc"], s["vc"])
        if c["op"] == "attend":
            s["workspace"] = jfa.jfa_cache_workspace(s["cache"], c["H"])
    return s


# ------------------------------------------------------------------------------ the operators

def run(s):
    if s["c"]["op"] == "append":
        return append(s)
    return attend(s)


def append(s):
    c = s["c"]
    if own:
        rotates = s["rot"] is not None
        s["jfa"].jfa_cache_append(s["cache"], s["K"], s["V"], s["q_off"], s["kv_len"], s["table"],
                                  Q=s["Q"] if rotates else None, Q_out=s["Q_out"] if rotates else None,
                                  rot=s["rot"], rot_kind=c["kind"])
        return {"k": s["kc"], "v": s["vc"], "q": s["Q_out"] if rotates else s["Q"]}
    q_off = s["q_off"].long()
    t = torch.arange(s["K"].shape[0], device=q_off.device)
    b = torch.searchsorted(q_off, t, right=True) - 1
    pos = s["kv_len"].long()[b] - q_off[b + 1] + t
    page, slot = s["table"].long()[b, pos // c["page"]], pos % c["page"]
    s["kc"][page, slot] = rotated(s["K"], s["rot"], pos, c["kind"])
    s["vc"][page, slot] = s["V"]
    return {"k": s["kc"], "v": s["vc"], "q": rotated(s["Q"], s["rot"], pos, c["kind"])}


def rotated(x, table, pos, kind):
    if table is None:
        return x
    R = table.shape[1]
    cos, sin = table[pos][:, None, :].chunk(2, -1)
    y = x.float()
    if kind == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, y[..., R:]], -1).to(x.dtype)


def attend(s):
    c = s["c"]
    if own:
        window = c["window"] if c["window"] >= 0 else None
        O, lse = s["jfa"].jfa_cache_fwd(s["cache"], s["Q"], s["q_off"], s["kv_len"], s["table"], bias=s["bias"],
                                        causal=c["causal"], window=window, max_q_len=s["q_max"], O=s["O"],
                                        lse=s["lse"], workspace=s["workspace"])
        return {"o": O, "lse": lse}
    B, H, Hkv, D, n, L = c["B"], c["H"], c["Hkv"], c["D"], s["q_max"], s["kv_max"]
    g, dev = H // Hkv, s["Q"].device
    q_off, kv_len = s["q_off"].long(), s["kv_len"].long()
    q_len = q_off[1:] - q_off[:-1]
    i, j = torch.arange(n, device=dev), torch.arange(L, device=dev)
    # padded copies: keys and values through the page table, queries by their offsets
    inside = (j < kv_len[:, None])[:, :, None, None]
    pages = s["table"].long().clamp(min=0)
    k = s["kc"][pages].reshape(B, -1, Hkv, D)[:, :L].float().masked_fill_(~inside, 0.0).permute(0, 2, 3, 1)
    v = s["vc"][pages].reshape(B, -1, Hkv, D)[:, :L].float().masked_fill_(~inside, 0.0).permute(0, 2, 1, 3)
    row = (q_off[:-1, None] + i).clamp(max=max(s["Q"].shape[0] - 1, 0))
    q = s["Q"][row].float().reshape(B, n, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * n, D)
    x = torch.matmul(q * (1.0 / math.sqrt(D)), k).reshape(B, Hkv, g, n, L)
    far = (i[None, :] + (kv_len - q_len)[:, None])[:, :, None] - j  # i' - j, [B, n, L]
    if s["bias"] is not None:
        r = far.abs() + 1  # bucket: floor(log2 r^2), at most 31, counted in whole numbers
        bucket = torch.bucketize(r * r, 2 ** torch.arange(1, 32, device=dev), right=True)
        x += s["bias"].reshape(Hkv, g, 32)[:, :, bucket].permute(2, 0, 1, 3, 4)
    out = ~inside[:, None, :, 0, 0]
    if c["causal"]:
        out = out | (far < 0)
        if c["window"] >= 0:
            out = out | (far > c["window"])
    x.masked_fill_(out[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(B, Hkv, g * n, L), v).reshape(B, Hkv, g, n, D) / total
    o = torch.where(total > 0, o, 0.0)
    lse = (m + total.log())[..., 0]
    there = (i < q_len[:, None]).reshape(-1)
    O = o.permute(0, 3, 1, 2, 4).reshape(B * n, H, D)[there].to(s["Q"].dtype)
    return {"o": O, "lse": lse.permute(0, 3, 1, 2).reshape(B * n, H)[there]}


# ------------------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    """The outputs from the definitions, sequence by sequence, in 64 bits."""
    s = prepare(c, seed)
    q, kv = lengths(c)
    if c["op"] == "append":
        k, v, Q = s["kc"].double(), s["vc"].double(), s["Q"].double()
        row = 0
        for b in range(c["B"]):
            n = int(q[b])
            p = torch.arange(int(kv[b]) - n, int(kv[b]), device=Q.device)
            page, slot = s["table"][b].long()[p // c["page"]], p % c["page"]
            k[page, slot] = _turn(s["K"][row:row + n].double(), s["rot"], p, c["kind"])
            v[page, slot] = s["V"][row:row + n].double()
            Q[row:row + n] = _turn(Q[row:row + n], s["rot"], p, c["kind"])
            row += n
        return {"k": k, "v": v, "q": Q}
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    g, row = H // Hkv, 0
    O = torch.zeros(s["Q"].shape, dtype=torch.float64, device=s["Q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=s["Q"].device)
    for b in range(c["B"]):
        n, L = int(q[b]), int(kv[b])
        pages = s["table"][b, :-(-L // c["page"])].long()
        k = s["kc"][pages].reshape(-1, Hkv, D)[:L].double()
        v = s["vc"][pages].reshape(-1, Hkv, D)[:L].double()
        Q = s["Q"][row:row + n].double()
        at = torch.arange(n, device=k.device)[:, None] + (L - n)
        key = torch.arange(L, device=k.device)[None, :]
        hidden = (key > at) if c["causal"] else torch.zeros(n, L, dtype=torch.bool, device=k.device)
        if c["window"] >= 0:
            hidden |= key < at - c["window"]
        if s["bias"] is not None:
            d = (at - key).abs().double() + 1
            bucket = torch.floor(2 * torch.log2(d) + 1e-12).clamp(max=31).long()
        for h in range(H):
            x = Q[:, h] @ k[:, h // g].T / math.sqrt(D)
            if s["bias"] is not None:
                x = x + s["bias"][h].double()[bucket]
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1)
            O[row:row + n, h] = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None]) @ v[:, h // g]
            lse[row:row + n, h] = z
        row += n
    return {"o": O, "lse": lse}


def _turn(x, table, pos, kind):
    """x times e^{i angle}, with the rotated elements read as complex numbers."""
    if table is None:
        return x
    half = table.shape[1] // 2
    w = torch.complex(*table.double()[pos].split(half, 1))[:, None, :]
    y = x.clone()
    re, im = (slice(0, half), slice(half, 2 * half)) if kind == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * w
    y[..., re], y[..., im] = z.real, z.imag
    return y
