"""Measured cases of the operators that make a paged cache's histories cheaper to read: the
cache held in 4 bits (appending to it, reading it back, attention over it), and attention
over the blocks that a cheap score selects for each query (the blocks' bounds, the
selection, the attention).

`run` computes them in plain torch operations, or, with `own` set, by the framework's
calls on the same inputs.  A batch holds B sequences; sequence b has q_len[b] new tokens,
the last of its kv_len[b] positions.  Position p of sequence b lies in page
page_table[b, p // page], slot p % page.  A 16-bit cache is bf16 [n_pages, page, Hkv, D].  A
4-bit cache holds e2m1 codes [n_pages, page, Hkv, D / 2] (head-major), element 2i in the low half of byte
i, and an e4m3 scale for each 16 elements [n_pages, Hkv, page, D / 16]; a value is
factor * scale * code, with one factor for all keys and one for all values.
"""
import math

import numpy as np
import torch

own = False

BF, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ cases

def listed():
    base = {"bits": 4, "factor": 1.0, "H": 32, "Hkv": 8, "D": 128, "page": 16, "prompts": 1.0, "lens": 1}
    append = dict(base, op="append", rot=128, kind="half")
    attend = dict(base, op="attend", causal=True, window=-1, bias=False)
    select = dict(base, op="select", bits=16, first=1, last=1)
    blocks = dict(base, op="blocks", bits=16, bias=False)
    return [
        # a decode step of a full serving batch enters the 4-bit cache
        dict(append, name="append4_step", B=256, q_lo=1, q_hi=1, past_lo=100, past_hi=4000, page=32, lens=2),
        # prompts of very different lengths entering it together
        dict(append, name="append4_prompts", B=24, q_lo=1, q_hi=2048, past_lo=0, past_hi=1500, lens=3),
        # one user's next token over a short history
        dict(attend, name="attend4_one_user", B=1, q_lo=1, q_hi=1, past_lo=1000, past_hi=1000),
        # a decode step of a full batch, ragged histories
        dict(attend, name="attend4_batch", B=64, q_lo=1, q_hi=1, past_lo=200, past_hi=16000, page=64, lens=5),
        # one very long history, what 4 bits are for
        dict(attend, name="attend4_long", B=1, q_lo=1, q_hi=1, past_lo=131000, past_hi=131000, page=128),
        # prompt chunks over long cached prefixes
        dict(attend, name="attend4_chunks", B=8, q_lo=700, q_hi=1024, past_lo=2000, past_hi=15000, page=64, lens=7),
        # one very long history: 128 of its 8188 blocks
        dict(select, name="select_long", B=1, q_lo=1, q_hi=1, past_lo=131000, past_hi=131000, n=128),
        # a decode step of a full batch of 4-bit histories, a few recent blocks always kept
        dict(select, name="select_batch", bits=4, B=64, q_lo=1, q_hi=1, past_lo=200, past_hi=16000, page=32, n=64,
             last=4, lens=5),
        # prompt chunks: every token selects for itself
        dict(select, name="select_chunks", B=4, q_lo=100, q_hi=500, past_lo=5000, past_hi=20000, page=64, n=32, lens=9),
        # the attention after select_long
        dict(blocks, name="blocks_long", B=1, q_lo=1, q_hi=1, past_lo=131000, past_hi=131000, n=128),
        # the attention after select_batch
        dict(blocks, name="blocks_batch4", bits=4, B=64, q_lo=1, q_hi=1, past_lo=200, past_hi=16000, page=32, n=64,
             lens=5),
        # drafts of a few tokens, every token over blocks of its own, ungrouped heads and the
        # relative-position table
        dict(blocks, name="blocks_drafts", B=32, H=8, Hkv=8, D=64, q_lo=1, q_hi=8, past_lo=500, past_hi=8000, page=64,
             n=16, bias=True, lens=10),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "select", "blocks"])
        c = {"op": op, "bits": 4 if op in ("append", "attend") else rng.choice([4, 16])}
        c["factor"] = rng.choice([1.0, 1.0, 0.25, 0.3125])
        c["D"] = rng.choice([64, 128, 128])
        c["Hkv"] = rng.choice([1, 2, 4, 8])
        c["H"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
        c["page"] = rng.choice([16, 32, 64, 128, 256] + ([8, 8] if c["bits"] == 4 and op in ("append", "attend") else []))
        c["prompts"] = rng.choice([0.0, 0.25, 1.0])
        c["B"] = _log(rng, 1, 256)
        c["q_lo"] = _log(rng, 1, 1024 if op in ("append", "attend") else 64)
        c["q_hi"] = _log(rng, c["q_lo"], 2048 if op in ("append", "attend") else 500)
        c["past_lo"] = _log(rng, 1, 16000) - 1
        c["past_hi"] = _log(rng, c["past_lo"] + 1, 131000) - 1
        c["lens"] = rng.randrange(1 << 30)
        if op == "append":
            c["rot"] = rng.choice([0, 16, c["D"] // 2, c["D"], c["D"]])
            c["kind"] = rng.choice(["half", "pairs"])
        elif op == "attend":
            c["causal"] = rng.random() < 0.8
            c["window"] = _log(rng, 1, 4096) if c["causal"] and rng.random() < 0.4 else -1
            c["bias"] = rng.random() < 0.4
        elif op == "select":
            c["n"] = _log(rng, 2, 256)
            c["first"] = rng.choice([0, 1])
            c["last"] = rng.randint(1, min(8, c["n"] - c["first"]))
        else:
            c["n"] = _log(rng, 1, 256)
            c["bias"] = rng.random() < 0.4
        w, q, kv = work(c), *lengths(c)
        B, T, L = c["B"], int(q.sum()), int(kv.max())
        rows = int(kv.sum()) * c["Hkv"] * c["D"]
        if op == "append":
            fits = w["bytes"] < 7e8 and rows < 5e8
        elif op == "attend":
            cells = B * c["H"] * int(q.max()) * L  # what the plain form holds of the scores
            fits = w["flops"] < 8e11 and w["bytes"] < 6e8 and cells < 3e9 and B * L * c["Hkv"] * c["D"] < 1.5e9
        elif op == "select":
            nb = -(-L // c["page"])
            fits = (rows < 7e8 and B * nb * c["Hkv"] * c["D"] < 5e7 and T * c["page"] * c["Hkv"] * c["D"] < 2e9
                    and B * int(q.max()) * c["Hkv"] * nb < 1e8 and T * c["Hkv"] < 2e4 and w["flops"] < 6e9)
        else:
            fits = rows < 7e8 and T * c["n"] * c["page"] * c["Hkv"] * c["D"] < 3e8
        if fits:
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


def _positions(c):
    """The position of every new token, and its sequence."""
    q, kv = lengths(c)
    b = np.repeat(np.arange(c["B"]), q)
    return np.arange(int(q.sum())) - np.repeat(np.cumsum(q) - q, q) + (kv - q)[b], b


def work(c):
    q, kv = lengths(c)
    T, H, Hkv, D, page = int(q.sum()), c["H"], c["Hkv"], c["D"], c["page"]
    row = D * 9 // 16 if c["bits"] == 4 else 2 * D          # bytes of one position of one head
    if c["op"] == "append":
        # bf16 rows in, 4-bit rows out and in again, bf16 rows out; rotated queries
        moved = 2 * Hkv * (2 * D + 2 * row + 2 * D) + (4 * H * D if c["rot"] else 0)
        return {"bytes": T * (moved + 4 * c["rot"]), "flops": T * (3 * (H + Hkv) * c["rot"] + 6 * Hkv * D)}
    if c["op"] == "attend":
        pairs, keys = _pairs(c)
        moved = int(keys.sum()) * 2 * Hkv * row + T * H * (2 * D * 2 + 4)
        return {"bytes": moved, "flops": 4 * D * H * int(pairs.sum())}
    pos, b = _positions(c)
    if c["op"] == "select":
        touched = int((kv - (kv - q) // page * page).sum())  # positions of the pages that get new tokens
        pages = int((-(-kv // page) - (kv - q) // page).sum())
        moved = Hkv * (touched * row + pages * 4 * D + int((-(-kv // page)).sum()) * 4 * D) + T * (2 * H * D + 4 * Hkv * c["n"])
        return {"bytes": moved, "flops": 4 * D * Hkv * int((pos // page + 1).sum())}
    own_block = pos // page
    listed_blocks = np.minimum(own_block + 1, c["n"])
    keys = listed_blocks * page - (page - 1 - pos % page)   # positions that a token's list lets it see
    once = np.minimum(np.bincount(b, listed_blocks * page, c["B"]), kv)
    moved = int(once.sum()) * 2 * Hkv * row + T * (H * (4 * D + 4) + 4 * Hkv * c["n"])
    return {"bytes": moved, "flops": 4 * D * H * int(keys.sum())}


# ------------------------------------------------------------------------------ inputs

def prepare(c, seed):
    """The batch on the GPU: pages dealt out in random order, slots that no position uses
    undefined (NaN: a fresh page holds anything)."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    q, kv = lengths(c)
    T, page, H, Hkv, D = int(q.sum()), c["page"], c["H"], c["Hkv"], c["D"]
    need = -(-kv // page)
    n_pages, width = int(need.sum()) + 3, int(need.max())
    order = torch.randperm(n_pages, generator=g, device=dev).int()
    first = torch.from_numpy(np.cumsum(need) - need).to(dev)
    col = torch.arange(width, device=dev)
    used = col[None, :] < torch.from_numpy(need).to(dev)[:, None]
    table = torch.where(used, order[(first[:, None] + col).clamp(max=n_pages - 1)], -1).int().contiguous()
    kv_len = torch.from_numpy(kv).to(dev)
    slot = col[:, None] * page + torch.arange(page, device=dev)  # [width, page] positions
    spare = torch.ones(n_pages, page, dtype=torch.bool, device=dev)
    spare[table[used].long()] = (slot[None] >= kv_len[:, None, None])[used]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=BF)

    s = {"c": c, "table": table, "kv_len": kv_len.int(), "q_max": int(q.max()), "kv_max": int(kv.max()), "T": T,
         "q_off": torch.from_numpy(np.concatenate([[0], np.cumsum(q)])).to(dev).int(), "Q": normal(T, H, D)}
    for name in ("k", "v") if c["op"] != "select" else ("k",):
        x = normal(n_pages, page, Hkv, D)
        if c["bits"] == 4:
            codes = torch.empty(n_pages, Hkv, page, D // 2, dtype=torch.uint8, device=dev).transpose(1, 2)
            scales = torch.empty(n_pages, Hkv, page, D // 16, dtype=E4M3, device=dev)
            for i in range(0, n_pages, 4096):  # (a long history in parts: less memory)
                codes[i:i + 4096], part = quantised(x[i:i + 4096].float(), c["factor"])
                scales[i:i + 4096] = part.transpose(1, 2)
            scales.view(torch.uint8).transpose(1, 2)[spare] = 0x7F
            s[name + "c"], s[name + "s"] = codes, scales
        else:
            x[spare] = float("nan")
            s[name + "c"] = x
    if c["op"] == "select" and c["bits"] == 4:  # (values are not read)
        s["vc"], s["vs"] = s["kc"], s["ks"]
    elif c["op"] == "select":
        s["vc"] = s["kc"]
    if c["op"] == "append":
        s["K"], s["V"] = normal(T, Hkv, D), normal(T, Hkv, D)
        s["Q_out"] = torch.empty_like(s["Q"])
        s["K_out"], s["V_out"] = torch.empty_like(s["K"]), torch.empty_like(s["V"])
        s["rot"] = None
        if c["rot"]:
            half = c["rot"] // 2
            f = 10000.0 ** (-torch.arange(half, device=dev, dtype=F64) / half)
            a = torch.arange(s["kv_max"], device=dev, dtype=F64)[:, None] * f
            s["rot"] = torch.cat([a.cos(), a.sin()], 1).float()
    if c["op"] in ("attend", "blocks"):
        s["bias"] = torch.randn(H, 32, generator=g, device=dev) * 0.1 if c["bias"] else None
        s["O"] = torch.empty_like(s["Q"])
        s["lse"] = torch.empty(T, H, device=dev)
    if c["op"] == "select":
        # the bounds as earlier steps left them: undefined for the pages that get new tokens
        s["bounds"] = normal(n_pages, Hkv, 2, D)
        old = torch.from_numpy((kv - q) // page).to(dev)
        page_of = table[(col[None, :] < old[:, None]) & used].long()
        for i in range(0, page_of.numel(), 4096):
            at = page_of[i:i + 4096]
            x = keys_of(s, at)
            s["bounds"][at] = torch.stack([x.amin(1), x.amax(1)], 2).to(BF)
        s["chosen"] = torch.empty(T, Hkv, c["n"], dtype=torch.int32, device=dev)
    if c["op"] == "blocks":
        # the first and the own block of every token, and a random choice between, ascending
        pos, b = _positions(c)
        own_block = torch.from_numpy(pos // page).to(dev)[:, None, None]
        nb, n = width, c["n"]
        x = torch.rand(T, Hkv, nb, generator=g, device=dev)
        k = torch.arange(nb, device=dev)
        x = torch.where(k == own_block, 3.0, torch.where(k == 0, 2.0, torch.where(k < own_block, x, -1.0)))
        best, at = x.topk(min(n, nb), -1)
        at = torch.where(best >= 0, at, nb).sort(-1)[0]
        at = torch.where(at < nb, at, -1)
        s["lists"] = torch.nn.functional.pad(at, (0, n - at.shape[-1]), value=-1).int().contiguous()
    if own:
        from jagged_sequence_attention_gb300 import jfa
        s["jfa"] = jfa
        if c["bits"] == 4:
            s["cache"] = jfa.jfa_cache_create_quantized(s["kc"], s["vc"], s["ks"], s["vs"], c["factor"], c["factor"])
        else:
            s["cache"] = jfa.jfa_cache_create(s["kc"], s["vc"])
        if c["op"] in ("attend", "blocks"):
            s["workspace"] = jfa.jfa_cache_workspace(s["cache"], H)
        if c["op"] == "select":
            s["workspace"] = jfa.jfa_cache_select_workspace(s["cache"], T, table.shape[1])
    return s


def quantised(x, factor):
    """Codes [.., D / 2] and scales [.., D / 16] of rows x [.., D], in x's precision."""
    y = (x / factor).unflatten(-1, (-1, 16))
    a = (y.abs().amax(-1) / 6).clamp(max=448)
    # rounded to e4m3's four bits here: by way of fp32 it would be rounded twice
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6)) + 1e-6) - 3)
    scale = (torch.round(a / step) * step).float().to(E4M3)
    s = scale.to(x.dtype)[..., None]
    t = torch.where(s > 0, y / torch.where(s > 0, s, 1.0), 0.0)
    a = t.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    # the middles between neighbours; a tie goes to the even code
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a > mid) if i % 2 == 0 else (a >= mid)
    code += 8 * (t < 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def values(codes, scales, factor, dtype=F32):
    """Rows [.., D] that codes [.., D / 2] and scales [.., D / 16] stand for."""
    table = torch.tensor([*CODES, *(-x for x in CODES)], dtype=dtype, device=codes.device)
    x = table[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, 16)) * scales.to(dtype)[..., None]).flatten(-2) * factor


def keys_of(s, pages, dtype=F32):
    """Keys [n, page, Hkv, D] of n pages (of a 4-bit cache without the factor)."""
    if s["c"]["bits"] == 4:
        return values(s["kc"][pages], s["ks"].view(torch.uint8)[pages].view(E4M3).transpose(1, 2), 1.0, dtype)
    return s["kc"][pages].to(dtype)


def gathered(s, name, pages, dtype=F32):
    """Keys or values [.., page, Hkv, D] of pages [..]."""
    c = s["c"]
    if c["bits"] == 4:
        scales = s[name + "s"].view(torch.uint8)[pages].view(E4M3).transpose(-2, -3)
        return values(s[name + "c"][pages], scales, c["factor"], dtype)
    return s[name + "c"][pages].to(dtype)


# ------------------------------------------------------------------------------ the operators

def run(s):
    return {"append": append, "attend": attend, "select": select, "blocks": blocks}[s["c"]["op"]](s)


def where(s):
    """Of every new token: its sequence, position, and the page and slot it lies in."""
    q_off = s["q_off"].long()
    t = torch.arange(s["T"], device=q_off.device)
    b = torch.searchsorted(q_off, t, right=True) - 1
    pos = s["kv_len"].long()[b] - q_off[b + 1] + t
    return b, pos, s["table"].long()[b, pos // s["c"]["page"]], pos % s["c"]["page"]


def append(s):
    """The new tokens into the cache, and their rows as the cache then holds them."""
    c = s["c"]
    if own:
        rotates = s["rot"] is not None
        s["jfa"].jfa_cache_append(s["cache"], s["K"], s["V"], s["q_off"], s["kv_len"], s["table"],
                                  Q=s["Q"] if rotates else None, Q_out=s["Q_out"] if rotates else None,
                                  rot=s["rot"], rot_kind=c["kind"])
        K, V = s["jfa"].jfa_cache_read(s["cache"], s["T"], s["q_off"], s["kv_len"], s["table"], K=s["K_out"], V=s["V_out"])
        return {"k": K, "v": V, "q": s["Q_out"] if rotates else s["Q"]}
    _, pos, page, slot = where(s)
    # (quantised in 64 bits: a value next to the middle of two codes)
    for name, x in (("k", rotated(s["K"], s["rot"], pos, c["kind"])), ("v", s["V"].double())):
        codes, scales = quantised(x, c["factor"])
        s[name + "c"][page, slot] = codes
        s[name + "s"].view(torch.uint8)[page, :, slot] = scales.view(torch.uint8)
    out = {"q": rotated(s["Q"], s["rot"], pos, c["kind"]).to(BF)}
    for name in ("k", "v"):
        scales = s[name + "s"].view(torch.uint8)[page, :, slot].view(E4M3)
        out[name] = values(s[name + "c"][page, slot], scales, c["factor"]).to(BF)
    return out


def rotated(x, table, pos, kind):
    """x rotated by its position, in 64 bits."""
    if table is None:
        return x.double()
    R = table.shape[1]
    cos, sin = table.double()[pos][:, None, :].chunk(2, -1)
    y = x.double()
    if kind == "half":
        a, b = y[..., :R // 2], y[..., R // 2:R]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:R:2], y[..., 1:R:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, y[..., R:]], -1)


def bucket_of(r):
    """floor(log2 (1 + |r|)^2), at most 31, counted in whole numbers."""
    r = r.abs() + 1
    return torch.bucketize(r * r, 2 ** torch.arange(1, 32, device=r.device), right=True)


def softmax_of(x, v):
    """Softmax of x [.., L] (-inf: not allowed) times v [.., L, D], and its log-sum."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / total
    return torch.where(total > 0, o, 0.0), (m + total.log())[..., 0]


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
    k = gathered(s, "k", pages).reshape(B, -1, Hkv, D)[:, :L].masked_fill(~inside, 0.0).permute(0, 2, 3, 1)
    v = gathered(s, "v", pages).reshape(B, -1, Hkv, D)[:, :L].masked_fill(~inside, 0.0).permute(0, 2, 1, 3)
    row = (q_off[:-1, None] + i).clamp(max=max(s["T"] - 1, 0))
    q = s["Q"][row].float().reshape(B, n, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * n, D)
    x = torch.matmul(q * (1.0 / math.sqrt(D)), k).reshape(B, Hkv, g, n, L)
    far = (i[None, :] + (kv_len - q_len)[:, None])[:, :, None] - j  # i' - j, [B, n, L]
    if s["bias"] is not None:
        x += s["bias"].reshape(Hkv, g, 32)[:, :, bucket_of(far)].permute(2, 0, 1, 3, 4)
    out = ~inside[:, None, :, 0, 0]
    if c["causal"]:
        out = out | (far < 0)
        if c["window"] >= 0:
            out = out | (far > c["window"])
    x.masked_fill_(out[:, None, None], -math.inf)
    o, lse = softmax_of(x.reshape(B, Hkv, g * n, L), v)
    there = (i < q_len[:, None]).reshape(-1)
    O = o.reshape(B, Hkv, g, n, D).permute(0, 3, 1, 2, 4).reshape(B * n, H, D)[there].to(BF)
    return {"o": O, "lse": lse.reshape(B, Hkv, g, n).permute(0, 3, 1, 2).reshape(B * n, H)[there]}


def select(s):
    """The bounds of the pages that got new tokens, and the blocks of every token."""
    c = s["c"]
    if own:
        s["jfa"].jfa_cache_summarize(s["cache"], s["bounds"], s["T"], s["q_off"], s["kv_len"], s["table"])
        chosen = s["jfa"].jfa_cache_select(s["cache"], s["bounds"], s["Q"], s["q_off"], s["kv_len"], s["table"], c["n"],
                                           n_first=c["first"], n_last=c["last"], max_q_len=s["q_max"],
                                           blocks=s["chosen"], workspace=s["workspace"])
        return {"bounds": s["bounds"], "blocks": chosen}
    b, pos, page, _ = where(s)
    P, Hkv, D, n, T, dev = c["page"], c["Hkv"], c["D"], s["q_max"], s["T"], s["Q"].device
    x = keys_of(s, page)
    filled = (pos // P * P)[:, None] + torch.arange(P, device=dev) < s["kv_len"].long()[b][:, None]
    filled = filled[:, :, None, None]
    s["bounds"][page] = torch.stack([x.masked_fill(~filled, math.inf).amin(1), x.masked_fill(~filled, -math.inf).amax(1)], 2).to(BF)
    # scores in 64 bits: two blocks may be next to each other, and their order is the answer
    q = s["Q"].double().reshape(T, Hkv, -1, D)
    both = torch.stack([q.clamp(max=0).sum(2), q.clamp(min=0).sum(2)], 2).flatten(2)  # [T, Hkv, 2 D]
    q_off = s["q_off"].long()
    row = (q_off[:-1, None] + torch.arange(n, device=dev)).clamp(max=T - 1)
    bound = s["bounds"][s["table"].long().clamp(min=0)].double().flatten(3)           # [B, nb, Hkv, 2 D]
    score = torch.matmul(both[row].transpose(1, 2), bound.permute(0, 2, 3, 1))        # [B, Hkv, n, nb]
    nb = score.shape[-1]
    score = score.transpose(1, 2).flatten(0, 1)[(torch.arange(n, device=dev) < (q_off[1:] - q_off[:-1])[:, None]).flatten()]
    k, own_block = torch.arange(nb, device=dev), (pos // P)[:, None, None]
    score = torch.where((k < c["first"]) | (k > own_block - c["last"]), math.inf, score)
    score = torch.where(k <= own_block, score, -math.inf)
    top = score.sort(stable=True, dim=-1, descending=True)[1][..., :c["n"]]
    top = torch.where(top <= own_block, top, nb).sort(-1)[0]
    top = torch.where(top < nb, top, -1).int()
    return {"bounds": s["bounds"], "blocks": torch.nn.functional.pad(top, (0, c["n"] - top.shape[-1]), value=-1)}


def blocks(s):
    c = s["c"]
    if own:
        O, lse = s["jfa"].jfa_cache_fwd_blocks(s["cache"], s["Q"], s["q_off"], s["kv_len"], s["table"], s["lists"],
                                               bias=s["bias"], O=s["O"], lse=s["lse"], workspace=s["workspace"])
        return {"o": O, "lse": lse}
    b, pos, _, _ = where(s)
    T, H, Hkv, D, P, dev = s["T"], c["H"], c["Hkv"], c["D"], c["page"], s["Q"].device
    lists = s["lists"].long()                                                          # [T, Hkv, n]
    pages = s["table"].long()[b[:, None, None], lists.clamp(min=0)].clamp(min=0)
    j = lists[..., None] * P + torch.arange(P, device=dev)                             # [T, Hkv, n, P]
    seen = ((lists[..., None] >= 0) & (j <= pos[:, None, None, None])).flatten(2)
    j, head = j.flatten(2), torch.arange(Hkv, device=dev)[:, None]
    kv = []
    for name in ("k", "v"):
        if c["bits"] == 4:
            scales = s[name + "s"].view(torch.uint8)[pages, head].view(E4M3)
            x = values(s[name + "c"][pages, :, head], scales, c["factor"])
        else:
            x = s[name + "c"][pages, :, head].float()
        kv.append(x.flatten(2, 3).masked_fill(~seen[..., None], 0.0))                  # [T, Hkv, n P, D]
    q = s["Q"].float().reshape(T, Hkv, -1, D)
    x = torch.matmul(q * (1.0 / math.sqrt(D)), kv[0].transpose(2, 3))
    if s["bias"] is not None:
        bucket = bucket_of(pos[:, None, None] - j)
        x += s["bias"].reshape(Hkv, -1, 32)[head[..., None], torch.arange(H // Hkv, device=dev)[:, None], bucket[:, :, None]]
    x.masked_fill_(~seen[:, :, None], -math.inf)
    o, lse = softmax_of(x, kv[1])
    return {"o": o.reshape(T, H, D).to(BF), "lse": lse.reshape(T, H)}


# ------------------------------------------------------------------------------ in 64 bits

def exact(c, seed):
    """The outputs from the definitions, in 64 bits, sequence by sequence (or token by token)."""
    s = prepare(c, seed)
    return {"append": _append, "attend": _attend, "select": _select, "blocks": _blocks}[c["op"]](c, s)


def _rows(c):
    """(sequence, its first row, its new tokens, its positions) of every sequence."""
    q, kv = lengths(c)
    row = 0
    for b in range(c["B"]):
        yield b, row, int(q[b]), int(kv[b])
        row += int(q[b])


def _turn(x, table, p, kind):
    """x times e^{i angle}, with the rotated elements read as complex numbers."""
    if table is None:
        return x
    half = table.shape[1] // 2
    w = torch.complex(*table.double()[p].split(half, 1))[:, None, :]
    y = x.clone()
    re, im = (slice(0, half), slice(half, 2 * half)) if kind == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(x[..., re].contiguous(), x[..., im].contiguous()) * w
    y[..., re], y[..., im] = z.real, z.imag
    return y


def _nearest(x, grid):
    """The index of the entry of an ascending grid nearest to x >= 0; of two equally near
    ones the even index."""
    at = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    low, high = x - grid[at - 1], grid[at] - x
    return torch.where((low < high) | ((low == high) & (at % 2 == 1)), at - 1, at)


def _held(x, factor):
    """What a 4-bit cache holds of rows x."""
    e4m3 = torch.arange(127, dtype=torch.uint8, device=x.device).view(E4M3).double()  # 0 .. 448
    e2m1 = torch.tensor(CODES, dtype=F64, device=x.device)
    y = x.unflatten(-1, (-1, 16))
    scale = factor * e4m3[_nearest(y.abs().amax(-1, keepdim=True) / (6 * factor), e4m3)]
    code = e2m1[_nearest(torch.where(scale > 0, y.abs() / scale, 0.0), e2m1)]
    return (torch.sign(y) * code * scale).flatten(-2)


def _append(c, s):
    K, V, Q = s["K"].double(), s["V"].double(), s["Q"].double()
    for b, row, n, L in _rows(c):
        p = torch.arange(L - n, L, device=Q.device)
        K[row:row + n] = _held(_turn(K[row:row + n], s["rot"], p, c["kind"]), c["factor"])
        V[row:row + n] = _held(V[row:row + n], c["factor"])
        Q[row:row + n] = _turn(Q[row:row + n], s["rot"], p, c["kind"])
    return {"k": K, "v": V, "q": Q}


def _history(c, s, name, b, L):
    pages = s["table"][b, :-(-L // c["page"])].long()
    return gathered(s, name, pages, F64).reshape(-1, c["Hkv"], c["D"])[:L]


def _softmax(x, v):
    z = torch.logsumexp(x, -1)
    return torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None]) @ v, z


def _bias(table, d):
    return table.double()[torch.floor(2 * torch.log2(d.abs().double() + 1) + 1e-12).clamp(max=31).long()]


def _attend(c, s):
    g = c["H"] // c["Hkv"]
    O = torch.zeros(s["Q"].shape, dtype=F64, device=s["Q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=F64, device=s["Q"].device)
    for b, row, n, L in _rows(c):
        k, v = _history(c, s, "k", b, L), _history(c, s, "v", b, L)
        Q = s["Q"][row:row + n].double()
        at = torch.arange(n, device=k.device)[:, None] + (L - n)
        key = torch.arange(L, device=k.device)[None, :]
        hidden = (key > at) if c["causal"] else torch.zeros(n, L, dtype=torch.bool, device=k.device)
        if c["window"] >= 0:
            hidden |= key < at - c["window"]
        for h in range(c["H"]):
            x = Q[:, h] @ k[:, h // g].T / math.sqrt(c["D"])
            if s["bias"] is not None:
                x = x + _bias(s["bias"][h], at - key)
            O[row:row + n, h], lse[row:row + n, h] = _softmax(x.masked_fill(hidden, -math.inf), v[:, h // g])
    return {"o": O, "lse": lse}


def _select(c, s):
    P, g = c["page"], c["H"] // c["Hkv"]
    bounds = s["bounds"].double()
    chosen = torch.full(s["chosen"].shape, -1, dtype=torch.int32, device=bounds.device)
    for b, row, n, L in _rows(c):
        pages = s["table"][b].long()
        for at in range((L - n) // P, -(-L // P)):
            x = keys_of(s, pages[at:at + 1], F64)[0, :L - at * P]
            bounds[pages[at], :, 0], bounds[pages[at], :, 1] = x.amin(0), x.amax(0)
        pos = torch.arange(L - n, L, device=bounds.device)
        lo, hi = bounds[pages[:-(-L // P)]].unbind(2)                                   # [nb, Hkv, D]
        for h in range(c["Hkv"]):
            score = 0.0
            for q in s["Q"][row:row + n, h * g:(h + 1) * g].double().unbind(1):
                up = q > 0
                score = score + (q * up) @ hi[:, h].T + (q * ~up) @ lo[:, h].T          # [n, nb]
            k = torch.arange(score.shape[1], device=score.device)
            for i in range(n):
                last = int(pos[i]) // P
                seen = k[:last + 1]
                kept = (seen < c["first"]) | (seen > last - c["last"])
                rest = seen[~kept]
                best = torch.argsort(-score[i, rest], stable=True)[:max(0, c["n"] - int(kept.sum()))]
                both = torch.cat([seen[kept], rest[best]]).sort()[0]
                chosen[row + i, h, :both.numel()] = both.int()
    return {"bounds": bounds, "blocks": chosen}


def _blocks(c, s):
    g, P = c["H"] // c["Hkv"], c["page"]
    O = torch.zeros(s["Q"].shape, dtype=F64, device=s["Q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=F64, device=s["Q"].device)
    for b, row, n, L in _rows(c):
        k, v = _history(c, s, "k", b, L), _history(c, s, "v", b, L)
        at = torch.arange(n, device=k.device)[:, None] + (L - n)
        key = torch.arange(L, device=k.device)[None, :]
        for h in range(c["Hkv"]):
            listed_here = torch.zeros(n, -(-L // P) + 1, dtype=torch.bool, device=k.device)
            listed_here.scatter_(1, torch.where(s["lists"][row:row + n, h] >= 0, s["lists"][row:row + n, h].long(), -(-L // P)), True)
            seen = listed_here[:, :-1].repeat_interleave(P, 1)[:, :L] & (key <= at)
            for i in range(h * g, (h + 1) * g):
                x = s["Q"][row:row + n, i].double() @ k[:, h].T / math.sqrt(c["D"])
                if s["bias"] is not None:
                    x = x + _bias(s["bias"][i], at - key)
                O[row:row + n, i], lse[row:row + n, i] = _softmax(x.masked_fill(~seen, -math.inf), v[:, h])
    return {"o": O, "lse": lse}
