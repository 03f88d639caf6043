"""A paged cache held in 4 bits on a GPU: appending and reading against the format in 64 bits,
bit for bit, and attention against the CPU oracle on the values that the cache stands for."""
import numpy as np
import pytest
import torch

from cache_cases import Case, np64
from quant_cases import BF, CODES, E4M3, F32, F64, QCase, arrays, quantise, values

pytestmark = pytest.mark.gpu

SINGLE = ([1] * 9, [1, 2, 63, 64, 65, 127, 129, 700, 2049])
CHUNKS = ([5, 64, 130, 1, 300, 17], [5, 64, 131, 900, 1300, 777])
RAGGED = ([0, 1, 3, 0, 33, 1, 200, 2], [0, 1, 3, 40, 33, 513, 260, 1025])
EMPTY_ROWS = ([4, 70, 1, 300, 2], [2, 0, 0, 150, 2])  # more rows than keys; no key at all


@pytest.fixture(scope="module")
def jfa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from jagged_sequence_attention_gb300 import _build
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    return m


# ------------------------------------------------------------------ appending, reading

class Batch:
    """New tokens for a cache of `bits` (4, 16 or 32), and what the cache has to hold afterwards."""

    def __init__(self, q_lens, kv_lens, *, H=4, Hkv=2, D=64, page=16, R=0, kind="half", factors=(1.0, 1.0), layout="heads",
                 seed=0, std=1.0, bits=4):
        c = Case(q_lens, kv_lens, H=H, Hkv=Hkv, D=D, page=page, unset=False, seed=seed,
                 dtype=F32 if bits == 32 else BF)
        self.c, self.bits, self.factors, self.R, self.kind = c, bits, factors, R, kind
        g = torch.Generator(device="cuda").manual_seed(seed + 5)
        self.K, self.V = ((torch.randn(c.T, Hkv, D, generator=g, device="cuda", dtype=F32) * std).to(c.dtype) for _ in range(2))
        self.rot = None
        if R:
            a = torch.randn(max(kv_lens) + 3, R // 2, generator=g, device="cuda", dtype=F64) * 3
            self.rot = torch.cat([a.cos(), a.sin()], 1).float()
        if bits == 4:
            self.kc, self.ks = arrays(c.n_pages, page, Hkv, D, layout)
            self.vc, self.vs = arrays(c.n_pages, page, Hkv, D, layout)
            for x in (self.kc, self.ks, self.vc, self.vs):
                x.copy_(torch.randint(0, 127, x.shape, generator=g, device="cuda", dtype=torch.uint8))
        b = np.repeat(np.arange(len(q_lens)), q_lens)
        i = np.arange(c.T) - np.repeat(np.cumsum(q_lens) - q_lens, q_lens)
        self.pos = torch.from_numpy(i + (c.kv - c.q)[b]).cuda()
        self.pages = torch.from_numpy(c.host_table[b, self.pos.cpu().numpy() // page]).long().cuda()
        self.slots = self.pos % page

    def cache(self, jfa):
        if self.bits == 4:
            return jfa.jfa_cache_create_quantized(self.kc, self.vc, self.ks, self.vs, *self.factors)
        return jfa.jfa_cache_create(self.c.Kc, self.c.Vc)

    def turned(self, x):
        if self.rot is None:
            return x.double()
        t, y, h = self.rot.double()[self.pos][:, None], x.double(), self.R // 2
        cos, sin = t[..., :h], t[..., h:]
        a, b = (y[..., :h], y[..., h:self.R]) if self.kind == "half" else (y[..., 0:self.R:2], y[..., 1:self.R:2])
        u, v = a * cos - b * sin, b * cos + a * sin
        r = torch.cat([u, v], -1) if self.kind == "half" else torch.stack([u, v], -1).flatten(-2)
        return torch.cat([r, y[..., self.R:]], -1)


def check_append(jfa, b, **kw):
    want = []
    for x, codes, scales, f in ((b.turned(b.K), b.kc, b.ks, b.factors[0]), (b.V.double(), b.vc, b.vs, b.factors[1])):
        c, s = codes.clone(), scales.clone()
        c[b.pages, b.slots], s[b.pages, :, b.slots] = quantise(x, f)
        want.append((c, s))
    cache = b.cache(jfa)
    q = b.c.Q if b.R else None
    out = jfa.jfa_cache_append(cache, b.K, b.V, b.c.q_off, b.c.kv_lens, b.c.table, Q=q, rot=b.rot, rot_kind=b.kind, **kw)
    K, V = jfa.jfa_cache_read(cache, b.c.T, b.c.q_off, b.c.kv_lens, b.c.table)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
    for (c, s), codes, scales, f, rows in ((want[0], b.kc, b.ks, b.factors[0], K), (want[1], b.vc, b.vs, b.factors[1], V)):
        assert torch.equal(s, scales)
        # (a code of zero may have either sign)
        assert torch.equal(values(codes, scales.transpose(1, 2).contiguous(), f), values(c, s.transpose(1, 2).contiguous(), f))
        held = values(c[b.pages, b.slots], s[b.pages, :, b.slots].contiguous(), f)
        if f == 1.0:
            assert torch.equal(rows.double() + 0.0, held)  # exact in bf16
        else:
            assert bool(((rows.double() - held).abs() <= (2.0 ** -8 + 2.0 ** -23) * held.abs()).all())
    if q is not None:
        x = b.turned(q)
        # two products and a sum in fp32, then one rounding to bf16
        mag = q.double().abs().amax(-1, keepdim=True) * 2
        assert bool(((out.double() - x).abs() <= 2.0 ** -8 * x.abs() + 2.0 ** -22 * mag).all())


@pytest.mark.parametrize("D,R", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 32), (128, 80), (128, 128)])
@pytest.mark.parametrize("kind", ["half", "pairs"])
@pytest.mark.parametrize("lens", [SINGLE, CHUNKS, RAGGED], ids=["single", "chunks", "ragged"])
def test_append_is_exact(jfa, D, R, kind, lens):
    check_append(jfa, Batch(*lens, D=D, R=R, kind=kind, seed=D + R))


@pytest.mark.parametrize("factors", [(1.0, 1.0), (0.25, 8.0), (0.3, 1.7), (0.3125, 2.0 ** -20)])
@pytest.mark.parametrize("std", [1.0, 1e-3, 300.0, 1e5, 1e-20])
def test_append_factors_and_ranges(jfa, factors, std):
    f = tuple(float(np.float32(x)) for x in factors)
    for R in (0, 64):
        check_append(jfa, Batch(*CHUNKS, D=64, R=R, factors=f, std=std, seed=int(1000 * factors[0])))


@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
@pytest.mark.parametrize("page", [8, 16, 64, 1024])
def test_append_layouts(jfa, layout, page):
    for D in (64, 128):
        check_append(jfa, Batch(*RAGGED, D=D, page=page, Hkv=3, H=6, R=D, layout=layout, seed=page))


def test_append_ties_zeros_and_ends(jfa):
    b = Batch([300], [300], D=128, seed=3)
    # every multiple of a sixteenth below 7, so that all middles between codes are met, with a
    # scale of 1 (a six in each group); rows of zeros; the largest and smallest numbers
    x = (torch.arange(300 * 2 * 128, device="cuda") % 225 - 112).float().reshape(300, 2, 128) / 16
    x[..., 0::16] = 6.0
    x[10] = 0.0
    x[11, :, :16] = -0.0
    x[12] = 3.0e38
    x[13] = 1e-38
    x[14] *= 1e-2
    x[15, :, 3] = 2000.0
    x[16, :, 5] = -3.3e38
    b.K, b.V = x.to(BF), (-x).to(BF)
    check_append(jfa, b)
    # at position 0 the rotation is the identity, where its interval meets the ties
    b = Batch([1] * 40, [1] * 40, D=128, R=128, seed=4)
    b.K, b.V = x[:40].to(BF), (-x[:40]).to(BF)
    b.rot[0, :64], b.rot[0, 64:] = 1.0, 0.0
    check_append(jfa, b)


def test_append_takes_slices_and_queries_in_place(jfa):
    b = Batch(*CHUNKS, D=64, R=64, seed=5)
    wide = torch.randn(b.c.T, 4 + 2 + 2, 64, device="cuda", dtype=F32).to(BF)
    wide[:, 4:6], wide[:, 6:] = b.K, b.V
    q = wide[:, :4].clone()
    b.c.Q, b.K, b.V = q, wide[:, 4:6], wide[:, 6:]
    check_append(jfa, b)
    cache = b.cache(jfa)
    want = jfa.jfa_cache_append(cache, b.K, b.V, b.c.q_off, b.c.kv_lens, b.c.table, Q=q, rot=b.rot)
    got = jfa.jfa_cache_append(cache, b.K, b.V, b.c.q_off, b.c.kv_lens, b.c.table, Q=wide[:, :4], Q_out=wide[:, :4], rot=b.rot)
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [4, 16, 32])
def test_bad_sequences_are_left_alone(jfa, bits):
    b = Batch([2, 7, 1, 3], [40, 30, 9, 5], D=64, bits=bits, seed=6)
    cache = b.cache(jfa)
    held = [x.clone() for x in ((b.kc, b.ks, b.vc, b.vs) if bits == 4 else (b.c.Kc, b.c.Vc))]
    lens, table = b.c.kv_lens.clone(), b.c.table.clone()
    lens[1] = 6                    # fewer positions than tokens
    table[2, 0] = b.c.n_pages      # a page that there is not
    lens[3] = 10 ** 6              # more than the table has room for
    K = torch.full((b.c.T, 2, 64), 7.0, device="cuda", dtype=b.c.dtype)
    V = K.clone()
    jfa.jfa_cache_read(cache, b.c.T, b.c.q_off, lens, table, K=K, V=V)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS
    assert bool((K[2:] == 7).all()) and bool((V[2:] == 7).all()) and bool((K[:2] != 7).any())
    jfa.jfa_cache_append(cache, b.K, b.V, b.c.q_off, lens, table)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS
    mine = torch.zeros(b.c.n_pages, dtype=torch.bool, device="cuda")
    mine[b.c.table[0, :3].long()] = True
    for x, y in zip((b.kc, b.ks, b.vc, b.vs) if bits == 4 else (b.c.Kc, b.c.Vc), held):
        assert torch.equal(x[~mine], y[~mine]) and not torch.equal(x[mine], y[mine])


@pytest.mark.parametrize("bits,D", [(16, 64), (16, 128), (32, 32), (32, 64)])
def test_read_gives_whole_histories(jfa, bits, D):
    b = Batch(*RAGGED, D=D, Hkv=3, H=3, bits=bits, seed=7)
    off = torch.nn.functional.pad(b.c.kv_lens.cumsum(0), (1, 0)).int()
    n = int(b.c.kv.sum())
    wide = torch.full((n + 4, 8, D), 9.0, device="cuda", dtype=b.c.dtype)
    K, V = jfa.jfa_cache_read(b.cache(jfa), n + 4, off, b.c.kv_lens, b.c.table, K=wide[:, 1:4], V=wide[:, 5:])
    torch.cuda.synchronize()
    assert np.array_equal(np64(K)[:n], b.c.gathered(b.c.Kc)) and np.array_equal(np64(V)[:n], b.c.gathered(b.c.Vc))
    assert bool((wide[n:] == 9).all()) and bool((wide[:, 0] == 9).all()) and bool((wide[:, 4] == 9).all())


def test_read_rounds_once(jfa):
    """Factors whose products with a value lie next to the middle of two bf16 numbers, on the
    side that a product rounded to fp32 before would lose."""
    grid = torch.arange(127, dtype=torch.uint8).view(E4M3).double().numpy()
    held = np.unique(np.outer([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], grid[1:]).ravel())
    mids = (2 * np.arange(128, 256) + 1) / 512.0                     # middles of bf16 numbers in [0.5, 1)
    a = held[:, None] / 2.0 ** np.floor(np.log2(held))[:, None]
    f = (mids[None] / a).astype(np.float32)
    x = a * f.astype(np.float64)                                     # exact: 6 bits by 24
    near = (x != mids) & (x.astype(np.float32).astype(np.float64) == mids)
    below, above = near & (x < mids), near & (x > mids)
    assert below.sum() > 20 and above.sum() > 20
    for side in (below, above):
        for i, j in np.argwhere(side)[::max(1, side.sum() // 8)][:8]:
            factor = float(f[i, j])
            for bits in range(126, 0, -1):
                codes = [c for c in range(1, 8) if np.isclose(CODES[c] * grid[bits], held[i], rtol=0, atol=0)]
                if codes:
                    break
            k, ks = arrays(2, 16, 1, 64, "heads")
            k[1, 3, 0], ks[1, 0, 3] = codes[0] | ((codes[0] | 8) << 4), bits
            cache = jfa.jfa_cache_create_quantized(k, k.clone(), ks, ks.clone(), factor, factor)
            one = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
            K, V = jfa.jfa_cache_read(cache, 4, one(0, 4), one(20), one(0, 1).view(1, 2))
            value = held[i] * factor
            unit = 2.0 ** (np.floor(np.log2(value)) - 7)
            want = np.round(value / unit) * unit                     # (not a middle: no tie)
            got = np64(K)[3, 0]
            assert np.all(got[0::2] == want) and np.all(got[1::2] == -want) and torch.equal(K, V)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (6, 2), (5, 1), (16, 1), (24, 1)])
@pytest.mark.parametrize("lens", [SINGLE, CHUNKS, RAGGED], ids=["single", "chunks", "ragged"])
@pytest.mark.parametrize("D", [64, 128])
def test_head_groups(jfa, H, Hkv, lens, D):
    c = QCase(*lens, H=H, Hkv=Hkv, D=D, page=16, seed=H + D)
    c.check(*c.run(jfa))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 1024])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
def test_page_sizes_and_layouts(jfa, page, D, layout):
    for lens in (RAGGED, SINGLE):
        c = QCase(*lens, H=4, Hkv=2, D=D, page=page, layout=layout, seed=page)
        c.check(*c.run(jfa))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [SINGLE, CHUNKS, RAGGED, EMPTY_ROWS], ids=["single", "chunks", "ragged", "empty"])
@pytest.mark.parametrize("causal,window,bias", [(True, None, True), (True, 0, False), (True, 100, True),
                                                (True, 1000, False), (False, None, False), (False, None, True)])
def test_masks(jfa, D, lens, causal, window, bias):
    c = QCase(*lens, H=8, Hkv=2, D=D, page=16, causal=causal, window=window, bias=bias, seed=3)
    c.check(*c.run(jfa))


def test_out_types_strides_and_factors(jfa):
    for lens in (SINGLE, CHUNKS):
        for D, f in ((64, (0.25, 3.0)), (128, (0.3, 2.0 ** -30)), (128, (5.0, 7.0))):
            f = tuple(float(np.float32(x)) for x in f)
            c = QCase(*lens, H=4, Hkv=2, D=D, page=16, factors=f, seed=6)
            ref = c.reference()
            c.check(*c.run(jfa, out_dtype=F32), ref)
            wide = torch.full((c.T, 8, D), float("nan"), dtype=BF, device="cuda")
            wide[:, :4] = c.Q
            c.check(*c.run(jfa, Q=wide[:, :4]), ref)


def test_queries_of_any_size(jfa):
    # rows of tiny, ordinary and (with keys to match) huge queries; within a row magnitudes far apart
    for f in (1.0, 2.0 ** -40):
        c = QCase([1, 3, 2], [300, 700, 65], H=4, Hkv=2, D=128, page=16, factors=(f, 1.0), seed=8)
        s = torch.tensor([1e-38, 1e-30, 1e-12, 1.0, 1.0, 1e-3], device="cuda") / f
        c.Q = (c.Q.double() * s[:, None, None]).to(BF)
        c.Q[3, 1, 5:] *= 1e-9
        c.Q[4, 2] = 0.0
        c.check(*c.run(jfa))


@pytest.mark.parametrize("lens", [SINGLE, CHUNKS, EMPTY_ROWS], ids=["single", "chunks", "empty"])
def test_masks_hold_where_scores_vanish(jfa, lens):
    # queries and a scale whose product is below fp32's numbers: all scores are 0, masked ones still -inf
    c = QCase(*lens, H=4, Hkv=2, D=64, page=16, seed=12)
    c.Q = torch.full_like(c.Q, 1e-37)
    O, lse = c.run(jfa, scale=1e-36)
    c.Q = torch.zeros_like(c.Q)
    c.check(O, lse)


def test_large_scores(jfa):
    c = QCase(*CHUNKS, H=4, Hkv=2, D=128, page=16, seed=9, std=6.0)
    O, lse = c.run(jfa)
    ro, rl, A = c.reference()
    # as over a bf16 cache: scores of 2000, whose fp32 sums move p by at most 2e-3
    assert np.all(np.abs(np64(O) - ro) <= (2 * 2.0 ** -8 + 2e-3) * A + c.tiny() + 1e-30)
    assert np.abs(np64(lse) - rl).max() <= 2e-3


def test_long_histories_are_split(jfa):
    for H, Hkv, q in ((8, 8, 1), (8, 1, 1), (12, 1, 1), (4, 1, 4), (4, 2, 70)):
        c = QCase([q, 1], [20011, 3], H=H, Hkv=Hkv, D=128, page=64, seed=7)
        c.check(*c.run(jfa))


@pytest.mark.parametrize("H,Hkv", [(128, 1), (66, 1), (34, 2)])
def test_many_grouped_heads(jfa, H, Hkv):
    for lens in (([1, 1], [700, 40]), ([3, 17], [130, 500])):
        c = QCase(*lens, H=H, Hkv=Hkv, D=64, page=32, bias=True, seed=H)
        c.check(*c.run(jfa))


def test_many_sequences(jfa):
    rs = np.random.RandomState(1)
    for B in (33, 1500, 8192):
        kv = rs.randint(1, 90, B)
        q = np.minimum(kv, np.where(rs.rand(B) < 0.9, 1, rs.randint(0, 80, B)))
        c = QCase(q, kv, H=4, Hkv=2, D=64, page=16, seed=B)
        c.check(*c.run(jfa))


def test_query_bound_only_chooses_the_kernel(jfa):
    c = QCase(*RAGGED, H=8, Hkv=2, D=128, page=16, bias=True, seed=10)
    ro, rl, A = c.reference()
    for n in (0, 1, 4, 16, 200, 100000):
        O, lse = c.run(jfa, max_q_len=n)
        # (a longer sequence than announced runs in the few-rows kernel, a shorter one in none else)
        assert np.all(np.abs(np64(O) - ro) <= (2 * 2.0 ** -8 + 1e-4) * A + c.tiny() + 1e-30)
        assert np.abs(np64(lse) - rl).max() <= 1e-4


def test_cache_past_32_bits(jfa):
    # codes past byte 2^32, in appends, attention and reading
    page, Hkv, D = 64, 8, 128
    c = QCase([1, 70, 1], [200, 300, 900], H=16, Hkv=Hkv, D=D, page=page, seed=31)
    n_pages = 2 ** 32 // (page * Hkv * D // 2) + 40
    far = n_pages - c.n_pages
    near_table = c.table
    big = []
    for codes, scales in c.held:
        k, s = (torch.empty(n_pages, Hkv, page, D // n, dtype=torch.uint8, device="cuda") for n in (2, 16))
        k.transpose(1, 2)[far:], s[far:] = codes, scales
        big.append((k.transpose(1, 2), s))
    K, V = (torch.randn(c.T, Hkv, D, device="cuda", dtype=F32).to(BF) for _ in range(2))
    near, away = c.cache(jfa), jfa.jfa_cache_create_quantized(big[0][0], big[1][0], big[0][1], big[1][1])
    far_table = torch.where(near_table >= 0, near_table + far, near_table)
    out = []
    for cache, table in ((near, near_table), (away, far_table)):
        jfa.jfa_cache_append(cache, K, V, c.q_off, c.kv_lens, table)
        O, lse = jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, table, max_q_len=70)
        out.append((O, lse, *jfa.jfa_cache_read(cache, c.T, c.q_off, c.kv_lens, table)))
        torch.cuda.synchronize()
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
    for x, y in zip(*out):
        assert torch.equal(x, y)
    for (codes, scales), (k, s) in zip(c.held, big):
        assert torch.equal(k[far:], codes) and torch.equal(s[far:], scales)


def test_rows_behind_the_last_sequence_are_left(jfa):
    for lens in (SINGLE, CHUNKS):
        c = QCase(*lens, H=4, Hkv=2, D=128, page=16, pad_rows=19, seed=11)
        O = torch.full_like(c.Q, 7.0)
        lse = torch.full((c.T + 19, 4), 9.0, device="cuda", dtype=F32)
        c.run(jfa, O=O, lse=lse)
        assert bool((O[c.T:] == 7.0).all()) and bool((lse[c.T:] == 9.0).all())
        c.check(O, lse)


def test_same_bits_on_every_run_and_workspace_left_zero(jfa):
    for lens in (SINGLE, CHUNKS, ([1, 40], [30000, 9000])):
        c = QCase(*lens, H=8, Hkv=2, D=128, page=64, seed=12)
        cache = c.cache(jfa)
        ws = jfa.jfa_cache_workspace(cache, 8)
        O, lse = c.run(jfa, cache, workspace=ws)
        for _ in range(4):
            ws[jfa.JFA_CACHE_ZERO_BYTES:].random_(0, 255)
            O2, lse2 = c.run(jfa, cache, workspace=ws)
            assert torch.equal(O, O2) and torch.equal(lse, lse2)
            assert not bool(ws[:jfa.JFA_CACHE_ZERO_BYTES].any())


def test_bad_pages_and_sequences_are_reported(jfa):
    for lens in (SINGLE, CHUNKS):
        c = QCase(*lens, H=8, Hkv=2, D=128, page=16, seed=13)
        cache, ref = c.cache(jfa), c.reference()
        ws = jfa.jfa_cache_workspace(cache, 8)
        for bad in (c.n_pages, -1, 2 ** 31 - 1):
            table = c.table.clone()
            table[3, 0] = bad
            O, lse = jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, table, max_q_len=int(c.q.max()), workspace=ws)
            torch.cuda.synchronize()
            assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS
            a, z = int(c.q_off[3]), int(c.q_off[4])   # the other sequences' rows are right
            O[a:z], lse[a:z] = torch.from_numpy(ref[0][a:z]).to(O), torch.from_numpy(ref[1][a:z]).to(lse)
            c.check(O, lse, ref)
        lens2 = c.kv_lens.clone()
        lens2[3] = -5
        O = torch.full_like(c.Q, 7.0)
        jfa.jfa_cache_fwd(cache, c.Q, c.q_off, lens2, c.table, max_q_len=int(c.q.max()), workspace=ws, O=O)
        torch.cuda.synchronize()
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS
        assert bool((O[a:z] == 7.0).all())


def served_step(jfa, cache, b, H, ws, O, lse, **kw):
    q = jfa.jfa_cache_append(cache, b.K, b.V, b.c.q_off, b.c.kv_lens, b.c.table, Q=b.c.Q, rot=b.rot, **kw)
    return jfa.jfa_cache_fwd(cache, q, b.c.q_off, b.c.kv_lens, b.c.table, max_q_len=int(b.c.q.max()), workspace=ws, O=O,
                             lse=lse, **kw)


def test_prompts_then_tokens(jfa):
    """Sequences served step by step: what is attended over is what was appended, quantised."""
    H, Hkv, D, page = 8, 2, 128, 16
    steps = [([70, 33, 1], [70, 33, 1]), ([1, 40, 1], [71, 73, 2]), ([1, 1, 1], [72, 74, 3]), ([3, 0, 2], [75, 74, 5])]
    b = Batch(*steps[-1], H=H, Hkv=Hkv, D=D, page=page, R=D, seed=20)
    cache, ws = b.cache(jfa), None
    ws = jfa.jfa_cache_workspace(cache, H)
    for n, (q, kv) in enumerate(steps):
        s = Batch(q, kv, H=H, Hkv=Hkv, D=D, page=page, R=D, seed=21 + n)
        s.rot, s.c.table = torch.cat([b.rot, b.rot])[:80], b.c.table
        O, lse = served_step(jfa, cache, s, H, ws, torch.empty_like(s.c.Q), None)
        c = QCase.__new__(QCase)
        c.__dict__.update(s.c.__dict__)
        c.host_table = b.c.host_table
        c.Kc = values(b.kc, b.ks.transpose(1, 2).contiguous(), 1.0)
        c.Vc = values(b.vc, b.vs.transpose(1, 2).contiguous(), 1.0)
        c.Q = jfa.jfa_cache_append(cache, s.K, s.V, s.c.q_off, s.c.kv_lens, s.c.table, Q=s.c.Q, rot=s.rot)
        c.check(O, lse)
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK


def test_captured_step_on_new_contents(jfa):
    H, Hkv, D = 8, 2, 128
    b = Batch(*CHUNKS, H=H, Hkv=Hkv, D=D, R=D, seed=30)
    cache = b.cache(jfa)
    ws = jfa.jfa_cache_workspace(cache, H)
    O, lse = torch.empty_like(b.c.Q), torch.empty(b.c.T, H, device="cuda", dtype=F32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        served_step(jfa, cache, b, H, ws, O, lse)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        served_step(jfa, cache, b, H, ws, O, lse)
    for n in range(3):
        b.K.copy_(torch.randn(b.K.shape, device="cuda", dtype=F32))
        b.V.copy_(torch.randn(b.V.shape, device="cuda", dtype=F32))
        b.c.Q.copy_(torch.randn(b.c.Q.shape, device="cuda", dtype=F32))
        if n == 2:  # other lengths, within the announced bound
            b.c.kv_lens.copy_(torch.tensor([5, 64, 130, 880, 1290, 700], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got, got_lse = O.clone(), lse.clone()
        served_step(jfa, cache, b, H, ws, O, lse)
        torch.cuda.synchronize()
        assert torch.equal(got, O) and torch.equal(got_lse, lse)
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK


def test_calls_at_once_on_two_streams(jfa):
    c = QCase(*CHUNKS, H=8, Hkv=2, D=128, page=16, seed=32)
    cache = c.cache(jfa)
    want, want_lse = c.run(jfa, cache)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [jfa.jfa_cache_workspace(cache, 8) for _ in range(2)]
    torch.cuda.synchronize()
    out = []
    for _ in range(10):
        for s, ws in zip(streams, spaces):
            out.append(jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, c.table, max_q_len=300, workspace=ws, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(O, want) and torch.equal(lse, want_lse) for O, lse in out)


def test_refusals(jfa):
    def status(fn, *a, **k):
        try:
            fn(*a, **k)
        except jfa.JFAError as e:
            return e.status
        return jfa.JFA_OK

    c = QCase(*SINGLE, H=4, Hkv=2, D=128, page=16, seed=14)
    (k, ks), (v, vs) = c.held
    make, bad = jfa.jfa_cache_create_quantized, jfa.JFA_ERR_INVALID_ARG
    assert status(make, k, v, ks, vs) == jfa.JFA_OK and status(make, k, v, ks.view(E4M3), vs.view(E4M3)) == jfa.JFA_OK
    for args in ((k.float(), v, ks, vs), (k, v[1:], ks, vs), (k, v, ks[1:], vs), (k, v, ks.transpose(1, 2), vs),
                 (k, v, ks, vs.float()), (k.cpu(), v, ks, vs), (k, v, ks, vs.cpu()), (k[..., ::2], v[..., ::2], ks, vs)):
        assert status(make, *args) == bad
    for f in (0.0, -1.0, float("nan"), float("inf"), 1e-30, 1e30):
        assert status(make, k, v, ks, vs, f) == bad and status(make, k, v, ks, vs, 1.0, f) == bad
    odd = torch.zeros(4, 2, 24, 64, dtype=torch.uint8, device="cuda").transpose(1, 2)
    assert status(make, odd, odd, *([torch.zeros(4, 2, 24, 8, dtype=torch.uint8, device="cuda")] * 2)) == jfa.JFA_ERR_UNSUPPORTED
    cache = c.cache(jfa)
    fwd = lambda **kw: status(jfa.jfa_cache_fwd, cache, kw.pop("Q", c.Q), c.q_off, c.kv_lens, c.table, **kw)  # noqa: E731
    assert fwd() == jfa.JFA_OK
    assert fwd(Q=c.Q.float()) == bad and fwd(scale=0.0) == bad and fwd(scale=1e38) == bad
    assert fwd(O=torch.empty_like(c.Q, dtype=torch.float16)) == jfa.JFA_ERR_UNSUPPORTED
    read = lambda T, **kw: status(jfa.jfa_cache_read, cache, T, c.q_off, c.kv_lens, c.table, **kw)  # noqa: E731
    assert read(c.T) == jfa.JFA_OK and read(-1, K=c.Q[:, :2].contiguous(), V=c.Q[:, :2].contiguous()) == bad
    assert read(c.T, K=torch.empty(c.T, 2, 128, device="cuda"), V=torch.empty(c.T, 2, 128, device="cuda")) == bad
    assert read(c.T, K=c.Q, V=c.Q) == bad
