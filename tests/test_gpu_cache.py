"""Paged-cache attention and appending on a GPU against the CPU oracle: head groups, page
sizes, layouts, masks that leave rows empty, undefined slots, ragged and empty sequences,
graphs and streams, and the refusals."""
import ctypes

import numpy as np
import pytest
import torch

from cache_cases import FP32_SLACK, Case, np64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def jfa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from jagged_sequence_attention_gb300 import _build
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    return m


def status_of(jfa, fn, *a, **k):
    try:
        fn(*a, **k)
    except jfa.JFAError as e:
        return e.status
    return jfa.JFA_OK


# ------------------------------------------------------------------ attention: parity

SINGLE = ([1] * 9, [1, 2, 63, 64, 65, 127, 129, 700, 2049])
CHUNKS = ([5, 64, 130, 1, 300, 17], [5, 64, 131, 900, 1300, 777])
RAGGED = ([0, 1, 3, 0, 33, 1, 200, 2], [0, 1, 3, 40, 33, 513, 260, 1025])
EMPTY_ROWS = ([4, 70, 1, 300, 2], [2, 0, 0, 150, 2])  # more rows than keys; no key at all


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (6, 2), (5, 1), (16, 1), (24, 1)])
@pytest.mark.parametrize("lens", [SINGLE, CHUNKS, RAGGED], ids=["single", "chunks", "ragged"])
@pytest.mark.parametrize("D", [64, 128])
def test_head_groups(jfa, H, Hkv, lens, D):
    c = Case(*lens, H=H, Hkv=Hkv, D=D, page=16, seed=H + D)
    c.check(*c.run(jfa))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64), (F32, 32)])
def test_page_sizes(jfa, page, dtype, D):
    c = Case(*RAGGED, H=4, Hkv=2, D=D, page=page, dtype=dtype, seed=page)
    c.check(*c.run(jfa))
    c = Case(*SINGLE, H=4, Hkv=2, D=D, page=page, dtype=dtype, seed=page + 1)
    c.check(*c.run(jfa))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64), (F32, 32)])
@pytest.mark.parametrize("lens", [SINGLE, CHUNKS, RAGGED, EMPTY_ROWS], ids=["single", "chunks", "ragged", "empty"])
@pytest.mark.parametrize("causal,window,bias", [(True, None, True), (True, 0, False), (True, 100, True),
                                                (True, 1000, False), (True, 10 ** 9, False), (False, None, False),
                                                (False, None, True)])
def test_masks(jfa, dtype, D, lens, causal, window, bias):
    c = Case(*lens, H=8, Hkv=2, D=D, page=16, dtype=dtype, causal=causal, window=window, bias=bias, seed=3)
    c.check(*c.run(jfa))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("layout", ["heads", "both"])
def test_layouts(jfa, dtype, D, layout):
    for lens in (SINGLE, CHUNKS):
        c = Case(*lens, H=8, Hkv=4, D=D, page=32, dtype=dtype, layout=layout, seed=5)
        c.check(*c.run(jfa))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_out_types_and_row_strides(jfa, dtype, D):
    for lens in (SINGLE, CHUNKS):
        c = Case(*lens, H=4, Hkv=2, D=D, page=16, dtype=dtype, seed=6)
        ref = c.reference()
        c.check(*c.run(jfa, out_dtype=F32), ref)
        wide = torch.full((c.T, 4 + 2 + 2, D), float("nan"), dtype=dtype, device="cuda")
        wide[:, :4] = c.Q
        c.check(*c.run(jfa, Q=wide[:, :4]), ref)


def test_long_history_is_split(jfa):
    for H, Hkv, q in ((8, 8, 1), (8, 1, 1), (4, 1, 70), (4, 2, 300)):
        c = Case([q, 1], [20011, 3], H=H, Hkv=Hkv, D=128, page=64, seed=7)
        c.check(*c.run(jfa))
    c = Case([1], [9001], H=3, Hkv=1, D=64, page=8, dtype=F32, seed=8)
    c.check(*c.run(jfa))


@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (12, 1)])
@pytest.mark.parametrize("D", [32, 64])
@pytest.mark.parametrize("causal", [True, False])
def test_fp32_products_are_fp32(jfa, H, Hkv, D, causal):
    # single tokens (CUDA cores), short sets, and chunks (tensor cores on split operands)
    c = Case([1, 3, 40, 130, 300], [900, 64, 41, 700, 2500], H=H, Hkv=Hkv, D=D, page=16, dtype=F32, causal=causal, seed=30)
    c.check(*c.run(jfa), slack=FP32_SLACK)


@pytest.mark.parametrize("H,Hkv", [(128, 1), (100, 1), (66, 1), (34, 2)])
def test_many_grouped_heads(jfa, H, Hkv):
    for lens in (([1, 1], [700, 40]), ([3, 17], [130, 500])):
        for bias in (False, True):
            c = Case(*lens, H=H, Hkv=Hkv, D=64, page=32, bias=bias, seed=H)
            c.check(*c.run(jfa))
    c = Case([1, 5], [70, 300], H=H, Hkv=Hkv, D=32, page=32, dtype=F32, seed=H)
    c.check(*c.run(jfa))


def test_cache_past_32_bits(jfa):
    # pages whose elements lie past 2^31 (and bytes past 2^32), in reads and in appends
    page, Hkv, D = 64, 8, 128
    n_pages = 2 ** 31 // (page * Hkv * D) + 40
    q, kv = [1, 70, 1], [200, 300, 900]
    c = append_case(q, kv, H=16, Hkv=Hkv, D=D, page=page, dtype=BF, R=D, kind="half", seed=31)
    small_k, small_v, table = c.Kc, c.Vc, c.host_table.copy()
    far = n_pages - small_k.shape[0]
    c.Kc = torch.empty(n_pages, page, Hkv, D, dtype=BF, device="cuda")
    c.Vc = torch.empty(n_pages, page, Hkv, D, dtype=BF, device="cuda")
    c.Kc[far:], c.Vc[far:] = small_k, small_v
    c.host_table = np.where(table >= 0, table + far, table).astype(np.int32)
    c.table = torch.from_numpy(c.host_table).cuda()
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    c.Q = jfa.jfa_cache_append(cache, c.K, c.V, c.q_off, c.kv_lens, c.table, Q=c.Q, rot=c.rot)
    O, lse = c.run(jfa, cache)
    # the same on the small copy
    near = jfa.jfa_cache_create(small_k, small_v)
    t0 = torch.from_numpy(table).cuda()
    jfa.jfa_cache_append(near, c.K, c.V, c.q_off, c.kv_lens, t0, rot=c.rot)
    O2, lse2 = jfa.jfa_cache_fwd(near, c.Q, c.q_off, c.kv_lens, t0, max_q_len=70)
    torch.cuda.synchronize()
    assert torch.equal(c.Kc[far:], small_k) and torch.equal(c.Vc[far:], small_v)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    c.Kc, c.Vc, c.host_table = small_k, small_v, table
    c.check(O, lse)


def test_many_sequences(jfa):
    rs = np.random.RandomState(1)
    for B, dtype in ((33, BF), (300, BF), (1500, BF), (1025, F32), (8192, BF)):
        kv = rs.randint(1, 90, B)
        q = np.minimum(kv, np.where(rs.rand(B) < 0.9, 1, rs.randint(0, 80, B)))
        c = Case(q, kv, H=4, Hkv=2, D=64, page=16, dtype=dtype, seed=B)
        c.check(*c.run(jfa))


def test_large_scores(jfa):
    # scores of several hundred: the running maximum moves far between key tiles
    c = Case(*CHUNKS, H=4, Hkv=2, D=128, page=16, seed=9, std=6.0)
    O, lse = c.run(jfa)
    ro, rl, A = c.reference()
    # scores reach 36 * 11.3 * 5 ~ 2000; their fp32 sums err by 2^-24 of the terms' sum
    # 128 * 36 * 0.64 / 11.3 = 260 times at most 128, so p by at most 2e-3 in the worst order
    assert np.all(np.abs(np64(O) - ro) <= (2 * 2.0 ** -8 + 2e-3) * A + 1e-30)
    assert np.abs(np64(lse) - rl).max() <= 2e-3


def test_query_bound_only_chooses_the_kernel(jfa):
    c = Case(*RAGGED, H=8, Hkv=2, D=128, page=16, bias=True, seed=10)
    ref = c.reference()
    for n in (0, 1, 4, 16, 200, 100000):
        c.check(*c.run(jfa, max_q_len=n), ref)


def test_rows_behind_the_last_sequence_are_left(jfa):
    for dtype, D in ((BF, 128), (F32, 64)):
        for lens in (SINGLE, CHUNKS):
            c = Case(*lens, H=4, Hkv=2, D=D, page=16, dtype=dtype, pad_rows=19, seed=11)
            O = torch.full_like(c.Q, 7.0)
            lse = torch.full((c.T + 19, 4), 9.0, device="cuda", dtype=F32)
            c.run(jfa, O=O, lse=lse)
            assert bool((O[c.T:] == 7.0).all()) and bool((lse[c.T:] == 9.0).all())
            c.check(O, lse)


def test_same_bits_on_every_run_and_workspace_left_zero(jfa):
    for lens in (SINGLE, CHUNKS, ([1, 40], [30000, 9000])):
        c = Case(*lens, H=8, Hkv=2, D=128, page=64, seed=12)
        cache = jfa.jfa_cache_create(c.Kc, c.Vc)
        ws = jfa.jfa_cache_workspace(cache, 8)
        O, lse = c.run(jfa, cache, workspace=ws)
        for _ in range(4):
            ws[jfa.JFA_CACHE_ZERO_BYTES:].random_(0, 255)
            O2, lse2 = c.run(jfa, cache, workspace=ws)
            assert torch.equal(O, O2) and torch.equal(lse, lse2)
            assert not bool(ws[:jfa.JFA_CACHE_ZERO_BYTES].any())


def test_shared_pages_are_read_by_many(jfa):
    # query sets over one user's history: rows of the page table repeat
    c = Case([7, 40, 1], [500, 500, 500], H=4, Hkv=4, D=64, page=32, causal=False, unset=False, seed=13)
    c.table[1:] = c.table[0]
    c.host_table[1:] = c.host_table[0]
    c.check(*c.run(jfa))


# ------------------------------------------------------------------ attention: bad contents

@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
@pytest.mark.parametrize("q", [1, 90])
def test_bad_contents_are_reported(jfa, dtype, D, q):
    def fresh():
        return Case([q, q, q], [300, 200, 100], H=4, Hkv=2, D=D, page=16, dtype=dtype, seed=14)

    def run(c):
        cache = jfa.jfa_cache_create(c.Kc, c.Vc)
        O = torch.full_like(c.Q, 5.0)
        jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, c.table, max_q_len=q, O=O)
        torch.cuda.synchronize()
        first = jfa.jfa_cache_device_status(cache)
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK  # read and cleared
        return O, first

    good, st = run(fresh())
    assert st == jfa.JFA_OK
    for page in (-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1):
        c = fresh()
        c.table[1, 3] = page
        O, st = run(c)
        assert st == jfa.JFA_ERR_DEVICE_BOUNDS
        assert torch.equal(O[:q], good[:q]) and torch.equal(O[2 * q:], good[2 * q:])
    for n in (-1, 10 ** 9, -2 ** 31):
        c = fresh()
        c.kv_lens[1] = n
        O, st = run(c)
        assert st == jfa.JFA_ERR_DEVICE_BOUNDS
        assert bool((O[q:2 * q] == 5.0).all())
    c = fresh()
    c.q_off[3] = 10 ** 8
    O, st = run(c)
    assert st == jfa.JFA_ERR_DEVICE_BOUNDS and torch.equal(O[:2 * q], good[:2 * q])
    c = fresh()
    c.q_off[1] = -7
    assert run(c)[1] == jfa.JFA_ERR_DEVICE_BOUNDS


# ------------------------------------------------------------------ appending

def rotated64(x, table, pos, kind):
    """x [n, heads, D] in 64 bits, and the sum of the terms' magnitudes."""
    R = table.shape[1]
    cos, sin = table[pos][:, None, :R // 2], table[pos][:, None, R // 2:]
    y, mag = x.copy(), np.zeros_like(x)
    ia, ib = (slice(0, R // 2), slice(R // 2, R)) if kind == "half" else (slice(0, R, 2), slice(1, R, 2))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    mag[..., ia], mag[..., ib] = np.abs(a * cos) + np.abs(b * sin), np.abs(b * cos) + np.abs(a * sin)
    return y, mag


def make_table(n, R):
    f = 10000.0 ** (-np.arange(R // 2) / (R // 2))
    a = np.arange(n)[:, None] * f
    return torch.tensor(np.concatenate([np.cos(a), np.sin(a)], 1), dtype=torch.float32, device="cuda")


def append_case(q, kv, *, H, Hkv, D, page, dtype, R, kind, layout="tokens", seed=0, pad_rows=0):
    c = Case(q, kv, H=H, Hkv=Hkv, D=D, page=page, dtype=dtype, layout=layout, unset=False, seed=seed,
             pad_rows=pad_rows)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.K = torch.randn(c.T + pad_rows, Hkv, D, generator=g, device="cuda", dtype=F32).to(dtype)
    c.V = torch.randn(c.T + pad_rows, Hkv, D, generator=g, device="cuda", dtype=F32).to(dtype)
    c.rot = make_table(max(1, int(max(kv))), R) if R else None
    c.kind = kind
    return c


def check_append(jfa, c, Q_out=None, K=None, V=None, Q=None):
    k0, v0 = c.Kc.clone(), c.Vc.clone()
    q_in = np64(c.Q)
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    rot = c.rot is not None
    out = jfa.jfa_cache_append(cache, c.K if K is None else K, c.V if V is None else V, c.q_off, c.kv_lens, c.table,
                               Q=(c.Q if Q is None else Q) if rot else None, Q_out=Q_out, rot=c.rot, rot_kind=c.kind)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
    pos = np.concatenate([np.arange(kv - q, kv) for q, kv in zip(c.q, c.kv)]).astype(np.int64)
    seq = np.repeat(np.arange(c.q.size), c.q)
    page, slot = c.host_table[seq, pos // c.page], pos % c.page
    # the values are stored as they are, and nothing else changes
    v0[page, slot] = c.V[:c.T]
    assert torch.equal(v0, c.Vc)
    got = np64(c.Kc)[page, slot]
    k0[page, slot] = c.Kc[page, slot]
    assert torch.equal(k0, c.Kc)
    if not rot:
        assert torch.equal(c.Kc[page, slot], c.K[:c.T])
        return out
    # two products and a sum in fp32 (2^-24 of each term, and of the sum), one rounding
    half = 2.0 ** -8 if c.dtype == BF else 2.0 ** -24
    for x, y in ((np64(c.K)[:c.T], got), (q_in[:c.T], np64(out)[:c.T])):
        ref, mag = rotated64(x, np64(c.rot), pos, c.kind)
        assert np.all(np.abs(y - ref) <= half * np.abs(ref) + 3 * 2.0 ** -24 * mag * (1 + half) + 1e-38)
    return out


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64), (F32, 32)])
@pytest.mark.parametrize("kind", ["half", "pairs"])
@pytest.mark.parametrize("R", [0, 16, 32, "D"])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (3, 3), (5, 1)])
def test_append(jfa, dtype, D, kind, R, H, Hkv):
    R = D if R == "D" else R
    q, kv = [1, 0, 40, 1, 7, 200], [1, 10, 40, 513, 100, 300]
    check_append(jfa, append_case(q, kv, H=H, Hkv=Hkv, D=D, page=16, dtype=dtype, R=R, kind=kind, seed=D + H))


@pytest.mark.parametrize("page", [8, 64, 1024])
@pytest.mark.parametrize("layout", ["tokens", "heads", "both"])
def test_append_pages_and_layouts(jfa, page, layout):
    q, kv = [1, 90, 33], [65, 90, 2000]
    check_append(jfa, append_case(q, kv, H=4, Hkv=2, D=128, page=page, dtype=BF, R=64, kind="half", layout=layout))


@pytest.mark.parametrize("B", [1, 31, 32, 33, 1023, 1025, 5000])
def test_append_finds_its_sequence(jfa, B):
    rs = np.random.RandomState(B)
    q = rs.randint(0, 3, B)
    q[rs.randint(B)] = 9
    kv = q + rs.randint(0, 30, B)
    c = append_case(q, kv, H=2, Hkv=1, D=64, page=8, dtype=BF, R=64, kind="half", seed=B, pad_rows=5)
    out = torch.full_like(c.Q, 3.0)
    check_append(jfa, c, Q_out=out)
    assert bool((out[c.T:] == 3.0).all())


def test_append_in_place_and_from_a_fused_projection(jfa):
    for kind in ("half", "pairs"):
        c = append_case([1, 50, 3], [9, 50, 700], H=4, Hkv=2, D=128, page=16, dtype=BF, R=128, kind=kind)
        check_append(jfa, c, Q_out=c.Q)
        c = append_case([1, 50, 3], [9, 50, 700], H=4, Hkv=2, D=128, page=16, dtype=BF, R=128, kind=kind)
        wide = torch.cat([c.Q, c.K, c.V], 1)
        check_append(jfa, c, Q=wide[:, :4], K=wide[:, 4:6], V=wide[:, 6:])


def test_append_bad_contents_are_reported(jfa):
    def fresh():
        return append_case([2, 3], [40, 50], H=4, Hkv=2, D=64, page=8, dtype=BF, R=64, kind="half")

    def run(c):
        cache = jfa.jfa_cache_create(c.Kc, c.Vc)
        jfa.jfa_cache_append(cache, c.K, c.V, c.q_off, c.kv_lens, c.table, Q=c.Q, rot=c.rot)
        torch.cuda.synchronize()
        return jfa.jfa_cache_device_status(cache)

    c = fresh()
    assert run(c) == jfa.JFA_OK
    for page in (-1, 10 ** 6, -2 ** 31):
        c = fresh()
        before = c.Kc.clone()
        c.table[1, 47 // 8:] = page
        assert run(c) == jfa.JFA_ERR_DEVICE_BOUNDS
        p0 = c.host_table[0, 38 // 8]
        before[p0, 38 % 8:38 % 8 + 2] = c.Kc[p0, 38 % 8:38 % 8 + 2]
        assert torch.equal(before, c.Kc)  # only the good sequence's tokens were written
    for n in (-1, 1, 10 ** 9):  # a length below the new tokens, or past the table
        c = fresh()
        c.kv_lens[0] = n
        assert run(c) == jfa.JFA_ERR_DEVICE_BOUNDS
    c = fresh()
    c.rot = c.rot[:45].contiguous()  # a position past the rotation's table
    assert run(c) == jfa.JFA_ERR_DEVICE_BOUNDS
    c = fresh()
    c.q_off[2] = 10 ** 8
    assert run(c) == jfa.JFA_ERR_DEVICE_BOUNDS


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_served_steps_equal_the_whole_sequence(jfa, dtype, D):
    """A model's sequences served in steps (a prompt, chunks, single tokens; append, then
    attend) give what the oracle gives for the whole causal sequences."""
    H, Hkv, page, R = 4, 2, 16, 32
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [150, 71, 5]
    B, T = len(lens), sum(lens)
    off = np.concatenate([[0], np.cumsum(lens)])
    X = {n: torch.randn(T, h, D, generator=g, device="cuda", dtype=F32).to(dtype) for n, h in (("Q", H), ("K", Hkv), ("V", Hkv))}
    rot, bias = make_table(max(lens), R), torch.randn(H, 32, generator=g, device="cuda", dtype=F32)
    n_pages = sum(-(-n // page) for n in lens)
    Kc = torch.full((n_pages, page, Hkv, D), float("nan"), dtype=dtype, device="cuda")
    Vc = torch.full_like(Kc, float("nan"))
    cache = jfa.jfa_cache_create(Kc, Vc)
    ws = jfa.jfa_cache_workspace(cache, H)
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    free = list(np.random.RandomState(0).permutation(n_pages))
    done, got, rq = [0] * B, torch.empty(T, H, D, dtype=dtype, device="cuda"), torch.empty_like(X["Q"])
    for step in ([60, 71, 0], [1, 0, 4], [50, 0, 1], [1, 0, 0], [1, 0, 0], [37, 0, 0]):
        rows = np.concatenate([np.arange(off[b] + done[b], off[b] + done[b] + n) for b, n in enumerate(step)])
        for b, n in enumerate(step):
            for p in range(-(-done[b] // page), -(-(done[b] + n) // page)):
                table[b, p] = int(free.pop())
            done[b] += n
        idx = torch.from_numpy(rows).cuda()
        q_off = torch.tensor(np.concatenate([[0], np.cumsum(step)]), dtype=torch.int32, device="cuda")
        kv = torch.tensor(done, dtype=torch.int32, device="cuda")
        q = jfa.jfa_cache_append(cache, X["K"][idx], X["V"][idx], q_off, kv, table, Q=X["Q"][idx], rot=rot)
        rq[idx] = q
        got[idx] = jfa.jfa_cache_fwd(cache, q, q_off, kv, table, bias=bias, max_q_len=max(step), workspace=ws)[0]
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK and done == lens
    c = Case(lens, lens, H=H, Hkv=Hkv, D=D, page=page, dtype=dtype, bias=True)
    c.Q, c.Kc, c.Vc, c.bias, c.host_table, c.table = rq, Kc, Vc, bias, table.cpu().numpy(), table
    ref = c.reference()
    lse = torch.from_numpy(ref[1])
    c.check(got, lse, ref)


def test_a_captured_step_is_replayed_on_new_contents(jfa):
    """One graph of append and attention, replayed as the sequences grow, while the same
    handle serves an eager call on another stream."""
    B, H, Hkv, D, page = 5, 8, 2, 128, 16
    c = append_case([1] * B, [30, 40, 50, 600, 1], H=H, Hkv=Hkv, D=D, page=page, dtype=BF, R=D, kind="half")
    c.rot = make_table(700, D)
    n = 60
    Kc = torch.zeros(n * B, page, Hkv, D, dtype=BF, device="cuda")
    Vc = torch.zeros_like(Kc)
    Kc.normal_(), Vc.normal_()
    table = torch.randperm(n * B, device="cuda").int().view(B, n).contiguous()
    cache = jfa.jfa_cache_create(Kc, Vc)
    ws = jfa.jfa_cache_workspace(cache, H)
    O, lse, q = torch.empty_like(c.Q), torch.empty(B, H, device="cuda", dtype=F32), torch.empty_like(c.Q)

    def step():
        jfa.jfa_cache_append(cache, c.K, c.V, c.q_off, c.kv_lens, table, Q=c.Q, Q_out=q, rot=c.rot)
        jfa.jfa_cache_fwd(cache, q, c.q_off, c.kv_lens, table, max_q_len=1, O=O, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = Case(*CHUNKS, H=H, Hkv=Hkv, D=D, page=page, seed=20)
    other_cache = jfa.jfa_cache_create(other.Kc, other.Vc)
    other_ref = other.reference()
    for k in range(4):
        c.kv_lens += 1
        c.K.normal_(), c.V.normal_(), c.Q.normal_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            eo, el = jfa.jfa_cache_fwd(other_cache, other.Q, other.q_off, other.kv_lens, other.table, max_q_len=300)
        torch.cuda.synchronize()
        other.check(eo, el, other_ref)
        chk = Case([1] * B, c.kv_lens.cpu().numpy(), H=H, Hkv=Hkv, D=D, page=page)
        chk.Q, chk.Kc, chk.Vc, chk.table, chk.host_table = q, Kc, Vc, table, table.cpu().numpy()
        chk.check(O, lse)
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_a_captured_mixed_batch_is_replayed_on_new_lengths(jfa, dtype, D):
    """One graph over every kernel of a mixed batch; between replays the offsets, lengths and
    page table change, so sequences move between the kernels."""
    H, Hkv, page, T = 4, 2, 16, 500
    Q = torch.randn(T, H, D, device="cuda", dtype=F32).to(dtype)
    Kc = torch.randn(400, page, Hkv, D, device="cuda", dtype=F32).to(dtype)
    Vc = torch.randn(400, page, Hkv, D, device="cuda", dtype=F32).to(dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    off, kv, table = torch.zeros(6, **i32), torch.zeros(5, **i32), torch.zeros(5, 100, **i32)
    cache = jfa.jfa_cache_create(Kc, Vc)
    ws = jfa.jfa_cache_workspace(cache, H)
    O, lse = torch.empty_like(Q), torch.empty(T, H, device="cuda", dtype=F32)

    def step():
        jfa.jfa_cache_fwd(cache, Q, off, kv, table, O=O, lse=lse, workspace=ws)  # (no bound on the query lengths)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rs = np.random.RandomState(5)
    for q, n in (([1, 300, 1, 0, 40], [900, 1300, 30, 77, 640]), ([1] * 5, [100, 1, 1500, 16, 17]),
                 ([0, 0, 0, 0, 500], [0, 5, 0, 0, 500]), ([90, 10, 300, 20, 80], [1500, 900, 301, 20, 1200])):
        off.copy_(torch.tensor(np.concatenate([[0], np.cumsum(q)])))
        kv.copy_(torch.tensor(n))
        table.copy_(torch.from_numpy(np.stack([rs.permutation(400)[:100] for _ in range(5)])))
        O.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
        c = Case(q, n, H=H, Hkv=Hkv, D=D, page=page, dtype=dtype)
        c.Q, c.Kc, c.Vc, c.table, c.host_table = Q, Kc, Vc, table, table.cpu().numpy()
        c.check(O, lse)
        assert bool((O[c.T:] == 3.0).all()) and not bool(ws[:jfa.JFA_CACHE_ZERO_BYTES].any())


def test_two_calls_at_once_on_one_handle(jfa):
    c = Case([1, 1, 200], [9000, 17, 5000], H=8, Hkv=2, D=128, page=64, seed=21)
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    ref = c.reference()
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [jfa.jfa_cache_workspace(cache, 8) for _ in streams]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, ws in zip(streams, spaces):
            with torch.cuda.stream(s):
                outs.append(jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, c.table, max_q_len=200, workspace=ws))
    torch.cuda.synchronize()
    for O, lse in outs:
        assert torch.equal(O, outs[0][0]) and torch.equal(lse, outs[0][1])
    c.check(*outs[0], ref)


# ------------------------------------------------------------------ refusals

def test_refusals(jfa):
    c = append_case([1, 5], [9, 50], H=4, Hkv=2, D=64, page=16, dtype=BF, R=32, kind="half")
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    ws = jfa.jfa_cache_workspace(cache, 4)
    bad, uns = jfa.JFA_ERR_INVALID_ARG, jfa.JFA_ERR_UNSUPPORTED

    def fwd(**k):
        a = dict(cache=cache, Q=c.Q, q_offsets=c.q_off, kv_lens=c.kv_lens, page_table=c.table, workspace=ws)
        a.update(k)
        return status_of(jfa, jfa.jfa_cache_fwd, **a)

    def app(**k):
        a = dict(cache=cache, K=c.K, V=c.V, q_offsets=c.q_off, kv_lens=c.kv_lens, page_table=c.table, Q=c.Q, rot=c.rot)
        a.update(k)
        return status_of(jfa, jfa.jfa_cache_append, **a)

    assert fwd() == jfa.JFA_OK and app() == jfa.JFA_OK
    assert fwd(window=-5) == bad and fwd(window=3, causal=False) == bad and fwd(max_q_len=-1) == bad
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert fwd(scale=scale) == bad
    assert fwd(Q=c.Q[:, :3]) == bad                       # not a multiple of the key heads
    assert fwd(Q=c.Q.float()) == bad and fwd(Q=c.Q.cpu()) == bad
    assert fwd(Q=c.Q.transpose(0, 1)) == bad              # heads not dense
    assert fwd(Q=torch.empty(6, 4 * 64 + 1, dtype=BF, device="cuda")[:, 1:].view(6, 4, 64)) == bad  # misaligned
    assert fwd(q_offsets=c.q_off.long()) == bad and fwd(page_table=c.table[:1]) == bad
    assert fwd(kv_lens=c.kv_lens.cpu()) == bad
    assert fwd(workspace=ws[:-256]) == bad and fwd(workspace=ws[16:]) == bad
    assert fwd(bias=torch.zeros(4, 31, device="cuda", dtype=F32)) == bad
    assert fwd(O=torch.empty(6, 4, 64, dtype=torch.float16, device="cuda")) == uns
    many = torch.zeros(8194, dtype=torch.int32, device="cuda")  # more sequences than a call takes
    assert fwd(q_offsets=many, kv_lens=many[1:], page_table=many[1:, None].contiguous()) == bad
    wide = torch.zeros(6, 258, 64, dtype=BF, device="cuda")     # more than 128 heads on one key head
    assert status_of(jfa, jfa.jfa_cache_fwd, cache, wide, c.q_off, c.kv_lens, c.table) == uns
    assert app(Q=None) == jfa.JFA_OK and app(rot=None) == bad and app(Q=None, rot=None) == jfa.JFA_OK
    assert app(rot=torch.zeros(60, 24, device="cuda", dtype=F32)) == bad and app(rot=torch.zeros(60, 80, device="cuda", dtype=F32)) == bad
    assert app(rot_kind="other") == bad and app(V=c.V[:3]) == bad and app(Q_out=c.Q[:3]) == bad
    L = jfa.lib()
    # a dense bias is not read through a page table
    r = L.jfa_cache_fwd(cache.handle, 2, 6, 5, c.q_off.data_ptr(), c.kv_lens.data_ptr(), c.table.data_ptr(),
                        c.table.shape[1], c.Q.data_ptr(), 256, 4, 1, -1, jfa.JFA_BIAS_DENSE, ws.data_ptr(), 0.1,
                        c.Q.data_ptr(), jfa.JFA_BF16, None, ws.data_ptr(), ws.numel(), jfa._stream())
    assert r == uns
    # lse is optional
    O = torch.empty_like(c.Q)
    r = L.jfa_cache_fwd(cache.handle, 2, 6, 5, c.q_off.data_ptr(), c.kv_lens.data_ptr(), c.table.data_ptr(),
                        c.table.shape[1], c.Q.data_ptr(), 256, 4, 1, -1, 0, None, 0.125, O.data_ptr(), jfa.JFA_BF16,
                        None, ws.data_ptr(), ws.numel(), jfa._stream())
    assert r == jfa.JFA_OK
    torch.cuda.synchronize()
    assert torch.equal(O, jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, c.table, workspace=ws, max_q_len=5)[0])
    # handles: head dimension, page size, strides
    def make(shape, dtype=BF):
        return status_of(jfa, jfa.jfa_cache_create, torch.zeros(shape, dtype=dtype, device="cuda"),
                         torch.zeros(shape, dtype=dtype, device="cuda"))
    assert make((2, 16, 2, 32)) == uns and make((2, 16, 2, 96)) == uns and make((2, 16, 2, 128), F32) == uns
    assert make((2, 4, 2, 64)) == uns and make((2, 24, 2, 64)) == uns and make((2, 2048, 1, 64)) == uns
    assert make((2, 16, 2, 64), torch.float16) == uns
    odd = torch.zeros(2, 16, 2, 68, dtype=BF, device="cuda")[..., :64]
    assert status_of(jfa, jfa.jfa_cache_create, odd, odd) == bad
    flat = torch.zeros(64, dtype=BF, device="cuda").expand(2, 16, 2, 64)
    assert status_of(jfa, jfa.jfa_cache_create, flat, flat) == bad


def test_empty_calls(jfa):
    Kc = torch.zeros(2, 16, 2, 64, dtype=BF, device="cuda")
    cache = jfa.jfa_cache_create(Kc, Kc.clone())
    i32 = dict(dtype=torch.int32, device="cuda")
    Q, K = torch.zeros(0, 4, 64, dtype=BF, device="cuda"), torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    for B in (0, 3):
        off, kv, table = torch.zeros(B + 1, **i32), torch.zeros(B, **i32), torch.zeros(B, 1, **i32)
        jfa.jfa_cache_append(cache, K, K, off, kv, table, Q=Q, rot=make_table(4, 64))
        O, lse = jfa.jfa_cache_fwd(cache, Q, off, kv, table)
        assert O.shape == (0, 4, 64) and lse.shape == (0, 4)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK


@pytest.mark.parametrize("dtype,D", [(BF, 64), (F32, 64)])
@pytest.mark.parametrize("max_q_len", [None, 1])
def test_offsets_that_go_back_and_forth(jfa, dtype, D, max_q_len):
    # every second sequence claims all 512 rows over a million keys: 4096 x 16 row tiles x 8
    # heads x 8192 key tiles are more than 2^31.  Nothing is computed, and the call says so.
    B, T, H, kv = 8192, 512, 64, 1 << 20
    Kc = torch.zeros(1, 1024, 8, D, dtype=dtype, device="cuda")
    cache = jfa.jfa_cache_create(Kc, Kc.clone())
    i32 = dict(dtype=torch.int32, device="cuda")
    off = torch.zeros(B + 1, **i32)
    off[1::2] = T
    lens, table = torch.full((B,), kv, **i32), torch.zeros(B, kv // 1024, **i32)
    Q = torch.zeros(T, H, D, dtype=dtype, device="cuda")
    O = torch.full_like(Q, 7.0)
    ws = jfa.jfa_cache_workspace(cache, H)
    jfa.jfa_cache_fwd(cache, Q, off, lens, table, max_q_len=max_q_len, O=O, workspace=ws)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS
    assert torch.all(O == 7.0) and not ws[:jfa.JFA_CACHE_ZERO_BYTES].any()
    # the same workspace afterwards: zero keys and queries give the mean of zero values
    off = torch.cat([torch.zeros(1, **i32), torch.full((B,), T, **i32)])
    lens[0], lens[1:] = 700, 0
    jfa.jfa_cache_fwd(cache, Q, off, lens, table, max_q_len=max_q_len, O=O, workspace=ws)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK and not O.any()


def test_outputs_made_by_a_call_belong_to_its_stream(jfa):
    c = Case(*RAGGED, H=4, Hkv=2, D=64, page=16, seed=8)
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    want = c.run(jfa, cache)
    rot = make_table(2048, 64)
    K, V = torch.randn(2, c.T, 2, 64, device="cuda", dtype=F32).to(BF)
    full = torch.arange(c.table.numel(), dtype=torch.int32, device="cuda").view_as(c.table)
    scratch = [jfa.jfa_cache_create(*torch.zeros(2, full.numel(), 16, 2, 64, device="cuda", dtype=BF)) for _ in range(2)]
    lens = torch.maximum(c.kv_lens, c.q_off[1:] - c.q_off[:-1])
    want_q = jfa.jfa_cache_append(scratch[0], K, V, c.q_off, lens, full, Q=c.Q, rot=rot)
    ws = jfa.jfa_cache_workspace(cache, 4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)  # the current stream is busy for about 50 ms
    freed = [torch.empty_like(x) for x in (*want, c.Q)]
    for x in freed:
        x.fill_(3.0)                # writes still to come to memory that is given back now
    del freed, x
    O, lse = jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, c.table, workspace=ws, max_q_len=200, stream=s)
    Qo = jfa.jfa_cache_append(scratch[1], K, V, c.q_off, lens, full, Q=c.Q, rot=rot, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(O, want[0]) and torch.equal(lse, want[1]) and torch.equal(Qo, want_q)


def test_output_over_the_queries_is_refused(jfa):
    c = Case([1, 5], [20, 9], H=4, Hkv=2, D=64, page=16, unset=False)
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    assert status_of(jfa, jfa.jfa_cache_fwd, cache, c.Q, c.q_off, c.kv_lens, c.table, O=c.Q) == jfa.JFA_ERR_INVALID_ARG


# Query sets of at most 64 packed rows at head dimension 64, items of one row tile, whose key
# steps take turns as tile A and tile B: odd and even numbers of steps, a single one, an item cut
# between CTAs, more rows than keys.
SETS = ([17, 33, 64, 63, 20, 48, 32, 21, 60], [17, 200, 640, 129, 5000, 257, 0, 20000, 9])


@pytest.mark.parametrize("H,Hkv,div", [(3, 3, 1), (4, 2, 2), (5, 1, 5), (3, 1, 3)])
@pytest.mark.parametrize("causal,window,bias", [(False, None, False), (True, None, True), (True, 300, False), (False, None, True)])
@pytest.mark.parametrize("page", [8, 128])
def test_short_query_sets(jfa, H, Hkv, div, causal, window, bias, page):
    q = [max(1, n // div) for n in SETS[0]]
    c = Case(q, SETS[1], H=H, Hkv=Hkv, D=64, page=page, causal=causal, window=window, bias=bias, seed=H + page)
    c.check(*c.run(jfa, out_dtype=F32))


def test_short_and_long_query_sets_take_turns(jfa):
    q = [40, 300, 18, 129, 64, 65, 500, 33] * 40
    kv = [n + 100 * (i % 7) for i, n in enumerate(q)]
    c = Case(q, kv, H=2, Hkv=1, D=64, page=32, seed=4)
    c.check(*c.run(jfa))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_many_short_chunks(jfa, dtype, D):
    # hundreds of items of one to four key tiles, with some that see no key among them
    rs = np.random.RandomState(D)
    q = rs.randint(5, 60, 700)
    kv = np.where(rs.rand(700) < 0.1, 0, rs.randint(1, 450, 700))
    c = Case(q, kv, H=8, Hkv=2, D=D, page=16, dtype=dtype, seed=D)
    c.check(*c.run(jfa))
