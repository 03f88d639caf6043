"""Attention over selected blocks of a paged cache on a GPU: the bounds and the selection against
64-bit torch, which they have to equal, and the attention against a dense softmax in 64 bits."""
import numpy as np
import pytest
import torch

from cache_cases import LSE_TOL, SLACK, Case, np64
from quant_cases import BF, F32, F64, QCase

pytestmark = pytest.mark.gpu

SINGLE = ([1] * 9, [1, 2, 63, 64, 65, 127, 129, 700, 2049])
SETS = ([5, 3, 0, 1, 30, 17], [5, 64, 31, 900, 1300, 177])
EMPTY_ROWS = ([4, 20, 1, 2], [2, 0, 0, 150])  # more rows than keys; no key at all


@pytest.fixture(scope="module")
def jfa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from jagged_sequence_attention_gb300 import _build
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    return m


def make(bits, *a, **kw):
    return QCase(*a, **kw) if bits == 4 else Case(*a, **kw)


def cache_of(jfa, c):
    return c.cache(jfa) if isinstance(c, QCase) else jfa.jfa_cache_create(c.Kc, c.Vc)


def tokens(c):
    """(sequence, position) of every new token."""
    b = np.repeat(np.arange(c.q.size), c.q)
    return b, np.arange(c.T) - np.repeat(np.cumsum(c.q) - c.q, c.q) + (c.kv - c.q)[b]


# ------------------------------------------------------------------ attention over listed blocks

def random_lists(c, n, seed, density=0.6, own=True):
    """Ascending blocks, then -1; some empty, some with blocks after the token's own."""
    rs = np.random.RandomState(seed)
    b, pos = tokens(c)
    lists = np.full((c.T + 3, c.Hkv, n), -1, np.int32)
    for t in range(c.T):
        nb = -(-int(c.kv[b[t]]) // c.page)
        for h in range(c.Hkv):
            pick = np.flatnonzero(rs.rand(nb) < density)
            if own and pos[t] >= 0 and rs.rand() < 0.8:
                pick = np.union1d(pick, [pos[t] // c.page])
            pick = np.sort(rs.permutation(pick)[:n])
            lists[t, h, :pick.size] = pick
    return lists[:c.T]


def reference(c, lists):
    """(O, lse, sum_j p_j |v_j|) in 64 bits."""
    b, pos = tokens(c)
    g = c.H // c.Hkv
    off = np.concatenate([[0], np.cumsum(c.kv)])
    K, V, Q = c.gathered(c.Kc), c.gathered(c.Vc), np64(c.Q)
    O, A = np.zeros((c.T, c.H, c.D)), np.zeros((c.T, c.H, c.D))
    lse = np.full((c.T, c.H), -np.inf)
    for t in range(c.T):
        for h in range(c.Hkv):
            pages = lists[t, h][lists[t, h] >= 0]
            j = (pages[:, None] * c.page + np.arange(c.page)).ravel()
            j = j[j <= pos[t]]
            if j.size == 0:
                continue
            k, v = K[off[b[t]] + j, h], V[off[b[t]] + j, h]
            for i in range(h * g, (h + 1) * g):
                x = k @ Q[t, i] / np.sqrt(c.D)
                if c.bias is not None:
                    d = (pos[t] - j).astype(np.int64) + 1
                    bucket = np.minimum(31, [int(e * e).bit_length() - 1 for e in d])
                    x = x + np64(c.bias)[i][bucket]
                m = x.max()
                p = np.exp(x - m)
                lse[t, i] = m + np.log(p.sum())
                O[t, i], A[t, i] = p @ v / p.sum(), p @ np.abs(v) / p.sum()
    return O, lse, A


def check(c, O, lse, ref):
    ro, rl, A = ref
    o, l = np64(O)[:c.T], np64(lse)[:c.T]
    # weights rounded to bf16 (16-bit caches) or fp16
    tol = SLACK * A + (2.0 ** -11 if isinstance(c, QCase) else 2.0 ** -8) * A + (c.tiny() if isinstance(c, QCase) else 0.0) + 1e-30
    if O.dtype == BF:
        tol = tol + 2.0 ** -8 * np.abs(ro)
    assert np.all(np.isfinite(o)) and (np.abs(o - ro) - tol).max(initial=-1.0) <= 0.0
    fin = np.isfinite(rl)
    assert np.array_equal(fin, np.isfinite(l)) and np.all(l[~fin] == -np.inf)
    assert np.abs(l[fin] - rl[fin]).max(initial=0.0) <= LSE_TOL


def attend(jfa, c, lists, cache=None, status=None, **kw):
    cache = cache or cache_of(jfa, c)
    t = torch.from_numpy(np.ascontiguousarray(lists)).cuda()
    O, lse = jfa.jfa_cache_fwd_blocks(cache, kw.pop("Q", c.Q), c.q_off, c.kv_lens, c.table, t, bias=c.bias, **kw)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == (jfa.JFA_OK if status is None else status)
    return O, lse


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [SINGLE, SETS, EMPTY_ROWS], ids=["single", "sets", "empty"])
def test_pages_and_lengths(jfa, bits, D, page, lens):
    for n, density in ((1, 1.0), (7, 0.4), (300, 0.7)):
        c = make(bits, *lens, H=4, Hkv=2, D=D, page=page, unset=True, seed=page + n)
        lists = random_lists(c, n, page + n, density)
        check(c, *attend(jfa, c, lists), reference(c, lists))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (5, 1), (16, 2), (9, 1), (32, 2)])
@pytest.mark.parametrize("bias", [False, True])
def test_head_groups_and_bias(jfa, bits, H, Hkv, bias):
    for D in (64, 128):
        c = make(bits, *SETS, H=H, Hkv=Hkv, D=D, page=16, bias=bias, seed=H)
        lists = random_lists(c, 40, H)
        ref = reference(c, lists)
        check(c, *attend(jfa, c, lists), ref)
        check(c, *attend(jfa, c, lists, out_dtype=F32), ref)


@pytest.mark.parametrize("bits", [16, 4])
def test_all_blocks_are_dense_attention(jfa, bits):
    c = make(bits, *SETS, H=8, Hkv=2, D=128, page=32, bias=True, seed=4)
    lists = np.tile(np.arange(60, dtype=np.int32), (c.T, 2, 1))  # past every history's end
    O, lse = attend(jfa, c, lists)
    c.check(O, lse)


@pytest.mark.parametrize("bits", [16, 4])
def test_long_lists_are_split(jfa, bits):
    c = make(bits, [1, 2], [40011, 9000], H=4, Hkv=1, D=128, page=16, seed=5)
    lists = random_lists(c, 2600, 5, 0.9)
    ref = reference(c, lists)
    cache = cache_of(jfa, c)
    ws = jfa.jfa_cache_workspace(cache, 4)
    O, lse = attend(jfa, c, lists, cache, workspace=ws)
    check(c, O, lse, ref)
    for _ in range(3):
        ws[jfa.JFA_CACHE_ZERO_BYTES:].random_(0, 255)
        O2, lse2 = attend(jfa, c, lists, cache, workspace=ws)
        assert torch.equal(O, O2) and torch.equal(lse, lse2) and not bool(ws[:jfa.JFA_CACHE_ZERO_BYTES].any())


@pytest.mark.parametrize("bits", [16, 4])
def test_lists_out_of_order_are_reported(jfa, bits):
    c = make(bits, [1, 1, 1], [300, 300, 300], H=4, Hkv=1, D=64, page=16, seed=6)
    good = np.array([[[0, 3, 7, 18]], [[1, 2, -1, -1]], [[-1, -1, -1, -1]]], np.int32)
    ref = reference(c, good)
    check(c, *attend(jfa, c, good), ref)
    for bad, same in (([0, 3, 3, 18], [0, 3, 18, -1]), ([5, 3, 7, 18], [5, 7, 18, -1]), ([0, -1, 3, -1], [0, -1, -1, -1]),
                      ([3, 0, 0, 0], [3, -1, -1, -1])):
        lists, kept = good.copy(), good.copy()
        lists[0, 0], kept[0, 0] = bad, same
        check(c, *attend(jfa, c, lists, status=jfa.JFA_ERR_DEVICE_BOUNDS), reference(c, kept))
    lists = good.copy()
    lists[0, 0], lists[1, 0] = [0, 3, 7, 2 ** 31 - 1], [-2 ** 31, -7, -1, -1]  # a block that nobody has; any negative number
    kept = good.copy()
    kept[0, 0], kept[1, 0] = [0, 3, 7, -1], -1
    check(c, *attend(jfa, c, lists), reference(c, kept))
    # a bad page of one sequence leaves the others right
    table = c.table.clone()
    c.table = table.clone()
    c.table[0, 3] = c.n_pages
    O, lse = attend(jfa, c, good, status=jfa.JFA_ERR_DEVICE_BOUNDS)
    O[0], lse[0] = torch.from_numpy(ref[0][0]).to(O), torch.from_numpy(ref[1][0]).to(lse)
    check(c, O, lse, ref)
    c.table[0, 3] = table[0, 3]
    c.table[0, 5] = -1  # (not listed: not read)
    check(c, *attend(jfa, c, good), ref)


def test_rows_behind_and_strides(jfa):
    for bits in (16, 4):
        c = make(bits, *SETS, H=4, Hkv=2, D=64, page=16, pad_rows=9, seed=7)
        lists = random_lists(c, 12, 7)
        ref = reference(c, lists)
        padded = np.concatenate([lists, np.full((9, 2, 12), 10 ** 9, np.int32)])
        O = torch.full_like(c.Q, 7.0)
        lse = torch.full((c.T + 9, 4), 9.0, device="cuda", dtype=F32)
        attend(jfa, c, padded, O=O, lse=lse)
        assert bool((O[c.T:] == 7.0).all()) and bool((lse[c.T:] == 9.0).all())
        check(c, O, lse, ref)
        wide = torch.full((c.T + 9, 8, 64), float("nan"), dtype=BF, device="cuda")
        wide[:, :4] = c.Q
        check(c, *attend(jfa, c, padded, Q=wide[:, :4]), ref)


# ------------------------------------------------------------------ bounds

def expected_bounds(c, bounds):
    b, pos = tokens(c)
    want = bounds.double().cpu().numpy().copy()
    k = np64(c.Kc) / (c.factors[0] if isinstance(c, QCase) else 1.0)
    for page_b, page_i in {(b[t], pos[t] // c.page) for t in range(c.T) if pos[t] >= 0}:
        n = min(c.page, int(c.kv[page_b]) - page_i * c.page)
        at = c.host_table[page_b, page_i]
        want[at, :, 0], want[at, :, 1] = k[at, :n].min(0), k[at, :n].max(0)
    return want


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_bounds(jfa, bits, page, D):
    for lens in (SINGLE, SETS, ([130, 1, 700], [131, 900, 1300])):
        kw = dict(factors=(0.25, 1.0)) if bits == 4 and page == 16 else {}
        c = make(bits, *lens, H=3, Hkv=3, D=D, page=page, layout="tokens" if page == 64 else "heads", seed=page, **kw)
        cache = cache_of(jfa, c)
        bounds = torch.randn(c.n_pages, c.Hkv, 2, D, device="cuda", dtype=F32).to(BF)
        want = expected_bounds(c, bounds)
        jfa.jfa_cache_summarize(cache, bounds, c.T, c.q_off, c.kv_lens, c.table)
        torch.cuda.synchronize()
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
        assert np.array_equal(np64(bounds), want)


# ------------------------------------------------------------------ selection

def expected_blocks(c, bounds, n, first, last):
    """By 64-bit scores; equal ones by the lower index."""
    b, pos = tokens(c)
    Q, bd = c.Q.double(), bounds.double()
    out = np.full((c.T, c.Hkv, n), -1, np.int32)
    for t in range(c.T):
        own = int(pos[t]) // c.page if pos[t] >= 0 else -1
        if own + 1 <= n:
            out[t, :, :own + 1] = np.arange(own + 1)
            continue
        pages = torch.from_numpy(c.host_table[b[t], :own + 1]).long().cuda()
        q = Q[t].reshape(c.Hkv, -1, c.D)
        score = (q.clamp(min=0).sum(1) * bd[pages, :, 1]).sum(-1) + (q.clamp(max=0).sum(1) * bd[pages, :, 0]).sum(-1)
        score = score.T.cpu().numpy()                              # [Hkv, blocks]
        for h in range(c.Hkv):
            middle = np.arange(first, own + 1 - last)
            best = middle[np.argsort(-score[h, middle], kind="stable")[:n - first - last]]
            out[t, h] = np.sort(np.concatenate([np.arange(first), best, np.arange(own + 1 - last, own + 1)]))
    return out


def bounds_for(c, seed, std=1.0):
    """Bounds of random pages, ordered; those of unused pages are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(c.n_pages, c.Hkv, 2, c.D, generator=g, device="cuda", dtype=F32) * std).to(BF).sort(2)[0]
    x[torch.from_numpy(np.setdiff1d(np.arange(c.n_pages), c.host_table)).cuda()] = float("nan")
    return x


def choose(jfa, c, bounds, n, first=1, last=1, cache=None, **kw):
    cache = cache or cache_of(jfa, c)
    out = jfa.jfa_cache_select(cache, bounds, kw.pop("Q", c.Q), c.q_off, c.kv_lens, c.table, n, first, last, **kw)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
    return out.cpu().numpy()


@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 64), (8, 2, 128), (5, 1, 64), (48, 3, 128), (100, 1, 64)])
@pytest.mark.parametrize("lens", [SINGLE, SETS, EMPTY_ROWS, ([64, 200], [3000, 4100])], ids=["single", "sets", "empty", "chunks"])
def test_selection(jfa, H, Hkv, D, lens):
    c = Case(*lens, H=H, Hkv=Hkv, D=D, page=16, seed=H)
    bounds = bounds_for(c, H)
    for n, first, last in ((1, 0, 1), (2, 1, 1), (5, 0, 1), (16, 1, 4), (33, 2, 31), (128, 1, 1), (300, 0, 2)):
        got = choose(jfa, c, bounds, n, first, last, max_q_len=int(c.q.max()))
        assert np.array_equal(got, expected_blocks(c, bounds, n, first, last))


def test_selection_from_long_histories(jfa):
    # more blocks than the selection keeps in shared memory
    c = Case([2, 1], [16 * 9000, 16 * 20000 + 5], H=4, Hkv=1, D=64, page=16, seed=1)
    bounds = bounds_for(c, 1)
    for n in (3, 64, 1000, 8700):
        assert np.array_equal(choose(jfa, c, bounds, n), expected_blocks(c, bounds, n, 1, 1))


@pytest.mark.parametrize("kinds", [1, 2, 7])
def test_equal_scores_go_by_index(jfa, kinds):
    """Pages of few kinds, so that most scores are equal: more candidates than are kept, and few."""
    for lens in (([1, 3], [16 * 700, 16 * 300 + 2]), ([2], [16 * 9000])):
        c = Case(*lens, H=2, Hkv=2, D=64, page=16, seed=kinds)
        base = bounds_for(c, kinds)
        base = torch.nan_to_num(base)
        bounds = base[torch.randint(0, kinds, (c.n_pages,), device="cuda")].contiguous()
        for n in (5, 100, 280):
            assert np.array_equal(choose(jfa, c, bounds, n), expected_blocks(c, bounds, n, 1, 1))
    c = Case([3], [16 * 500], H=2, Hkv=2, D=64, page=16, seed=kinds)
    zero = torch.zeros(c.n_pages, 2, 2, 64, device="cuda", dtype=BF)
    assert np.array_equal(choose(jfa, c, zero, 40), expected_blocks(c, zero, 40, 1, 1))


@pytest.mark.parametrize("kinds", [1, 3])
def test_equal_scores_of_many_tokens(jfa, kinds):
    # (items of a warp each, more candidates than it keeps, and few)
    c = Case([90, 2], [16 * 400, 16 * 350], H=4, Hkv=2, D=128, page=16, seed=kinds)
    base = torch.nan_to_num(bounds_for(c, kinds))
    bounds = base[torch.randint(0, kinds, (c.n_pages,), device="cuda")].contiguous()
    for n in (5, 60, 200, 340):
        for m in (None, 1):
            assert np.array_equal(choose(jfa, c, bounds, n, max_q_len=m), expected_blocks(c, bounds, n, 1, 1))
    some = torch.rand(c.n_pages, device="cuda") < 0.1
    bounds[some] = base[some]
    assert np.array_equal(choose(jfa, c, bounds, 60), expected_blocks(c, bounds, 60, 1, 1))


@pytest.mark.parametrize("pages,tokens", [(400, 420), (400, 60), (900, 420), (900, 5), (1200, 20)])
def test_numbers_of_items_and_pages(jfa, pages, tokens):
    # (a warp, four or 32 an item, by both numbers)
    c = Case([tokens, 1], [16 * pages, 16 * pages - 3], H=3, Hkv=3, D=64, page=16, seed=pages + tokens)
    random = torch.nan_to_num(bounds_for(c, tokens))
    few = random[torch.randint(0, 3, (c.n_pages,), device="cuda")].contiguous()
    for bounds in (random, few):
        for n in (4, 300):
            assert np.array_equal(choose(jfa, c, bounds, n), expected_blocks(c, bounds, n, 1, 1))


@pytest.mark.parametrize("pages,tokens", [(68, 1), (400, 420), (400, 60), (1200, 2)])
def test_scores_past_fp32(jfa, pages, tokens):
    """Finite bounds and queries whose products are not finite in fp32, or only just."""
    c = Case([tokens, 1], [16 * pages, 16 * pages - 3], H=12, Hkv=3, D=128, page=16, seed=pages + tokens)
    Q = c.Q.float()
    for big in (1e14, 1e16, 1e18):
        bounds = torch.nan_to_num(bounds_for(c, tokens, std=1e20))
        c.Q = (Q * big).to(BF)
        for n, m in ((4, None), (60, 1)):
            assert np.array_equal(choose(jfa, c, bounds, n, max_q_len=m), expected_blocks(c, bounds, n, 1, 1))


def test_nearly_equal_scores(jfa):
    """Scores that fp32 sums cannot tell apart: large parts that cancel, and differences in the
    last bits."""
    c = Case([1, 2], [16 * 900, 16 * 120], H=2, Hkv=1, D=128, page=16, seed=3)
    bounds = torch.nan_to_num(bounds_for(c, 3))
    bounds[..., :32] = (bounds[..., :32].float() * 1e-6).to(BF)
    bounds[..., 32:] = bounds[:1, ..., 32:]        # the same on every page
    bounds[..., 64:96] *= 1000.0
    assert np.array_equal(choose(jfa, c, bounds, 50), expected_blocks(c, bounds, 50, 1, 1))
    bounds[..., 40:] = bounds_for(c, 4)[..., 40:].nan_to_num()
    assert np.array_equal(choose(jfa, c, bounds, 50), expected_blocks(c, bounds, 50, 1, 1))


def test_selection_leaves_what_is_not_its(jfa):
    c = Case(*SETS, H=4, Hkv=2, D=64, page=16, pad_rows=5, seed=8)
    bounds = bounds_for(c, 8)
    blocks = torch.full((c.T + 5, 2, 9), 77, dtype=torch.int32, device="cuda")
    got = choose(jfa, c, bounds, 9, blocks=blocks)
    assert (got[c.T:] == 77).all()
    want = expected_blocks(c, bounds, 9, 1, 1)
    assert np.array_equal(got[:c.T], want)
    wide = torch.full((c.T + 5, 8, 64), float("nan"), dtype=BF, device="cuda")
    wide[:, 2:6] = c.Q
    assert np.array_equal(choose(jfa, c, bounds, 9, Q=wide[:, 2:6])[:c.T], want)
    cache = cache_of(jfa, c)
    lens = c.kv_lens.clone()
    lens[1] = -1
    blocks.fill_(77)
    jfa.jfa_cache_select(cache, bounds, c.Q, c.q_off, lens, c.table, 9, blocks=blocks)
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS
    got = blocks.cpu().numpy()
    assert (got[5:8] == 77).all() and np.array_equal(got[:5], want[:5]) and np.array_equal(got[8:c.T], want[8:])


# ------------------------------------------------------------------ the calls of a step together

def step(jfa, cache, c, K, V, bounds, n, ws, sel_ws, lists, O, lse, **kw):
    jfa.jfa_cache_append(cache, K, V, c.q_off, c.kv_lens, c.table, **kw)
    jfa.jfa_cache_summarize(cache, bounds, c.T, c.q_off, c.kv_lens, c.table, **kw)
    jfa.jfa_cache_select(cache, bounds, c.Q, c.q_off, c.kv_lens, c.table, n, 1, 2, blocks=lists, workspace=sel_ws, **kw)
    return jfa.jfa_cache_fwd_blocks(cache, c.Q, c.q_off, c.kv_lens, c.table, lists, O=O, lse=lse, workspace=ws, **kw)


@pytest.mark.parametrize("bits", [16, 4])
def test_served_steps(jfa, bits):
    """Prompts, then tokens: the selection is that of the bounds of what was appended, and the
    attention that over it; then the step captured and replayed on new contents."""
    D, H, Hkv, page, n = 128, 8, 2, 16, 6
    full = make(bits, [1, 1, 1], [420, 130, 17], H=H, Hkv=Hkv, D=D, page=page, unset=False, seed=9)
    cache = cache_of(jfa, full)
    bounds = torch.full((full.n_pages, Hkv, 2, D), float("nan"), device="cuda", dtype=BF)
    for q, kv in (([400, 128, 3], [400, 128, 3]), ([19, 1, 1], [419, 129, 4]), ([1, 1, 13], [420, 130, 17])):
        c = make(bits, q, kv, H=H, Hkv=Hkv, D=D, page=page, unset=False, seed=10)
        c.table, c.host_table, c.n_pages = full.table, full.host_table, full.n_pages
        K, V = (torch.randn(c.T, Hkv, D, device="cuda", dtype=F32).to(BF) for _ in range(2))
        ws, sel = jfa.jfa_cache_workspace(cache, H), jfa.jfa_cache_select_workspace(cache, c.T, c.table.shape[1])
        lists = torch.empty(c.T, Hkv, n, dtype=torch.int32, device="cuda")
        O, lse = torch.empty_like(c.Q), torch.empty(c.T, H, device="cuda", dtype=F32)
        step(jfa, cache, c, K, V, bounds, n, ws, sel, lists, O, lse)
        torch.cuda.synchronize()
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK
        off = torch.nn.functional.pad(c.kv_lens.cumsum(0), (1, 0)).int()
        rows_k, rows_v = jfa.jfa_cache_read(cache, int(c.kv.sum()), off, c.kv_lens, c.table)
        c.gathered = lambda which, k=np64(rows_k), v=np64(rows_v), c=c: k if which is c.Kc else v
        got = lists.cpu().numpy()
        assert np.array_equal(got, expected_blocks(c, bounds, n, 1, 2))
        check(c, O, lse, reference(c, got))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = (jfa, cache, c, K, V, bounds, n, ws, sel, lists, O, lse)
    with torch.cuda.stream(s):
        step(*args)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*args)
    for _ in range(2):
        for x in (K, V, c.Q):
            x.copy_(torch.randn(x.shape, device="cuda", dtype=F32))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (bounds, lists, O, lse)]
        step(*args, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(torch.nan_to_num(x), torch.nan_to_num(y)) for x, y in zip(got, (bounds, lists, O, lse)))
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK


@pytest.mark.parametrize("bits", [16, 4])
def test_steps_at_once_on_two_streams(jfa, bits):
    """Selections and attention over them, each stream with workspaces of its own, and then two
    graphs that share one, replayed in turn."""
    cases = [make(bits, *lens, H=8, Hkv=2, D=128, page=16, seed=21) for lens in (SETS, ([1, 40, 2], [5000, 700, 1900]))]
    runs = []
    for c in cases:
        cache, bounds = cache_of(jfa, c), torch.nan_to_num(bounds_for(c, 21))
        lists, O, lse = torch.empty(c.T, 2, 7, dtype=torch.int32, device="cuda"), torch.empty_like(c.Q), torch.empty(c.T, 8, device="cuda", dtype=F32)
        ws, sel = jfa.jfa_cache_workspace(cache, 8), jfa.jfa_cache_select_workspace(cache, 200, 1024)

        def run(c=c, cache=cache, bounds=bounds, lists=lists, O=O, lse=lse, ws=ws, sel=sel, **kw):
            jfa.jfa_cache_select(cache, bounds, c.Q, c.q_off, c.kv_lens, c.table, 7, blocks=lists, workspace=sel, **kw)
            jfa.jfa_cache_fwd_blocks(cache, c.Q, c.q_off, c.kv_lens, c.table, lists, O=O, lse=lse, workspace=ws, **kw)
            return lists, O, lse

        assert np.array_equal(run()[0].cpu().numpy(), expected_blocks(c, bounds, 7, 1, 1))
        runs.append((run, [x.clone() for x in run()], ws, sel))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, (run, *_) in zip(streams, runs):
            run(stream=s)
    torch.cuda.synchronize()
    for run, want, *_ in runs:
        assert all(torch.equal(x, y) for x, y in zip(run(), want))
    ws, sel = runs[0][2:]
    graphs = []
    for run, *_ in runs:
        run(ws=ws, sel=sel)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out = run(ws=ws, sel=sel)
        for x in out:
            x.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for run, want, *_ in runs:
        got = [x.clone() for x in run.__defaults__[3:6]]
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_the_query_bound_changes_no_selection(jfa):
    for lens in (SINGLE, SETS, ([64, 200, 1], [3000, 4100, 2000])):
        c = Case(*lens, H=8, Hkv=2, D=128, page=16, seed=22)
        bounds = bounds_for(c, 22)
        want = expected_blocks(c, bounds, 12, 1, 1)
        for n in (None, 1, 4, 5, 10 ** 6):
            assert np.array_equal(choose(jfa, c, bounds, 12, max_q_len=n), want)


def test_no_tokens_and_no_pages(jfa):
    c = Case([0, 0], [40, 0], H=4, Hkv=2, D=64, page=16, seed=23)
    cache, bounds = cache_of(jfa, c), torch.zeros(c.n_pages, 2, 2, 64, dtype=BF, device="cuda")
    a = (c.q_off, c.kv_lens, c.table)
    jfa.jfa_cache_summarize(cache, bounds, 0, *a)
    lists = jfa.jfa_cache_select(cache, bounds, c.Q[:0], *a, 3)
    O, lse = jfa.jfa_cache_fwd_blocks(cache, c.Q[:0], *a, lists)
    assert lists.shape == (0, 2, 3) and O.shape == (0, 4, 64) and lse.shape == (0, 4)
    # rows with no position: no block is theirs
    c = Case([3, 2], [1, 0], H=4, Hkv=2, D=64, page=16, seed=23)
    got = choose(jfa, c, torch.zeros(c.n_pages, 2, 2, 64, dtype=BF, device="cuda"), 2)
    assert np.array_equal(got, np.repeat([[[-1, -1]], [[-1, -1]], [[0, -1]], [[-1, -1]], [[-1, -1]]], 2, axis=1))
    torch.cuda.synchronize()
    assert jfa.jfa_cache_device_status(cache) == jfa.JFA_OK


def test_refusals(jfa):
    def status(fn, *a, **k):
        try:
            fn(*a, **k)
        except jfa.JFAError as e:
            return e.status
        return jfa.JFA_OK

    bad, uns = jfa.JFA_ERR_INVALID_ARG, jfa.JFA_ERR_UNSUPPORTED
    c = Case(*SETS, H=4, Hkv=2, D=64, page=16, seed=11)
    cache, bounds = cache_of(jfa, c), bounds_for(c, 11)
    a = (c.q_off, c.kv_lens, c.table)
    sel = lambda n=9, first=1, last=1, b=bounds, Q=c.Q, **kw: status(jfa.jfa_cache_select, cache, b, Q, *a, n, first, last, **kw)  # noqa: E731
    assert sel() == jfa.JFA_OK
    for n, first, last in ((0, 0, 1), (-3, 0, 1), (9, -1, 1), (9, 1, 0), (9, 5, 5), (2 ** 27, 1, 1)):
        assert sel(n, first, last, blocks=torch.empty(c.T, 2, max(n, 0) % 1000, dtype=torch.int32, device="cuda")) == bad
    assert sel(b=bounds.float()) == bad and sel(b=bounds[1:]) == bad and sel(b=bounds.transpose(2, 3)) == bad
    assert sel(Q=c.Q.float()) == bad and sel(max_q_len=-1) == bad
    assert sel(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")) == bad
    assert sel(blocks=torch.empty(c.T, 2, 8, dtype=torch.int32, device="cuda")) == bad
    assert sel(blocks=torch.empty(c.T, 2, 9, dtype=torch.int64, device="cuda")) == bad
    lists = torch.zeros(c.T, 2, 3, dtype=torch.int32, device="cuda")
    fwd = lambda x=lists, Q=c.Q, **kw: status(jfa.jfa_cache_fwd_blocks, cache, Q, *a, x, **kw)  # noqa: E731
    assert status(jfa.jfa_cache_fwd_blocks, cache, c.Q, *a, torch.full_like(lists, -1)) == jfa.JFA_OK
    for kw in (dict(x=lists.long()), dict(x=lists[1:]), dict(x=lists[:, :1]), dict(x=lists[..., :0]), dict(Q=c.Q.float()), dict(O=c.Q),
               dict(scale=0.0), dict(scale=float("nan")), dict(bias=torch.zeros(4, 31, device="cuda")),
               dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        assert fwd(**kw) == bad, kw
    assert fwd(O=torch.empty_like(c.Q, dtype=torch.float16)) == uns
    summ = lambda b, T=c.T: status(jfa.jfa_cache_summarize, cache, b, T, *a)  # noqa: E731
    assert summ(bounds) == jfa.JFA_OK and summ(bounds[..., :32]) == bad and summ(bounds, -1) == bad
    many = torch.zeros(c.T, 34, 64, dtype=BF, device="cuda")
    assert fwd(Q=many) == uns                              # 17 grouped heads
    for other in (Case(*SETS, H=4, Hkv=2, D=64, page=8, seed=11), Case(*SETS, H=4, Hkv=2, D=64, page=16, dtype=F32, seed=11)):
        ch, b = cache_of(jfa, other), torch.zeros(other.n_pages, 2, 2, 64, dtype=BF, device="cuda")
        o = (other.q_off, other.kv_lens, other.table)
        assert status(jfa.jfa_cache_summarize, ch, b, other.T, *o) == uns
        assert status(jfa.jfa_cache_select, ch, b, other.Q, *o, 3) == uns
        assert status(jfa.jfa_cache_fwd_blocks, ch, other.Q, *o, lists) == uns
