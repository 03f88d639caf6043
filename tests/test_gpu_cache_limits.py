"""The 4-bit cache and attention over selected blocks on a GPU, at the ends of what their calls take:
sums next to fp32's largest number, positions past 2^30, lists out of order, scales that only
their product with the cache's factor brings into range, rows at the smallest of the cache's scales."""
import numpy as np
import pytest
import torch

from cache_cases import Case, np64
from quant_cases import BF, F32, QCase
from test_gpu_cache_blocks import SETS, attend, bounds_for, check, choose, expected_blocks, make, random_lists, reference, tokens
from test_gpu_cache_quantized import Batch, check_append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def jfa():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from jagged_sequence_attention_gb300 import _build
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    return m


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("pages,tokens", [(400, 420), (400, 3), (1200, 200)])
@pytest.mark.parametrize("D", [64, 128])
def test_selection_by_sums_past_bf16(jfa, pages, tokens, D):
    """Sums of grouped heads that are finite in fp32 but round to infinity in bf16: 2^127, 255/256 of it and
    2^118 add up to 2^128 - 2^118, and bf16's largest number is 2^128 - 2^120."""
    c = Case([tokens, 1], [16 * pages, 16 * pages - 3], H=12, Hkv=3, D=D, page=16, seed=pages + tokens)
    big = torch.tensor([2.0 ** 127, 255 / 256 * 2.0 ** 127, 2.0 ** 118, 0.0], device="cuda")
    Q = c.Q.float().unflatten(1, (3, 4))
    Q[::2, ..., 5] = big
    Q[1::4, ..., 7] = -big
    c.Q = Q.flatten(1, 2).to(BF)
    bounds = torch.nan_to_num(bounds_for(c, tokens, std=0.1))
    assert float(bounds.abs().max()) < 0.88  # so that no score leaves fp32's range
    flat = bounds.clone()
    flat[..., 5] = flat[:1, ..., 5]          # the largest sum tells no page from another
    for b in (bounds, flat, torch.zeros_like(bounds)):
        for n, m in ((4, None), (60, None), (60, 1)):
            assert np.array_equal(choose(jfa, c, b, n, max_q_len=m), expected_blocks(c, b, n, 1, 1))


# ------------------------------------------------------------------ positions past 2^30

class Histories:
    """Rows of histories that are longer than their pages: position j of sequence b by the page table."""

    def __init__(self, c, which):
        self.c, self.which, self.off = c, np64(which), np.concatenate([[0], np.cumsum(c.kv)])

    def __getitem__(self, at):
        i, h = at
        b = np.searchsorted(self.off, i, "right") - 1
        j = i - self.off[b]
        return self.which[self.c.host_table[b, j // self.c.page], j % self.c.page, h]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bias", [False, True])
def test_lists_of_a_history_past_2_30(jfa, bits, D, bias):
    """A list's end, and its blocks past the token, hold no key whatever the token's position."""
    page = 1024
    c = make(bits, [2, 1], [40 * page, 3000], H=4, Hkv=2, D=D, page=page, bias=bias, unset=False, seed=D + bits)
    for kv in (2 ** 30 + 5000, (2 ** 31 - 1 - c.T - 1024) // page * page):  # (the second: the longest there is in whole pages)
        width = -(-kv // page)
        table = np.full((2, width), -1, np.int32)
        table[0] = c.host_table[0, np.arange(width) % 40]
        table[1, :3] = c.host_table[1, :3]
        c.kv, at = np.array([kv, 3000]), c.host_table
        c.kv_lens = torch.tensor(c.kv, dtype=torch.int32, device="cuda")
        c.host_table, c.table = table, torch.from_numpy(table).cuda()
        c.gathered = lambda which: Histories(c, which)
        own = (kv - 1) // page
        lists = np.full((3, 2, 11), -1, np.int32)
        lists[0, 0, :3], lists[0, 1, :5] = [0, 7, own], [2, 3, own - 1, own, own + 1]
        lists[1, 0, :1], lists[1, 1] = own, own - 10 + np.arange(11)
        lists[2, 0, :2], lists[2, 1, :1] = [0, 2], 1
        ref = reference(c, lists)
        check(c, *attend(jfa, c, lists), ref)
        check(c, *attend(jfa, c, lists, out_dtype=F32), ref)
        c.host_table = at


def test_selection_from_a_history_past_2_30(jfa):
    page, kinds = 1024, 40
    c = Case([2], [kinds * page], H=2, Hkv=1, D=64, page=page, unset=False, seed=2)
    c.kv = np.array([2 ** 30 + 5000])
    width = -(-int(c.kv[0]) // page)
    c.host_table = np.ascontiguousarray(c.host_table[:, np.arange(width) % kinds])
    c.table, c.kv_lens = torch.from_numpy(c.host_table).cuda(), torch.tensor(c.kv, dtype=torch.int32, device="cuda")
    bounds = torch.nan_to_num(bounds_for(c, 2))
    for n in (3, 50, 40000):
        assert np.array_equal(choose(jfa, c, bounds, n, 1, 2), expected_blocks(c, bounds, n, 1, 2))


# ------------------------------------------------------------------ lists out of order

def in_order(lists):
    """The entries that ascend over all before them and follow no -1, as a list; whether others were left out (of each list:
    up to which entry there is none)."""
    kept, wrong = np.full_like(lists, -1), np.full(lists.shape[:-1], lists.shape[-1])
    for at in np.ndindex(lists.shape[:-1]):
        top, n = -1, 0
        for e, x in enumerate(lists[at]):
            if x < 0:
                top = np.iinfo(np.int64).max
            elif x > top:
                kept[at][n] = top = x
                n += 1
            else:
                wrong[at] = min(wrong[at], e)
    return kept, wrong


@pytest.mark.parametrize("bits", [16, 4])
def test_entries_out_of_order_are_left_out(jfa, bits):
    c = make(bits, [1], [300], H=4, Hkv=1, D=64, page=16, seed=6)
    for bad, same in (([0, -1, 2, 3], [0]), ([5, 3, 5], [5]), ([-1, 0, 1, 2], []), ([7, 1, 6, 2, 7, 8], [7, 8]), ([4, -1, -1, 9], [4])):
        assert [x for x in in_order(np.array([bad]))[0][0] if x >= 0] == same
        lists = np.array([[bad]], np.int32)
        kept = np.full_like(lists, -1)
        kept[0, 0, :len(same)] = same
        check(c, *attend(jfa, c, lists, status=jfa.JFA_ERR_DEVICE_BOUNDS), reference(c, kept))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 1024])
@pytest.mark.parametrize("D", [64, 128])
def test_long_lists_out_of_order(jfa, bits, page, D):
    """Lists that are cut between CTAs: what comes before a CTA's part decides about it too."""
    blocks = min(700, 120000 // page)
    c = make(bits, [1, 3, 1], [blocks * page, blocks * page // 2, blocks * page - 5], H=4, Hkv=2, D=D, page=page, seed=page + D)
    good = random_lists(c, blocks, 1, 0.9)
    rs = np.random.RandomState(page + D + bits)
    looked = np.minimum(blocks, tokens(c)[1] // page + 1)  # entries that a token looks at
    for change in range(5):
        lists = good.copy()
        if change == 0:
            lists[0, 0, 0] = blocks - 2          # nearly all lie before it
            lists[1, 1, 2] = -1
        elif change == 1:
            lists[0, 0, blocks // 3] = blocks - 1
            lists[4, 1, blocks // 2] = -5
        elif change == 2:
            lists[:, :, 1:] = rs.randint(0, blocks, lists[:, :, 1:].shape)
        elif change == 3:
            lists[:, 0] = blocks - 1 - np.arange(blocks)
        kept, wrong = in_order(lists)
        reported = bool((wrong < looked[:, None]).any())
        assert reported == (change < 4)
        O, lse = attend(jfa, c, lists, status=jfa.JFA_ERR_DEVICE_BOUNDS if reported else None)
        check(c, O, lse, reference(c, kept))


# ------------------------------------------------------------------ scales

@pytest.mark.parametrize("factor,scale", [(2.0 ** -60, 3e38), (2.0 ** -60, 2.5e38), (2.0 ** 60, 1e-45), (2.0 ** 60, 7e-45), (1e18, 3e-44), (1e-3, 3e38)])
def test_scales_that_the_factor_brings_into_range(jfa, factor, scale):
    """scale * k_factor lies in the documented range; scale * log2(e) alone would not be a number, or lose its bits."""
    factor, scale = float(np.float32(factor)), float(np.float32(scale))
    for lens in (([1, 2, 1], [70, 1000, 33]), ([40, 1, 300], [900, 65, 301])):
        c = QCase(*lens, H=8, Hkv=2, D=64, page=16, factors=(factor, 1.0), seed=3)
        c.Q = (c.Q.double() / (scale * factor * 8)).to(BF)  # scores of the usual size
        assert bool(torch.isfinite(c.Q).all())
        lists = np.tile(np.arange(70, dtype=np.int32), (c.T, 2, 1))
        dense, listed = c.run(jfa, scale=scale, out_dtype=F32), attend(jfa, c, lists, scale=scale, out_dtype=F32)
        c.Q = c.Q.double() * (scale * 8)  # (the reference's scale is 1 / 8)
        ref = c.reference()
        c.check(*dense, ref)
        c.check(*listed, ref)


def test_scales_out_of_range_are_refused(jfa):
    for factor, scale in ((2.0 ** -60, 1e-20), (2.0 ** 60, 1e20), (1.0, 1e-45), (1.0, 3e38)):
        c = QCase(*SETS, H=4, Hkv=2, D=64, page=16, factors=(factor, 1.0), seed=4)
        for call in (lambda: c.run(jfa, scale=scale), lambda: attend(jfa, c, np.zeros((c.T, 2, 3), np.int32), scale=scale)):
            with pytest.raises(jfa.JFAError) as e:
                call()
            assert e.value.status == jfa.JFA_ERR_INVALID_ARG


# ------------------------------------------------------------------ the smallest scale

@pytest.mark.parametrize("factors", [(1.0, 1.0), (0.3, 1.7), (2.0 ** -20, 0.7)])
@pytest.mark.parametrize("R", [0, 32, 128])
def test_append_at_the_smallest_scale(jfa, factors, R):
    """Groups whose largest magnitude is 0.4 to 1.6 times 6 steps of the smallest scale, 2^-9: it rounds to that scale, to 0
    or to the next one, and quotients reach 9."""
    factors = tuple(float(np.float32(f)) for f in factors)
    b = Batch([300, 1], [300, 7], D=128, R=R, factors=factors, seed=R)
    g = torch.Generator(device="cuda").manual_seed(R)
    rows = []
    for f in factors:
        x = torch.rand(b.c.T, 2, 8, 16, generator=g, device="cuda") * 2 - 1
        x[..., 3] = 1.0
        size = torch.rand(b.c.T, 2, 8, 1, generator=g, device="cuda") * 1.2 + 0.4
        size[::2] = size[::2].clamp(1.3, 1.5)
        rows.append((x * size * (6 * f * 2.0 ** -9)).flatten(-2).to(BF))
    b.K, b.V = rows
    if R:
        b.rot[5::7, :R // 2], b.rot[5::7, R // 2:] = 1.0, 0.0  # (as they are)
    check_append(jfa, b)
    assert bool((b.vs == 1).any() and (b.vs == 0).any() and (b.vs == 2).any())
