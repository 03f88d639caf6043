"""The 4-bit cache and attention over selected blocks on a GPU, at the ends of what their calls take:
sums next to fp32's largest number."""
import numpy as np
import pytest
import torch

from cache_cases import Case
from quant_cases import BF
from test_gpu_cache_blocks import bounds_for, choose, expected_blocks, tokens

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
