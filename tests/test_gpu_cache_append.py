"""Appending to a paged cache on a GPU: what a bad sequence must not touch."""
import pytest
import torch

from cache_cases import Case

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


@pytest.mark.parametrize("dtype,D", [(BF, 64), (F32, 32)])
@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("n", [0, 1, 6])
def test_fewer_positions_than_new_tokens(jfa, dtype, D, rotate, n):
    """Sequence 1 claims n positions for 7 new tokens: none of its tokens is appended, over the
    positions it may hold, and none of its queries is written; the others are."""
    c = Case([2, 7, 1], [40, 30, 9], H=4, Hkv=2, D=D, page=8, dtype=dtype, unset=False, seed=n)
    K, V = torch.randn(2, c.T, 2, D, device="cuda", dtype=F32).to(dtype)
    rot = torch.randn(64, 16, device="cuda", dtype=F32) if rotate else None
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)

    def append(lens):
        out = torch.full_like(c.Q, 5.0) if rotate else None
        jfa.jfa_cache_append(cache, K, V, c.q_off, lens, c.table, Q=c.Q if rotate else None, Q_out=out, rot=rot)
        torch.cuda.synchronize()
        return out, jfa.jfa_cache_device_status(cache)

    k0, v0 = c.Kc.clone(), c.Vc.clone()
    bad = c.kv_lens.clone()
    bad[1] = n
    out, st = append(bad)
    assert st == jfa.JFA_ERR_DEVICE_BOUNDS
    mine = torch.unique(c.table[1][c.table[1] >= 0].long())
    assert torch.equal(c.Kc[mine], k0[mine]) and torch.equal(c.Vc[mine], v0[mine])
    if rotate:
        assert bool((out[2:9] == 5.0).all())
    k1, v1 = c.Kc.clone(), c.Vc.clone()
    assert not torch.equal(k1, k0) and not torch.equal(v1, v0)
    # the other sequences' tokens are as in a call without a bad one
    good = c.kv_lens.clone()
    good[1] = 7                       # a fresh prompt: as many positions as tokens
    out2, st = append(good)
    assert st == jfa.JFA_OK
    rest = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    rest[mine] = False
    assert torch.equal(c.Kc[rest], k1[rest]) and torch.equal(c.Vc[rest], v1[rest])
    assert not torch.equal(c.Kc[mine], k0[mine])
    if rotate:
        assert torch.equal(out2[:2], out[:2]) and torch.equal(out2[9:], out[9:]) and bool((out2[2:9] != 5.0).any())
