"""The paged-cache workspace on a GPU: what a call leaves in it, whatever its outcome."""
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


# Batches whose row tiles x key tiles the chunk kernel could count, the few-rows kernel not.
@pytest.mark.parametrize("dtype,Hkv,max_kv", [(F32, 32, 131072), (F32, 8, 524288), (BF, 32, 524288)])
def test_a_refused_call_leaves_outputs_and_workspace(jfa, dtype, Hkv, max_kv):
    B, T, D, page = 8192, 64, 64, 1024
    c = Case([40, 1, 300, 17], [4000, 900, 5000, 17], H=Hkv, Hkv=Hkv, D=D, page=page, dtype=dtype, seed=Hkv)
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    ws = jfa.jfa_cache_workspace(cache, Hkv)
    i32 = dict(dtype=torch.int32, device="cuda")
    off = torch.full((B + 1,), T, **i32)
    off[0] = 0
    lens, table = torch.zeros(B, **i32), torch.zeros(B, max_kv // page, **i32)
    lens[0] = 4000
    Q = torch.zeros(T, Hkv, D, dtype=dtype, device="cuda")
    O, lse = torch.full_like(Q, 7.0), torch.full((T, Hkv), 9.0, device="cuda", dtype=F32)
    with pytest.raises(jfa.JFAError) as e:
        jfa.jfa_cache_fwd(cache, Q, off, lens, table, max_q_len=T, O=O, lse=lse, workspace=ws)
    assert e.value.status == jfa.JFA_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert bool((O == 7.0).all()) and bool((lse == 9.0).all()) and not ws[:jfa.JFA_CACHE_ZERO_BYTES].any()
    c.check(*c.run(jfa, cache, workspace=ws))  # the same workspace afterwards
    assert not ws[:jfa.JFA_CACHE_ZERO_BYTES].any()


# A record of a cut item as the chunk kernels leave it for the merge: first token, rows, first
# row, first head, first and last block, two words of padding; four flags a block say that its
# record is set.  Words of the zeroed part before the flags: 64 + 3 x 320.
FLAGS = 64 + 3 * 320


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64), (F32, 32)])
def test_records_of_another_batch_are_not_merged(jfa, dtype, D):
    H, Hkv, T, big = 4, 2, 40, 1 << 20
    c = Case([T], [100], H=H, Hkv=Hkv, D=D, page=16, dtype=dtype, seed=D)
    cache = jfa.jfa_cache_create(c.Kc, c.Vc)
    ws = jfa.jfa_cache_workspace(cache, H)
    words = ws.view(torch.int32)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    want, want_lse = c.run(jfa, cache, workspace=ws)
    O, lse = torch.full((3 * T, H, D), 7.0, dtype=dtype, device="cuda"), torch.full((3 * T, H), 9.0, device="cuda", dtype=F32)
    block = sms - 1  # (one that a call this small does not cut at)
    for record in ((big, 64, 0, 0, block, block), (T, 64, 0, 0, block, block), (T - 1, 64, 0, 0, block, block),
                   (0, 64, 2 * T, 0, block, block), (0, 64, 2 ** 31 - 1, 0, block, block), (-5, 64, 0, 0, block, block),
                   (0, 64, -9, 0, block, block), (0, 0, 0, 0, block, block), (0, big, 0, 0, block, block),
                   (0, 64, 0, H, block, block), (0, 64, 0, -1, block, block), (0, 64, 0, 0, block, block - 1),
                   (0, 64, 0, 0, -1, block), (0, 64, 0, 0, block, big), (0, 64, 0, 0, block, 4 * sms)):
        at = jfa.JFA_CACHE_ZERO_BYTES // 4 + 8 * block
        words[at:at + 8] = torch.tensor((*record, 0, 0), dtype=torch.int32, device="cuda")
        words[FLAGS + 4 * block:FLAGS + 4 * block + 4] = 1
        # (outputs in the middle of larger arrays: what the record names lies inside them)
        jfa.jfa_cache_fwd(cache, c.Q, c.q_off, c.kv_lens, c.table, max_q_len=T, O=O[T:2 * T], lse=lse[T:2 * T], workspace=ws)
        torch.cuda.synchronize()
        assert jfa.jfa_cache_device_status(cache) == jfa.JFA_ERR_DEVICE_BOUNDS, record
        assert torch.equal(O[T:2 * T], want) and torch.equal(lse[T:2 * T], want_lse), record
        assert bool((O[:T] == 7.0).all()) and bool((O[2 * T:] == 7.0).all())
        assert bool((lse[:T] == 9.0).all()) and bool((lse[2 * T:] == 9.0).all())
        assert not ws[:jfa.JFA_CACHE_ZERO_BYTES].any()
