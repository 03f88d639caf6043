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
