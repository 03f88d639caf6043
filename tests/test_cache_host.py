"""Paged-cache entry points without a GPU: argument errors are found on the host before
any CUDA call, the binding refuses what it would misread, and planning without a device
fails loudly."""
import ctypes

import pytest
import torch

from jagged_sequence_attention_gb300 import _build


@pytest.fixture(scope="module")
def jfa():
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    m.lib()
    return m


def create(jfa, dtype=0, Hkv=2, D=64, page=16, n=4, K=4096, V=8192, ks=(2048, 128, 64), vs=(2048, 128, 64)):
    s = lambda x: None if x is None else (ctypes.c_int64 * 3)(*x)  # noqa: E731
    h = ctypes.c_void_p(1)
    r = jfa.lib().jfa_cache_create(dtype, Hkv, D, page, n, K, V, s(ks), s(vs), None, ctypes.byref(h))
    return r, h.value


def test_create_checks_its_arguments(jfa):
    bad, uns = jfa.JFA_ERR_INVALID_ARG, jfa.JFA_ERR_UNSUPPORTED
    for kw in (dict(dtype=2), dict(Hkv=0), dict(n=0), dict(n=2 ** 31), dict(K=None), dict(V=None), dict(K=4104),
               dict(ks=None), dict(vs=None), dict(ks=(2048, 128, 63)), dict(ks=(2048, 132, 64)), dict(vs=(0, 128, 64)),
               dict(vs=(-2048, 128, 64)), dict(ks=(2 ** 39, 128, 64))):
        assert create(jfa, **kw) == (bad, None), kw
    for kw in (dict(D=32), dict(D=96), dict(dtype=1, D=128), dict(page=4), dict(page=24), dict(page=2048)):
        assert create(jfa, **kw) == (uns, None), kw
    assert jfa.lib().jfa_cache_create(0, 2, 64, 16, 4, 4096, 8192, None, None, None, None) == bad


def test_create_without_a_gpu_fails_loudly(jfa):
    if torch.cuda.is_available():
        pytest.skip("checks the behaviour without a GPU")
    assert create(jfa) == (jfa.JFA_ERR_NO_DEVICE, None)


def test_null_handles(jfa):
    L = jfa.lib()
    bad = jfa.JFA_ERR_INVALID_ARG
    assert L.jfa_cache_destroy(None) == jfa.JFA_OK
    assert L.jfa_cache_device_status(None, None) == bad
    assert L.jfa_cache_workspace_size(None, 8) == 0
    assert L.jfa_cache_append(None, 1, 1, 4, 4, 4, 1, 16, 64, 16, 64, None, 0, 0, None, 0, None, 0, 0, 0, None) == bad
    assert L.jfa_cache_fwd(None, 1, 1, 1, 4, 4, 4, 1, 16, 64, 1, 1, -1, 0, None, 1.0, 16, 0, None, 256, 0, None) == bad


def test_binding_refuses_what_it_would_misread(jfa):
    K = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(jfa.JFAError) as e:  # host tensors
        jfa.jfa_cache_create(K, K)
    assert e.value.status == jfa.JFA_ERR_INVALID_ARG
    cache = jfa.Cache(None, K, K)
    off, kv, table = (torch.zeros(n, dtype=torch.int32) for n in (3, 2, 10))
    table = table.view(2, 5)
    assert jfa._cache_batch("f", cache, off, kv, table) == (2, 5)
    for a in ((off.long(), kv, table), (off[:2], kv, table), (off, kv, table.view(-1)), (off, kv, table.t()),
              (off, kv, table[:1]), (off, kv, torch.zeros(2, 10, dtype=torch.int32)[:, ::2])):
        with pytest.raises(jfa.JFAError):
            jfa._cache_batch("f", cache, *a)
    wide = torch.zeros(7, 8, 64, dtype=torch.bfloat16)
    assert jfa._cache_rows("f", cache, wide, 8) == 512
    assert jfa._cache_rows("f", cache, wide[:, 2:4], 2) == 512     # a slice of a fused projection
    assert jfa._cache_rows("f", cache, wide[:1, 2:4], 2) == 128    # one token: its stride says nothing
    for t, heads in ((wide, 4), (wide.float(), 8), (wide[..., :32], 8), (wide[:, ::2], 4), (wide.transpose(0, 1), 7),
                     (wide[:, :, ::2], 8)):
        with pytest.raises(jfa.JFAError):
            jfa._cache_rows("f", cache, t, heads)
