"""Paged-cache entry points without a GPU: argument errors are found on the host before
any CUDA call, the binding refuses what it would misread, and planning without a device
fails loudly."""
import ctypes
import os
import re

import pytest
import torch

F32 = torch.float32

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


def test_binding_constant_matches_the_header(jfa):
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "jfa.h")).read()
    m = re.search(r"#define\s+JFA_CACHE_ZERO_BYTES\s+\(\(size_t\)(\d+)\)", text)
    assert m and jfa.JFA_CACHE_ZERO_BYTES == int(m.group(1))


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
    # on host tensors every check of the compiled calls passes or fails as it would on a GPU; a
    # call that passes them reaches the library, which refuses the null handle
    cache = jfa.Cache(ctypes.c_void_p(), K, K)
    calls = jfa._cache_calls()
    off, kv, table = (torch.zeros(n, dtype=torch.int32) for n in (3, 2, 10))
    table = table.view(2, 5)
    wide = torch.zeros(7, 8, 64, dtype=torch.bfloat16)
    k, v, q, rot = wide[:, 2:4], wide[:, 4:6], wide[:, :2], torch.zeros(9, 32, dtype=F32)
    good = dict(K=k, V=v, off=off, kv=kv, table=table, Q=q, Qo=q.clone(), rot=rot, kind=0, stream=0)

    def append(**kw):
        a = dict(good, **kw)
        return calls.append(cache.info, *(a[n] for n in good))

    bad = jfa.JFA_ERR_INVALID_ARG
    assert append() == bad and append(Q=None, Qo=None) == bad and append(K=k[:1], V=v[:1], Q=q[:1], Qo=q[:1]) == bad
    for kw in (dict(off=off.long()), dict(off=off[:2]), dict(table=table.view(-1)), dict(table=table.t()),
               dict(table=table[:1]), dict(table=torch.zeros(2, 10, dtype=torch.int32)[:, ::2]), dict(K=wide),
               dict(K=k.float()), dict(K=k[..., :32]), dict(K=wide[:, ::4]), dict(V=v[:3]), dict(Q=q.transpose(0, 1)),
               dict(Qo=q[:, :1]), dict(Qo=None), dict(Q=None), dict(rot=rot.double()), dict(rot=rot.t()),
               dict(K=None), dict(kind=None)):
        with pytest.raises((ValueError, TypeError)):
            append(**kw)
    fgood = dict(Q=q, off=off, kv=kv, table=table, bias=torch.zeros(2, 32, dtype=F32), scale=0.1, causal=True, window=None, n=None,
                 O=torch.zeros(7, 2, 64, dtype=F32), lse=torch.zeros(7, 2, dtype=F32), ws=torch.zeros(8, dtype=torch.uint8), stream=0)

    def fwd(**kw):
        a = dict(fgood, **kw)
        return calls.fwd(cache.info, *(a[n] for n in fgood))

    assert fwd() == bad and fwd(bias=None, window=3, n=7) == bad
    assert fwd(O=torch.zeros(7, 2, 64, dtype=torch.float16)) == jfa.JFA_ERR_UNSUPPORTED
    for kw in (dict(kv=kv.long()), dict(Q=q.double()), dict(Q=wide[0]), dict(bias=torch.zeros(2, 31, dtype=F32)),
               dict(bias=torch.zeros(3, 32, dtype=F32)), dict(O=torch.zeros(7, 3, 64, dtype=F32)), dict(O=torch.zeros(2, 7, 64, dtype=F32).transpose(0, 1)),
               dict(lse=torch.zeros(7, dtype=F32)), dict(lse=torch.zeros(7, 2, dtype=F32).double()), dict(ws=torch.zeros(8, 2, dtype=F32).t()),
               dict(scale=None), dict(window=1.5), dict(O=None)):
        with pytest.raises((ValueError, TypeError)):
            fwd(**kw)
    with pytest.raises(jfa.JFAError) as e:  # the public call, with the binding's own error
        jfa.jfa_cache_append(cache, wide, v, off, kv, table)
    assert e.value.status == bad
    for kw in (dict(window=2 ** 70), dict(max_q_len=-2 ** 70)):
        with pytest.raises(jfa.JFAError) as e:
            jfa.jfa_cache_fwd(cache, q, off, kv, table, O=fgood["O"], lse=fgood["lse"], workspace=fgood["ws"], **kw)
        assert e.value.status == bad
    cache.handle = cache.info = None        # as after jfa_cache_destroy
    with pytest.raises(jfa.JFAError):
        jfa.jfa_cache_append(cache, k, v, off, kv, table)
