"""Entry points of 4-bit caches and of selected blocks without a GPU: argument errors are found on the
host before any CUDA call, the binding refuses what it would misread, and planning without a
device fails loudly."""
import ctypes

import pytest
import torch

from jagged_sequence_attention_gb300 import _build

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


@pytest.fixture(scope="module")
def jfa():
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    m.lib()
    return m


def create(jfa, Hkv=2, D=64, page=16, n=4, K=4096, V=8192, ks=(1024, 64, 32), vs=(1024, 64, 32), Ks=4096, Vs=8192, kss=(128, 64),
           vss=(128, 64), kf=1.0, vf=1.0):
    s = lambda x: None if x is None else (ctypes.c_int64 * len(x))(*x)  # noqa: E731
    h = ctypes.c_void_p(1)
    r = jfa.lib().jfa_cache_create_quantized(Hkv, D, page, n, K, V, s(ks), s(vs), Ks, Vs, s(kss), s(vss), kf, vf, None, ctypes.byref(h))
    return r, h.value


def test_create_checks_its_arguments(jfa):
    bad, uns = jfa.JFA_ERR_INVALID_ARG, jfa.JFA_ERR_UNSUPPORTED
    for kw in (dict(Hkv=0), dict(n=0), dict(n=2 ** 31), dict(K=None), dict(V=None), dict(Ks=None), dict(Vs=None), dict(K=4104), dict(Vs=8200),
               dict(ks=None), dict(vs=None), dict(kss=None), dict(vss=None), dict(ks=(1024, 64, 16)), dict(ks=(1024, 64, 40)),
               dict(vs=(0, 64, 32)), dict(vs=(-1024, 64, 32)), dict(kss=(128, 48)), dict(kss=(136, 64)), dict(vss=(128, -64)),
               dict(kss=(2 ** 62, 64)), dict(kf=0.0), dict(kf=-1.0), dict(vf=float("nan")), dict(vf=float("inf")), dict(kf=2.0 ** -61),
               dict(vf=2.0 ** 61)):
        assert create(jfa, **kw) == (bad, None), kw
    for kw in (dict(D=32), dict(D=96), dict(D=256), dict(page=4), dict(page=24), dict(page=2048)):
        assert create(jfa, **kw) == (uns, None), kw
    assert jfa.lib().jfa_cache_create_quantized(2, 64, 16, 4, 4096, 8192, None, None, 4096, 8192, None, None, 1.0, 1.0, None, None) == bad


def test_create_without_a_gpu_fails_loudly(jfa):
    if torch.cuda.is_available():
        pytest.skip("checks the behaviour without a GPU")
    assert create(jfa) == (jfa.JFA_ERR_NO_DEVICE, None)


def test_null_handles(jfa):
    L, bad = jfa.lib(), jfa.JFA_ERR_INVALID_ARG
    assert L.jfa_cache_read(None, 1, 1, 4, 4, 4, 1, 16, 64, 16, 64, None) == bad
    assert L.jfa_cache_summarize(None, 1, 1, 4, 4, 4, 1, 16, None) == bad
    assert L.jfa_cache_select_workspace_size(None, 1, 1) == 0
    assert L.jfa_cache_select(None, 1, 1, 1, 4, 4, 4, 1, 16, 16, 64, 1, 1, 0, 1, 16, 256, 0, None) == bad
    assert L.jfa_cache_fwd_blocks(None, 1, 1, 4, 4, 4, 1, 16, 64, 1, 16, 1, 0, None, 1.0, 16, 0, None, 256, 0, None) == bad


def test_binding_refuses_what_it_would_misread(jfa):
    codes, scales = torch.zeros(4, 16, 2, 32, dtype=U8), torch.zeros(4, 2, 16, 4, dtype=U8)
    bad = jfa.JFA_ERR_INVALID_ARG
    for args in ((codes, codes, scales, scales), (codes.float(), codes, scales, scales), (codes, codes, scales[:2], scales)):
        with pytest.raises(jfa.JFAError) as e:  # host tensors, other types, other shapes
            jfa.jfa_cache_create_quantized(*args)
        assert e.value.status == bad
    # on host tensors every check of the compiled calls passes or fails as it would on a GPU; a
    # call that passes them reaches the library, which refuses the null handle
    cache = jfa.Cache(ctypes.c_void_p(), codes, codes, (scales, scales))
    calls = jfa._cache_calls()
    off, kv, table = (torch.zeros(n, dtype=I32) for n in (3, 2, 10))
    table = table.view(2, 5)
    wide = torch.zeros(7, 8, 64, dtype=BF)
    batch = dict(off=off, kv=kv, table=table)
    batches = (dict(off=off.long()), dict(off=off[:2]), dict(table=table.view(-1)), dict(table=table.t()), dict(table=table[:1]), dict(kv=None))

    def refused(call, good, wrong):
        assert call(cache.info, *good.values()) == bad
        for kw in wrong:
            with pytest.raises((ValueError, TypeError)):
                call(cache.info, *dict(good, **kw).values())

    refused(calls.read, dict(T=7, **batch, K=wide[:, 2:4], V=wide[:, 4:6], stream=0),
            (*batches, dict(T=8), dict(T=-1), dict(T=None), dict(K=wide), dict(V=wide[:, ::4]), dict(K=wide[:, :2].float()), dict(V=None)))
    bounds = torch.zeros(4, 2, 2, 64, dtype=BF)
    refused(calls.summarize, dict(n_pages=4, bounds=bounds, T=7, **batch, stream=0),
            (*batches, dict(bounds=bounds.float()), dict(bounds=bounds[:3]), dict(bounds=bounds[..., :32]), dict(bounds=bounds.transpose(1, 2)),
             dict(bounds=bounds.view(4, 4, 64)), dict(T=1.5)))
    lists, ws = torch.zeros(7, 2, 3, dtype=I32), torch.zeros(512, dtype=U8)
    refused(calls.select, dict(n_pages=4, bounds=bounds, Q=wide, **batch, n=3, first=1, last=1, max_q=None, blocks=lists, ws=ws, stream=0),
            (*batches, dict(bounds=bounds[:3]), dict(Q=wide.float()), dict(Q=wide[:, ::2]), dict(Q=wide[:6]), dict(n=4), dict(n=0),
             dict(first=None), dict(last=1.5), dict(max_q="7"), dict(blocks=lists.long()), dict(blocks=lists[:, :1]),
             dict(blocks=lists.transpose(1, 2)), dict(ws=ws[::2]), dict(ws=None)))
    O, lse = torch.zeros(7, 8, 64, dtype=BF), torch.zeros(7, 8, dtype=F32)
    good = dict(Q=wide, **batch, blocks=lists, bias=None, scale=0.1, O=O, lse=lse, ws=ws, stream=0)
    refused(calls.fwd_blocks, good,
            (*batches, dict(Q=wide.double()), dict(Q=wide[0]), dict(blocks=lists[:6]), dict(blocks=lists.float()), dict(blocks=lists[..., ::2]),
             dict(bias=torch.zeros(8, 31, dtype=F32)), dict(bias=torch.zeros(7, 32, dtype=F32)), dict(scale=None), dict(O=O[:, :4]), dict(O=O.transpose(0, 1)),
             dict(lse=lse.double()), dict(lse=lse.view(-1)), dict(ws=None)))
    assert calls.fwd_blocks(cache.info, *dict(good, O=O.half()).values()) == jfa.JFA_ERR_UNSUPPORTED


def test_public_calls_have_the_binding_s_error(jfa):
    codes, scales = torch.zeros(4, 16, 2, 32, dtype=U8), torch.zeros(4, 2, 16, 4, dtype=U8)
    cache = jfa.Cache(ctypes.c_void_p(), codes, codes, (scales, scales))
    off, kv, table = torch.zeros(3, dtype=I32), torch.zeros(2, dtype=I32), torch.zeros(2, 5, dtype=I32)
    Q, bounds, lists, ws = torch.zeros(7, 8, 64, dtype=BF), torch.zeros(4, 2, 2, 64, dtype=BF), torch.zeros(7, 2, 3, dtype=I32), torch.zeros(512, dtype=U8)
    O, lse = torch.zeros(7, 8, 64, dtype=F32), torch.zeros(7, 8, dtype=F32)
    for call in (lambda: jfa.jfa_cache_read(cache, 7, off, kv, table, K=Q, V=Q),
                 lambda: jfa.jfa_cache_summarize(cache, bounds[:1], 7, off, kv, table),
                 lambda: jfa.jfa_cache_select(cache, bounds, Q, off, kv, table, 4, blocks=lists, workspace=ws),
                 lambda: jfa.jfa_cache_select(cache, bounds, Q, off, kv, table, 2 ** 70, blocks=lists, workspace=ws),
                 lambda: jfa.jfa_cache_select(cache, bounds, Q, off, kv, table, 0, blocks=lists, workspace=ws),
                 lambda: jfa.jfa_cache_fwd_blocks(cache, Q, off, kv, table, lists.long(), O=O, lse=lse, workspace=ws)):
        with pytest.raises(jfa.JFAError) as e:
            call()
        assert e.value.status == jfa.JFA_ERR_INVALID_ARG
    cache.handle = cache.info = None        # as after jfa_cache_destroy
    for call in (lambda: jfa.jfa_cache_read(cache, 7, off, kv, table), lambda: jfa.jfa_cache_summarize(cache, bounds, 7, off, kv, table),
                 lambda: jfa.jfa_cache_select(cache, bounds, Q, off, kv, table, 3),
                 lambda: jfa.jfa_cache_fwd_blocks(cache, Q, off, kv, table, lists)):
        with pytest.raises(jfa.JFAError):
            call()
