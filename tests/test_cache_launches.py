"""What the paged-cache calls launch, and in which order they check: the library's host code
against a stand-in for the CUDA runtime and the kernels (fake_cuda.cpp), without a GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

from jagged_sequence_attention_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
WS = 1 << 20  # the workspace's address


@pytest.fixture(scope="module")
def jfa():
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def fake(jfa, tmp_path_factory):
    path = str(tmp_path_factory.mktemp("fake") / "libcache_fake.so")
    # (symbols bind within the library: torch has loaded a CUDA runtime of its own)
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-Wl,-z,defs",
                    "-I/usr/local/cuda/include", os.path.join(HERE, "fake_cuda.cpp"),
                    os.path.join(_build.BUILD, "cache.o"), "-o", path], check=True)
    L = ctypes.CDLL(path)
    for name in ("jfa_cache_create", "jfa_cache_destroy", "jfa_cache_append", "jfa_cache_workspace_size", "jfa_cache_fwd"):
        f = getattr(L, name)
        f.argtypes, f.restype = getattr(jfa.lib(), name).argtypes, getattr(jfa.lib(), name).restype
    L.fake_log.argtypes, L.fake_log.restype = [ctypes.c_char_p], ctypes.c_char_p
    return L


class Calls:
    """A cache of `Hkv` heads of 64 in pages of 1024, and attention over it."""

    def __init__(self, L, dtype, Hkv, g=1):
        self.L, self.H, self.D = L, Hkv * g, 64
        s = (ctypes.c_int64 * 3)(1024 * Hkv * 64, Hkv * 64, 64)
        self.h = ctypes.c_void_p()
        assert L.jfa_cache_create(dtype, Hkv, 64, 1024, 4, 1 << 16, 1 << 17, s, s, None, ctypes.byref(self.h)) == 0
        L.fake_log(b"")
        self.o_dtype = 1

    def fwd(self, B, T, max_q_len, max_kv, fail=""):
        """(status, what was launched)"""
        self.L.fake_log(fail.encode())
        n = self.L.jfa_cache_workspace_size(self.h, self.H)
        r = self.L.jfa_cache_fwd(self.h, B, T, max_q_len, 4096, 4096, 4096, max_kv // 1024, 1 << 18, self.H * self.D, self.H, 1, -1,
                                 0, None, 0.125, 1 << 19, self.o_dtype, None, WS, n, None)
        return r, self.L.fake_log(b"").decode()


BF16, F32 = 0, 1


@pytest.mark.parametrize("dtype,chunk,few", [(BF16, "chunk", "decode"), (F32, "split", "simt")])
def test_launches(jfa, fake, dtype, chunk, few):
    c = Calls(fake, dtype, 4, 2)
    assert c.fwd(3, 3, 1, 4096) == (jfa.JFA_OK, few)
    assert c.fwd(3, 100, 8, 4096) == (jfa.JFA_OK, few)
    assert c.fwd(3, 100, 9, 4096) == (jfa.JFA_OK, f"{chunk} {few} merge")
    assert c.fwd(3, 100, 0, 4096) == (jfa.JFA_OK, f"{chunk} {few} merge")
    assert c.fwd(0, 0, 0, 4096) == (jfa.JFA_OK, "")


# Batches that the chunk kernel could count and the few-rows kernel, with shorter key tiles and
# in fp32 four items a sequence, could not; and ones that neither could.
@pytest.mark.parametrize("dtype,Hkv,max_kv", [(F32, 32, 131072), (F32, 8, 524288), (BF16, 32, 524288), (F32, 64, 1 << 24),
                                              (BF16, 64, 1 << 24)])
def test_a_refused_call_launches_nothing(jfa, fake, dtype, Hkv, max_kv):
    c = Calls(fake, dtype, Hkv)
    for T, max_q_len in ((64, 64), (8192 * 17, 17), (8192, 0)):
        assert c.fwd(8192, T, max_q_len, max_kv) == (jfa.JFA_ERR_UNSUPPORTED, "")


def test_a_failed_tensor_map_launches_nothing(jfa, fake):
    c = Calls(fake, BF16, 4, 2)
    assert c.fwd(3, 100, 0, 4096, fail="encode") == (jfa.JFA_ERR_CUDA, "")


@pytest.mark.parametrize("dtype,chunk,few", [(BF16, "chunk", "decode"), (F32, "split", "simt")])
def test_a_failed_launch_leaves_the_workspace_zero(jfa, fake, dtype, chunk, few):
    """The chunk kernel sets flags that the merge clears: once its launch was tried, the merge
    follows, and where that fails, the zeroed part is zeroed on the stream."""
    c = Calls(fake, dtype, 4, 2)
    assert c.fwd(3, 100, 0, 4096, fail=chunk) == (jfa.JFA_ERR_CUDA, f"{chunk}! merge")
    assert c.fwd(3, 100, 0, 4096, fail=few) == (jfa.JFA_ERR_CUDA, f"{chunk} {few}! merge")
    zeroed = f"memset({WS},0,{jfa.JFA_CACHE_ZERO_BYTES})"
    assert c.fwd(3, 100, 0, 4096, fail="merge") == (jfa.JFA_ERR_CUDA, f"{chunk} {few} merge! {zeroed}")
    assert c.fwd(3, 3, 1, 4096, fail=few) == (jfa.JFA_ERR_CUDA, f"{few}!")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_arrays_of_another_device_are_refused(jfa, fake, dtype):
    """The handle's device is the current one; keys and values that lie on another would be read
    there by its kernels."""
    s = (ctypes.c_int64 * 3)(1024 * 64, 64, 64)

    def create(K, V, fail=""):
        h = ctypes.c_void_p()
        fake.fake_log(fail.encode())
        r = fake.jfa_cache_create(dtype, 1, 64, 1024, 4, K, V, s, s, None, ctypes.byref(h))
        assert (h.value is not None) == (r == jfa.JFA_OK)
        fake.jfa_cache_destroy(h)
        return r

    here, there, host = 1 << 20, 1 << 40, 1 << 41
    assert create(here, here) == jfa.JFA_OK
    for K, V in ((there, there), (here, there), (there, here)):
        assert create(K, V) == jfa.JFA_ERR_INVALID_ARG
    assert create(host, here) == jfa.JFA_OK             # memory of no device (managed, or the host's) is the caller's matter
    assert create(here, here, "attributes") == jfa.JFA_OK


class OnGpu:
    """What jfa_cache_create asks of an array, as on a machine with several GPUs."""

    dtype, shape, is_cuda = torch.bfloat16, (4, 16, 2, 64), True

    def __init__(self, device):
        self.device = torch.device("cuda", device)

    def dim(self):
        return 4

    def stride(self, i):
        return (2048, 128, 64, 1)[i]

    def data_ptr(self):
        return 4096


def test_binding_refuses_arrays_of_another_device(jfa, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(jfa, "_stream", lambda s=None: None)

    class Library:
        jfa_status_string = jfa.lib().jfa_status_string

        def jfa_cache_create(self, *a):
            pytest.fail("reached the library")

    monkeypatch.setattr(jfa, "lib", lambda: Library())
    for K, V in ((OnGpu(1), OnGpu(1)), (OnGpu(0), OnGpu(1))):
        with pytest.raises(jfa.JFAError) as e:
            jfa.jfa_cache_create(K, V)
        assert e.value.status == jfa.JFA_ERR_INVALID_ARG


def test_appending_keys_alone_ignores_the_queries_arguments(jfa, fake):
    c = Calls(fake, BF16, 4)

    def append(Q=None, Q_out=None, H=0, q_stride=0, qo_stride=0, rot=1 << 20):
        r = fake.jfa_cache_append(c.h, 2, 5, 4096, 4096, 4096, 3, 1 << 18, 256, 1 << 19, 256, Q, q_stride, H, Q_out, qo_stride, rot,
                                  64, 100, 0, None)
        return r, fake.fake_log(b"").decode()

    ok, bad = (jfa.JFA_OK, "append"), (jfa.JFA_ERR_INVALID_ARG, "")
    assert append() == ok and append(rot=None) == ok and append(H=-3) == ok
    assert append(q_stride=512, qo_stride=3) == ok
    q = 1 << 21
    assert append(q, q, 8, 512, 512) == ok and append(q, q + (1 << 16), 8, 512, 1024) == ok
    assert append(q, q, 8, 512, 1024) == bad and append(q, q, 8, 511, 511) == bad and append(q, None, 8, 512) == bad
    assert append(q, q, 0, 512, 512) == bad and append(q, q, 8, 512, 512, rot=None) == bad
