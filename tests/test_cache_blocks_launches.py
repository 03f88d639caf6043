"""What the calls on 4-bit caches and selected blocks launch, and in which order they check: the library's host
code against a stand-in for the CUDA runtime and the kernels (fake_cuda_blocks.cpp), without a GPU."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from jagged_sequence_attention_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))
WS, Q, K, V, O, L, BOUNDS, LISTS = (1 << i for i in range(20, 28))  # addresses
CALLS = ("jfa_cache_create", "jfa_cache_create_quantized", "jfa_cache_destroy", "jfa_cache_append", "jfa_cache_workspace_size",
         "jfa_cache_fwd", "jfa_cache_read", "jfa_cache_summarize", "jfa_cache_select_workspace_size", "jfa_cache_select",
         "jfa_cache_fwd_blocks")


@pytest.fixture(scope="module")
def jfa():
    _build.build()
    from jagged_sequence_attention_gb300 import jfa as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def fake(jfa, tmp_path_factory):
    path = str(tmp_path_factory.mktemp("fake") / "libblocks_fake.so")
    # (symbols bind within the library: torch has loaded a CUDA runtime of its own)
    subprocess.run([_build._nvcc(), "-O1", "-std=c++17", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC", *_build.ARCH,
                    "-Xlinker", "-Bsymbolic", "-Xlinker", "-z", "-Xlinker", "defs", "-I", _build.CSRC, "-I", _build.INCLUDE,
                    os.path.join(HERE, "fake_cuda_blocks.cpp"), os.path.join(HERE, "fake_cuda_blocks.cu"),
                    *(os.path.join(_build.BUILD, f"cache{x}.o") for x in ("", "_quant", "_blocks")), "-o", path], check=True)
    return load(jfa, path)


def load(jfa, path):
    lib = ctypes.CDLL(path)
    for name in CALLS:
        f = getattr(lib, name)
        f.argtypes, f.restype = getattr(jfa.lib(), name).argtypes, getattr(jfa.lib(), name).restype
    lib.fake_log.argtypes, lib.fake_log.restype = [ctypes.c_char_p], ctypes.c_char_p
    lib.fake_scale_log2.restype = ctypes.c_float
    lib.path = path
    return lib


class Calls:
    """A cache of `Hkv` heads of 64 (bits 4 or 16), and the calls on it."""

    def __init__(self, lib, bits, Hkv=4, g=2, page=1024, factor=1.0):
        self.lib, self.bits, self.Hkv, self.H, self.D, self.page = lib, bits, Hkv, Hkv * g, 64, page
        self.h = ctypes.c_void_p()
        s = lambda *x: (ctypes.c_int64 * len(x))(*x)  # noqa: E731
        if bits == 4:
            k, sc = s(page * Hkv * 32, Hkv * 32, 32), s(Hkv * page * 4, page * 4)
            r = lib.jfa_cache_create_quantized(Hkv, 64, page, 4, K, V, k, k, K, V, sc, sc, factor, 1.0, None, ctypes.byref(self.h))
        else:
            k = s(page * Hkv * 64, Hkv * 64, 64)
            r = lib.jfa_cache_create(bits == 32, Hkv, 64, page, 4, K, V, k, k, None, ctypes.byref(self.h))
        assert r == 0
        lib.fake_log(b"")

    def logged(self, call, fail):
        self.lib.fake_log(fail.encode())
        r = call()
        return r, self.lib.fake_log(b"").decode()

    def fwd(self, B, T, max_q_len, max_kv, fail="", scale=0.125, causal=1, window=-1):
        n = self.lib.jfa_cache_workspace_size(self.h, self.H)
        return self.logged(lambda: self.lib.jfa_cache_fwd(
            self.h, B, T, max_q_len, 4096, 4096, 4096, max_kv // self.page, Q, self.H * self.D, self.H, causal, window, 0, None, scale, O,
            1, None, WS, n, None), fail)

    def fwd_blocks(self, B, T, n_blocks, max_kv, fail="", scale=0.125):
        n = self.lib.jfa_cache_workspace_size(self.h, self.H)
        return self.logged(lambda: self.lib.jfa_cache_fwd_blocks(
            self.h, B, T, 4096, 4096, 4096, max_kv // self.page, Q, self.H * self.D, self.H, LISTS, n_blocks, 0, None, scale, O, 1, None,
            WS, n, None), fail)

    def select(self, B, T, max_q_len, pages, n_blocks, fail="", first=1, last=1, short=0):
        n = self.lib.jfa_cache_select_workspace_size(self.h, T, pages) - short
        return self.logged(lambda: self.lib.jfa_cache_select(
            self.h, B, T, max_q_len, 4096, 4096, 4096, pages, BOUNDS, Q, self.H * self.D, self.H, n_blocks, first, last, LISTS, WS, n,
            None), fail)

    def summarize(self, T, fail=""):
        return self.logged(lambda: self.lib.jfa_cache_summarize(self.h, 2, T, 4096, 4096, 4096, 9, BOUNDS, None), fail)

    def rows(self, name, T, fail=""):
        n = self.Hkv * self.D
        tail = (None,) if name == "read" else (None, 0, 0, None, 0, None, 0, 0, 0, None)
        return self.logged(lambda: getattr(self.lib, "jfa_cache_" + name)(self.h, 2, T, 4096, 4096, 4096, 9, Q, n, O, n, *tail), fail)


def test_launches_over_4_bits(jfa, fake):
    c = Calls(fake, 4)
    assert c.fwd(3, 3, 1, 4096) == (jfa.JFA_OK, "decode4:8")
    assert c.fwd(3, 100, 4, 4096) == (jfa.JFA_OK, "decode4:8")        # 8 packed rows
    assert c.fwd(3, 100, 5, 4096) == (jfa.JFA_OK, "decode4:16")
    assert c.fwd(3, 100, 8, 4096) == (jfa.JFA_OK, "decode4:16")
    both = "chunk4:256 decode4:16:early merge"
    for max_q_len in (9, 0, 10 ** 6):
        assert c.fwd(3, 100, max_q_len, 4096) == (jfa.JFA_OK, both)
    assert c.fwd(3, 100, 0, 4096, causal=0) == c.fwd(3, 100, 0, 4096, window=7) == (jfa.JFA_OK, both)
    assert c.fwd(0, 0, 0, 4096) == (jfa.JFA_OK, "")
    assert c.fwd(1, 4, 0, 4096) == (jfa.JFA_OK, "decode4:8")          # no more tokens than T
    assert Calls(fake, 4, 2, 24).fwd(3, 3, 1, 4096) == (jfa.JFA_OK, "chunk4:240 decode4:16:early merge")
    assert Calls(fake, 4, 1, 129).fwd(3, 3, 1, 4096) == (jfa.JFA_ERR_UNSUPPORTED, "")
    assert Calls(fake, 16).fwd(3, 100, 0, 4096) == (jfa.JFA_OK, "chunk decode merge")
    # (the records of cut items come on top)
    assert fake.jfa_cache_workspace_size(c.h, 8) > fake.jfa_cache_workspace_size(Calls(fake, 16).h, 8)


@pytest.mark.parametrize("Hkv,max_kv", [(32, 524288), (64, 1 << 24)])
def test_a_refused_call_over_4_bits_launches_nothing(jfa, fake, Hkv, max_kv):
    c = Calls(fake, 4, Hkv, 1)
    for T, max_q_len in ((64, 64), (8192 * 17, 17), (8192, 0)):
        assert c.fwd(8192, T, max_q_len, max_kv) == (jfa.JFA_ERR_UNSUPPORTED, "")
    assert c.fwd(3, 100, 0, 4096, fail="encode") == (jfa.JFA_ERR_CUDA, "")


def test_a_failed_launch_over_4_bits_leaves_the_workspace_zero(jfa, fake):
    c = Calls(fake, 4)
    assert c.fwd(3, 100, 0, 4096, fail="chunk4") == (jfa.JFA_ERR_CUDA, "chunk4!:256 merge")
    assert c.fwd(3, 100, 0, 4096, fail="decode4") == (jfa.JFA_ERR_CUDA, "chunk4:256 decode4!:16:early merge")
    zeroed = f"memset({WS},0,{jfa.JFA_CACHE_ZERO_BYTES})"
    assert c.fwd(3, 100, 0, 4096, fail="merge") == (jfa.JFA_ERR_CUDA, f"chunk4:256 decode4:16:early merge! {zeroed}")
    assert c.fwd(3, 3, 1, 4096, fail="decode4") == (jfa.JFA_ERR_CUDA, "decode4!:8")


@pytest.mark.parametrize("factor,scale", [(1.0, 0.125), (2.0 ** -60, 3e38), (2.0 ** 60, 1e-45), (0.3, 0.7), (2.0 ** -60, 1e-20), (2.0 ** 60, 1e20)])
def test_the_scale_takes_the_factor_first(jfa, fake, factor, scale):
    f32 = np.float32
    c = Calls(fake, 4, factor=factor)
    want = f32(scale) * f32(factor)
    for call in (lambda: c.fwd(3, 3, 1, 4096, scale=scale), lambda: c.fwd(3, 100, 0, 4096, scale=scale),
                 lambda: c.fwd_blocks(3, 3, 2, 4096, scale=scale)):
        status, log = call()
        if 1e-37 <= want <= 1e37:
            assert status == jfa.JFA_OK and fake.fake_scale_log2() == want * f32(1.4426950408889634)
        else:
            assert (status, log) == (jfa.JFA_ERR_INVALID_ARG, "")


@pytest.mark.parametrize("bits,name", [(4, "lists4"), (16, "lists")])
def test_attention_over_blocks(jfa, fake, bits, name):
    for g in (1, 2, 16):
        c = Calls(fake, bits, 4, g)
        assert c.fwd_blocks(3, 100, 5, 4096) == (jfa.JFA_OK, f"{name}:{g}")
        assert c.fwd_blocks(3, 100, 5, 4096, fail=name) == (jfa.JFA_ERR_CUDA, f"{name}!:{g}")
    assert c.fwd_blocks(0, 0, 5, 4096) == (jfa.JFA_OK, "")
    for n in (0, -1, (1 << 20) + 1):
        assert c.fwd_blocks(3, 100, n, 4096) == (jfa.JFA_ERR_INVALID_ARG, "")
    assert c.fwd_blocks(3, 1 << 20, 1 << 20, 1 << 30) == (jfa.JFA_ERR_UNSUPPORTED, "")     # more units than can be counted
    assert Calls(fake, bits, 4, 17).fwd_blocks(3, 100, 5, 4096) == (jfa.JFA_ERR_UNSUPPORTED, "")
    assert Calls(fake, bits, 4, page=8).fwd_blocks(3, 100, 5, 4096) == (jfa.JFA_ERR_UNSUPPORTED, "")


@pytest.mark.parametrize("bits", [4, 16])
def test_selection(jfa, fake, bits):
    c = Calls(fake, bits)
    # scores by the token or in tiles, the choice by a warp, four or 32
    assert c.select(3, 3, 1, 200, 5) == (jfa.JFA_OK, "score64 choose4:early")
    assert c.select(3, 400, 4, 200, 5) == (jfa.JFA_OK, "score64 choose1:early")
    assert c.select(3, 400, 0, 200, 5) == (jfa.JFA_OK, "score_tile64 choose1:early")
    assert c.select(3, 400, 0, 513, 5) == (jfa.JFA_OK, "score_tile64 choose4:early")
    assert c.select(60, 400, 0, 513, 5) == (jfa.JFA_OK, "score64 choose4:early")
    assert c.select(3, 3, 1, 1025, 5) == (jfa.JFA_OK, "score64 choose32:early")
    assert c.select(3, 3, 1, 5, 5) == (jfa.JFA_OK, "choose4")                              # nothing competes
    assert c.select(0, 0, 0, 200, 5) == (jfa.JFA_OK, "")
    assert c.select(3, 3, 1, 200, 5, fail="score64") == (jfa.JFA_ERR_CUDA, "score64!")
    assert c.select(3, 400, 0, 200, 5, fail="score_tile64") == (jfa.JFA_ERR_CUDA, "score_tile64!")
    assert c.select(3, 3, 1, 200, 5, fail="choose4") == (jfa.JFA_ERR_CUDA, "score64 choose4!:early")
    assert c.select(3, 3, 1, 200, 5) == (jfa.JFA_OK, "score64 choose4:early")              # (an error is one call's)
    bad = (jfa.JFA_ERR_INVALID_ARG, "")
    assert c.select(3, 3, 1, 200, 5, short=1) == bad and c.select(3, 3, -1, 200, 5) == bad
    assert c.select(3, 3, 1, 200, 5, first=-1) == c.select(3, 3, 1, 200, 5, last=0) == c.select(3, 3, 1, 200, 5, first=3, last=3) == bad
    assert c.select(3, 3, 1, 65535 * 64 + 1, 5) == (jfa.JFA_ERR_UNSUPPORTED, "")
    assert Calls(fake, bits, 1, 129).select(3, 3, 1, 200, 5) == (jfa.JFA_ERR_UNSUPPORTED, "")
    for call in (lambda x: x.select(3, 3, 1, 200, 5), lambda x: x.summarize(3)):
        assert call(Calls(fake, 32)) == call(Calls(fake, bits, page=8)) == (jfa.JFA_ERR_UNSUPPORTED, "")


def test_select_workspace_of_sizes_past_its_limits(jfa, fake):
    size = fake.jfa_cache_select_workspace_size
    c = Calls(fake, 16, 8, 1)
    for T, pages in ((0, 0), (1, 1), (1, 64), (1, 65), (2 ** 28 - 1, 65535 * 64)):
        assert size(c.h, T, pages) == 256 + 4 * T * 8 * (pages + max(1, -(-pages // 64)))
    # what the call refuses, past 64 bits or not
    for T, pages in ((1, 65535 * 64 + 1), (1, 2 ** 31 - 1), (2 ** 28, 1), (2 ** 30, 2 ** 30), (-1, 1), (1, -1)):
        assert size(c.h, T, pages) == 0
    assert c.select(3, 2 ** 28, 1, 200, 5) == (jfa.JFA_ERR_INVALID_ARG, "")
    assert c.select(3, 3, 1, 2 ** 31 - 1, 5) == (jfa.JFA_ERR_UNSUPPORTED, "")


@pytest.mark.parametrize("bits,append,read", [(4, "append4", "read4"), (16, "append", "read16"), (32, "append", "read32")])
def test_rows_and_bounds(jfa, fake, bits, append, read):
    c = Calls(fake, bits)
    for name, kernel in (("append", append), ("read", read)):
        assert c.rows(name, 7) == (jfa.JFA_OK, kernel) and c.rows(name, 0) == (jfa.JFA_OK, "")
        assert c.rows(name, 7, fail=kernel) == (jfa.JFA_ERR_CUDA, kernel + "!")
    if bits < 32:
        assert c.summarize(7) == (jfa.JFA_OK, "summarize") and c.summarize(0) == (jfa.JFA_OK, "")
        assert c.summarize(7, fail="summarize") == (jfa.JFA_ERR_CUDA, "summarize!")


def test_arrays_of_another_device_are_refused(jfa, fake):
    s = lambda *x: (ctypes.c_int64 * len(x))(*x)  # noqa: E731
    here, there = 1 << 20, 1 << 40
    for at in range(5):
        a = [there if i == at else here for i in range(4)]
        h = ctypes.c_void_p()
        r = fake.jfa_cache_create_quantized(2, 64, 16, 4, a[0], a[1], s(1024, 64, 32), s(1024, 64, 32), a[2], a[3], s(128, 64), s(128, 64), 1.0,
                                            1.0, None, ctypes.byref(h))
        assert r == (jfa.JFA_OK if at == 4 else jfa.JFA_ERR_INVALID_ARG) and (h.value is not None) == (at == 4)
        fake.jfa_cache_destroy(h)


def test_libraries_of_a_process_share_nothing(jfa, fake, tmp_path):
    """Tensor maps are encoded by what each library has found itself: the library that runs on a GPU must not use
    what a stand-in in the same process has."""
    assert Calls(fake, 4).fwd(3, 100, 0, 4096) == (jfa.JFA_OK, "chunk4:256 decode4:16:early merge")
    other = load(jfa, shutil.copy(fake.path, tmp_path / "libother.so"))
    c = Calls(other, 4)
    assert c.fwd(3, 100, 0, 4096, fail="encode") == (jfa.JFA_ERR_CUDA, "")
    # (a call that fails in the first is none of the second's)
    fake.fake_log(b"encode")
    assert c.fwd(3, 100, 0, 4096) == (jfa.JFA_OK, "chunk4:256 decode4:16:early merge")
    fake.fake_log(b"")
