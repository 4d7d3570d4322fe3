"""The host side of the window decodes and of the table builder over a stand-in for the device
(``tests/fakes/window_host.cpp``): which device a call's arrays may be on, and what a launch gets."""
import ctypes
import importlib
import os
import subprocess

import pytest

import paged_kv_decode_attn_gb300 as oxd

B = importlib.import_module("paged_kv_decode_attn_gb300.build")  # (the package's name is the function)
HERE = os.path.dirname(os.path.abspath(__file__))
BASE, GAP = 1 << 40, 1 << 32
DEVICE, MANAGED = 2, 3  # cudaMemoryType


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("fakes") / "window_host.so")
    subprocess.run([B.nvcc(), "-std=c++17", "-O1", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC",
                    "-Xlinker", "-Bsymbolic", "-I", os.path.join(B.ROOT, "include"), "-I", B.CSRC,
                    os.path.join(HERE, "fakes", "window_host.cpp"),
                    os.path.join(B.CSRC, "oxd_window_host.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    L.fake_allocate.argtypes = [vp, sz, ctypes.c_int, ctypes.c_int]
    L.oxd_window_decode.argtypes = [vp] * 7 + [ctypes.c_float, vp, vp, vp, sz, vp]
    L.oxd_quant_window_decode.argtypes = [vp] * 6 + [ctypes.c_float, vp, vp, vp, sz, vp]
    L.oxd_build_tables.argtypes = [vp] * 18 + [sz, vp]
    return L


def at(i):
    return BASE + i * GAP


def call_window(L, four):
    d = oxd.make_window_decode_desc(3, 8, 2, 32, "HND", 50, 20, 64, 4)
    tail = (at(5), at(6), at(7), -0.5, at(8), at(9), at(10), 256, None)
    if four:
        cache = oxd.KvPools(at(1), at(2), at(3), at(4))
        return L.oxd_quant_window_decode(ctypes.addressof(d), at(0), ctypes.addressof(cache.struct), *tail)
    return L.oxd_window_decode(ctypes.addressof(d), at(0), at(1), at(2), *tail)


def call_tables(L, missing=(), **kw):
    d = oxd.make_build_tables_desc(**{**dict(batch=5, page_size=8, row_pages=30, num_pages=200, num_indices=150,
                                             num_tokens=40, num_free=100, window=64, sinks=4), **kw})
    a = [None if i in missing else at(i) for i in range(17)]
    return L.oxd_build_tables(ctypes.addressof(d), *a, 256, None)


WINDOW = {False: [0, 1, 2, 5, 6, 7, 8, 9, 10], True: list(range(11))}


def on(fake, arrays, other=None, kind=DEVICE):
    fake.fake_reset(0)
    for i in arrays:
        fake.fake_allocate(at(i), 1 << 24, 1 if i == other else 0, kind)


@pytest.mark.parametrize("four", [False, True])
def test_window_decodes_take_arrays_of_the_current_device_alone(fake, four):
    on(fake, WINDOW[four])
    assert call_window(fake, four) == 0 and fake.fake_launches() == 1
    assert [fake.fake_window_shape(i) for i in range(9)] == [3, 8, 2, 4, 5, 1, 20, 64, 4]
    assert fake.fake_window_scale_sign() == -1
    for i in WINDOW[four]:
        on(fake, WINDOW[four], other=i)
        assert call_window(fake, four) == 1 and fake.fake_launches() == 0, i
        on(fake, WINDOW[four], other=i, kind=MANAGED)
        assert call_window(fake, four) == 0, i


def test_tables_take_arrays_of_the_current_device_alone(fake):
    every = list(range(17))
    on(fake, every)
    assert call_tables(fake) == 0 and fake.fake_launches() == 1
    assert [fake.fake_tables_shape(i) for i in range(10)] == [5, 3, 30, 150, 40, 100, 64, 4, 1, 1]
    for i in every:
        on(fake, every, other=i)
        assert call_tables(fake) == 1 and fake.fake_launches() == 0, i
        on(fake, every, other=i, kind=MANAGED)
        assert call_tables(fake) == 0, i


def test_tables_without_maps_write_none(fake):
    on(fake, list(range(17)))
    assert call_tables(fake, missing=(1, 12, 13, 14, 15), num_tokens=0) == 0
    assert [fake.fake_tables_shape(i) for i in (8, 9)] == [0, 0]
    assert call_tables(fake, missing=(8, 15)) == 0  # no reference counts, no slots
    assert [fake.fake_tables_shape(i) for i in (8, 9)] == [1, 0]
    assert call_tables(fake, missing=(5, 6, 7), num_free=0) == 0
    assert fake.fake_launches() == 3
