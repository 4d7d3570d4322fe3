"""The host side of the appends and the page copies over a stand-in for the device
(``tests/fakes/quant_host.cpp``): which device a call's tensors may be on, and the frequencies of the
rotation."""
import ctypes
import importlib
import os
import subprocess
from decimal import Decimal, localcontext

import pytest

import paged_kv_decode_attn_gb300 as oxd

B = importlib.import_module("paged_kv_decode_attn_gb300.build")  # (the package's name is the function)
HERE = os.path.dirname(os.path.abspath(__file__))
BASE, GAP = 1 << 40, 1 << 32
DEVICE, MANAGED = 2, 3  # cudaMemoryType


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("fakes") / "quant_host.so")
    subprocess.run([B.nvcc(), "-std=c++17", "-O1", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC",
                    "-Xlinker", "-Bsymbolic", "-I", os.path.join(B.ROOT, "include"), "-I", B.CSRC,
                    os.path.join(HERE, "fakes", "quant_host.cpp"),
                    os.path.join(B.CSRC, "oxd_quant_host.cpp"), "-o", so], check=True)
    L = ctypes.CDLL(so)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    L.fake_allocate.argtypes = [vp, sz, ctypes.c_int, ctypes.c_int]
    L.fake_turns.restype = ctypes.POINTER(ctypes.c_float)
    L.oxd_rope_axes_append.argtypes = [vp] * 14 + [sz, vp]
    L.oxd_quant_rope_append.argtypes = [vp] * 13 + [sz, vp]
    L.oxd_copy_pages.argtypes = [vp] * 7 + [sz, vp]
    return L


def at(i):
    return BASE + i * GAP


def call_append(L, four):
    d = oxd.make_axes_append_desc(10, 3, 8, 2, 16, "NHD", 50, 20, sections=(16, 24, 24))
    head = [ctypes.addressof(d)] + [at(i) for i in range(10)]
    if four:
        cache = oxd.KvPools(at(10), at(11), at(12), at(13))
        return L.oxd_quant_rope_append(*head, ctypes.addressof(cache.struct), at(14), 256, None)
    return L.oxd_rope_axes_append(*head, at(10), at(11), at(14), 256, None)


def call_copy(L, four):
    src = oxd.KvPools(at(0), at(1))
    dst = oxd.KvPools(at(2), at(3), at(4), at(5)) if four else oxd.KvPools(at(2), at(3))
    d = oxd.make_copy_pages_desc(4, 2, 16, "bf16", "NHD", 30, "e2m1" if four else "bf16", "NHD", 20)
    return L.oxd_copy_pages(ctypes.addressof(d), ctypes.addressof(src.struct),
                            ctypes.addressof(dst.struct), at(6), at(7), at(8), at(9), 256, None)


APPEND = {False: [*range(12), 14], True: list(range(15))}
COPY = {False: [0, 1, 2, 3, 6, 7, 8, 9], True: list(range(10))}


@pytest.mark.parametrize("call,used", [(call_append, APPEND), (call_copy, COPY)])
@pytest.mark.parametrize("four", [False, True])
def test_every_tensor_must_be_on_the_current_device(fake, call, used, four):
    for wrong in [None, *used[four]]:
        fake.fake_reset(1)
        for i in used[four]:
            fake.fake_allocate(at(i), GAP, 0 if i == wrong else 1, DEVICE)
        assert call(fake, four) == (0 if wrong is None else 1), wrong
        assert fake.fake_launches() == (1 if wrong is None else 0)


@pytest.mark.parametrize("call,used", [(call_append, APPEND), (call_copy, COPY)])
def test_managed_memory_and_memory_of_no_device_is_taken(fake, call, used):
    fake.fake_reset(1)
    for i in used[True][1:]:
        fake.fake_allocate(at(i), GAP, 0, MANAGED)
    assert call(fake, True) == 0 and fake.fake_launches() == 1


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 5e6, 1e9, 1.5, 1.0000001, 12345.678])
def test_frequencies_hold_up_to_the_farthest_position(fake, theta):
    """Three floats hold 72 bits: within 2^-70 of the frequency, a turn's angle at position 2^24 is
    good to 2^-43. (A double's 2^-53 would leave 2^-29, where the rotation is good to 2^-32.)"""
    d = oxd.make_axes_append_desc(10, 3, 8, 2, 16, "NHD", 50, 20, rope_theta=theta, sections=(16, 24, 24))
    fake.fake_reset(0)
    assert fake.oxd_rope_axes_append(ctypes.addressof(d), *[at(i) for i in range(12)], at(14), 256,
                                     None) == 0
    got = fake.fake_turns()
    with localcontext() as c:
        c.prec = 50
        for i in range(64):
            want = (-Decimal(theta).ln() * i / 64).exp() / (2 * PI)
            have = sum((Decimal(got[4 * i + j]) for j in range(3)), Decimal(0))
            assert abs(have - want) <= want * Decimal(2) ** -70, i
