"""CPU checks of what the decode-step calls accept: refusals before any launch, and sizes."""
import ctypes

import pytest

from dequant_gemv_packed_b200 import build as B
from dequant_gemv_packed_b200 import qlin as Q


@pytest.fixture(scope="module")
def lib():
    B.build()
    return Q.lib()


P = ctypes.c_void_p(0x10000)  # aligned stand-ins, never dereferenced
P2 = ctypes.c_void_p(0x20000)
P3 = ctypes.c_void_p(0x30000)
ODD = ctypes.c_void_p(0x10008)  # 8-byte aligned


@pytest.mark.parametrize("scale", [2.0 ** 41, -2.0 ** 41, 1e30, -3e38, float("inf"), float("-inf"), float("nan")])
def test_attention_refuses_scales_past_its_range(lib, scale):
    d = Q.KVDesc(4, 16, 2, 128, 8, 8)
    assert lib.qlin_attn_decode(d.ref(), P, P, 512, 4, P, 2, P, 1, None, scale, P2, P3, 1 << 40, None) == -1
