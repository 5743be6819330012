"""CPU checks of what the decode-step calls accept: refusals before any launch, and sizes."""
import ctypes

import pytest
import torch

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


def attend(lib, d, pages, ws, size, group=2):
    return lib.qlin_attn_decode(d.ref(), P, P, 512 * group, 2 * group, P, pages, P, 1, None, 1.0, P2, ws, size, None)


@pytest.mark.parametrize("dim", [128, 256])
def test_attention_workspace(lib, dim):
    """None for tables of up to 512 tokens, whose sequences are never cut; beyond, two pieces of each query of a block
    (dim sums, maximum and denominator) for at least 148 CTAs, refused if missing, short or misaligned."""
    d = Q.KVDesc(4, 16, 2, dim, 8, 8)
    assert Q.qlin_attn_workspace_bytes(d, 4, 1, 32) == 0
    sizes = {}
    for group, block in ((1, 1), (2, 2), (4, 4), (8, 8), (9, 5), (16, 8)):
        size = sizes[group] = Q.qlin_attn_workspace_bytes(d, 2 * group, 1, 33)
        assert size >= 148 * 2 * block * (dim + 2) * 4
        assert Q.qlin_attn_workspace_bytes(d, 2 * group, 7, 4096) == size
        for pages in (33, 4096):
            assert attend(lib, d, pages, None, size, group) == -6
            assert attend(lib, d, pages, None, 0, group) == -6
            assert attend(lib, d, pages, P3, size - 1, group) == -6
            assert attend(lib, d, pages, ODD, size, group) == -4
    assert sizes[1] < sizes[2] < sizes[4] < sizes[8] == sizes[16]
    assert sizes[4] < sizes[9] < sizes[8]


def test_cache_calls_refuse_more_groups_than_they_count(lib):
    """2^31 - 2^20 groups a side and more; one less passes the check and would be launched."""
    for heads, dim in ((2, 128), (1, 256), (8, 256), (1 << 20, 128)):
        d = Q.KVDesc(1, 16, heads, dim, 4, 4)
        groups = heads * dim // 128
        for t in (-(-(2 ** 31 - 2 ** 20) // groups), 2 ** 31 // groups - 1, 2 ** 31 - 1):
            assert lib.qlin_kv_write(d.ref(), P, P, P, heads * dim, heads * dim, P, t, None, None) == -3
            assert lib.qlin_kv_read(d.ref(), P, P, t, None, P2, P3, None) == -3


def test_cache_refuses_more_heads_than_it_counts(lib):
    """A token of 2^31 values and more; up to there the pool's bytes are those of the layout, counted without a limit."""
    for dim in (128, 256):
        for heads, ok in ((2 ** 31 // dim - 1, True), (2 ** 31 // dim, False), (1 << 28, False), (2 ** 31 - 1, False)):
            for pages, page in ((1, 16), (2 ** 27 - 1, 16), (1, 2 ** 31 - 16)):
                for kb, vb, row in ((4, 4, dim + dim // 16), (16, 16, 4 * dim)):
                    d = Q.KVDesc(pages, page, heads, dim, kb, vb)
                    assert Q.qlin_kv_cache_bytes(d) == (pages * page * heads * row if ok else 0)
                    if not ok:
                        width = heads * dim
                        assert lib.qlin_kv_write(d.ref(), P, P, P, width, width, P, 1, None, None) == -3
                        assert lib.qlin_kv_read(d.ref(), P, P, 1, None, P2, P3, None) == -3


def test_stream_of_another_device_is_refused():
    """It was made current with its device, after which the call ran on the buffers' device in its default stream."""
    class OnDevice0(torch.Tensor):
        is_cuda = property(lambda self: True)
        device = property(lambda self: torch.device("cuda", 0))

        def get_device(self):
            return 0

    class Stream1:
        cuda_stream, device = 0, torch.device("cuda", 1)

    t = torch.zeros(1, 2, 128).as_subclass(OnDevice0)
    d = Q.KVDesc(4, 16, 2, 128, 8, 8)
    for call in (lambda s: Q.qlin_kv_write(d, t, t, t, t, stream=s), lambda s: Q.qlin_kv_read(d, t, t, stream=s),
                 lambda s: Q.qlin_attn_decode(d, t, t, t, t, stream=s), lambda s: Q.qlin_rmsnorm(t, t, 1e-6, stream=s)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call(Stream1())


def test_norm_refuses_to_write_over_its_weight(lib):
    assert lib.qlin_rmsnorm(P, None, P2, 1e-6, P2, None, 1, 128, None) == -1
    assert lib.qlin_rmsnorm(P, P3, P2, 1e-6, ctypes.c_void_p(0x40000), P2, 1, 128, None) == -1
