"""CPU checks of the decode-step operators: sizes, refusals before any launch, and
the pins of their oracle."""
import ctypes

import numpy as np
import pytest
import torch

from dequant_gemv_packed_b200 import build as B
from dequant_gemv_packed_b200 import qlin as Q
from oracle import decode_oracle as D
from oracle import qlin_oracle as O


@pytest.fixture(scope="module")
def lib():
    B.build()
    return Q.lib()


P = ctypes.c_void_p(0x10000)    # aligned stand-ins, never dereferenced
P2 = ctypes.c_void_p(0x20000)
P3 = ctypes.c_void_p(0x30000)
ODD = ctypes.c_void_p(0x10008)  # 8-byte aligned
BYTE = ctypes.c_void_p(0x10002)


def desc(pages=4, page=16, heads=2, dim=128, kb=8, vb=8):
    return Q.KVDesc(pages, page, heads, dim, kb, vb)


@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (8, 4), (4, 8), (16, 16)])
def test_cache_bytes(lib, dim, kb, vb):
    d = desc(7, 48, 3, dim, kb, vb)
    assert Q.qlin_kv_cache_bytes(d) == D.Cache(7, 48, 3, dim, kb, vb).bytes.size


BAD = [(dict(pages=0), -3), (dict(page=0), -3), (dict(page=8), -3), (dict(page=24), -3), (dict(heads=0), -3),
       (dict(dim=64), -3), (dict(dim=384), -3), (dict(pages=1 << 27, page=16), -3), (dict(kb=3), -2), (dict(kb=6), -2),
       (dict(kb=16), -2), (dict(vb=16), -2), (dict(kb=16, vb=8), -2), (dict(kb=0), -2)]


@pytest.mark.parametrize("bad,status", BAD)
def test_descriptor_refusals(lib, bad, status):
    d = desc(**bad)
    assert Q.qlin_kv_cache_bytes(d) == 0
    assert Q.qlin_attn_workspace_bytes(d, 4, 1, 1) == 0
    assert lib.qlin_kv_write(d.ref(), P, P, P, 1024, 1024, P, 1, None, None) == status
    assert lib.qlin_kv_read(d.ref(), P, P, 1, None, P, P2, None) == status
    assert lib.qlin_attn_decode(d.ref(), P, P, 4096, 4, P, 1, P, 1, None, 1.0, P2, P3, 1 << 40, None) == status


def test_cache_refusals(lib):
    d = desc()
    r = d.ref()
    assert lib.qlin_kv_write(None, P, P, P, 256, 256, P, 1, None, None) == -1
    for bad in range(4):
        a = [None if i == bad else P for i in range(4)]
        assert lib.qlin_kv_write(r, a[0], a[1], a[2], 256, 256, a[3], 1, None, None) == -1
        a = [None if i == bad else (P, P, P, P2)[i] for i in range(4)]
        assert lib.qlin_kv_read(r, a[0], a[1], 1, None, a[2], a[3], None) == -1
    assert lib.qlin_kv_read(r, P, P, 1, None, P2, P2, None) == -1  # k and v in one place
    for t, ks, vs in ((0, 256, 256), (-1, 256, 256), (1, 255, 256), (1, 256, 248), (1, 260, 256), (1, 256, 0)):
        assert lib.qlin_kv_write(r, P, P, P, ks, vs, P, t, None, None) == -3
    assert lib.qlin_kv_read(r, P, P, 0, None, P, P2, None) == -3
    for i in range(5):
        a = [ODD if i == j else P for j in range(3)]
        slots, signs = BYTE if i == 3 else P, ODD if i == 4 else P
        assert lib.qlin_kv_write(r, a[0], a[1], a[2], 256, 256, slots, 1, signs, None) == -4
        assert lib.qlin_kv_read(r, a[0], slots, 1, signs, a[1], P2 if i != 2 else ODD, None) == -4


def test_attention_refusals(lib):
    d = desc()
    r = d.ref()

    def call(cache=P, q=P, qs=512, hq=4, table=P, pages=2, lens=P, b=1, signs=None, scale=1.0, out=P2, ws=P3,
             wl=1 << 40, ref=r):
        return lib.qlin_attn_decode(ref, cache, q, qs, hq, table, pages, lens, b, signs, scale, out, ws, wl, None)

    assert call(ref=None) == -1
    for name in ("cache", "q", "table", "lens", "out"):
        assert call(**{name: None}) == -1, name
    assert call(out=P) == -1  # in place
    assert call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    for bad in (dict(hq=3), dict(hq=0), dict(b=0), dict(pages=0), dict(qs=504), dict(qs=516), dict(b=-1),
                dict(pages=1 << 27), dict(b=1 << 20, pages=1 << 10)):
        assert call(**bad) == -3, bad
    for name in ("cache", "q", "out", "signs"):
        assert call(**{name: ODD}) == -4, name
    for name in ("table", "lens"):
        assert call(**{name: BYTE}) == -4, name
    big = Q.qlin_attn_workspace_bytes(d, 4, 1, 4096)
    if big:
        assert call(pages=4096, ws=None) == -6
        assert call(pages=4096, wl=big - 1) == -6
        assert call(pages=4096, ws=ODD) == -4


def test_norm_refusals(lib):
    def call(x=P, res=None, w=P, eps=1e-6, y=P2, ro=None, m=1, k=128):
        return lib.qlin_rmsnorm(x, res, w, eps, y, ro, m, k, None)

    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(res=P3), dict(ro=P3), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(y=P), dict(res=P2, ro=P3), dict(res=P3, ro=P2),
                dict(res=P3, ro=P)):
        assert call(**bad) == -1, bad
    for bad in (dict(m=0), dict(k=0), dict(k=4), dict(k=100), dict(k=65544), dict(m=-3)):
        assert call(**bad) == -3, bad
    for bad in (dict(x=ODD), dict(w=ODD), dict(y=ODD), dict(res=ODD, ro=P3), dict(res=P3, ro=ODD)):
        assert call(**bad) == -4, bad


def test_binding_takes_cuda_tensors_only(lib):
    d = desc()
    cache = torch.zeros(Q.qlin_kv_cache_bytes(d), dtype=torch.uint8)
    k = torch.zeros(1, 2, 128, dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    for f in (lambda: Q.qlin_kv_write(d, cache, k, k, i), lambda: Q.qlin_kv_read(d, cache, i),
              lambda: Q.qlin_attn_decode(d, cache, k, i.view(1, 1), i), lambda: Q.qlin_rmsnorm(k[0], k[0, 0], 1e-6)):
        with pytest.raises(TypeError, match="CUDA tensor"):
            f()


# ------------------------------------------------------------------ oracle pins

def test_oracle_rotation_matches_the_layers_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 256)).astype(np.float16)
    sb = rng.integers(0, 2 ** 32, 8, dtype=np.uint64).astype(np.uint32)
    ref = O.rht64(x, sb)
    assert np.abs(D.rotate32(x, sb) - ref).max() <= 2.0 ** -20 * np.abs(x).max() * 128
    assert np.abs(x.astype(np.float64) @ D.rotation64(sb, 256).T - ref).max() < 1e-12
    back = D.unrotate32(D.rotate32(x, sb), sb)
    assert np.abs(back - x).max() < 1e-5


@pytest.mark.parametrize("bits", [4, 8])
def test_oracle_grid(bits):
    """Zero is on the grid, every value is within half a step (and the zero's rounding) of its
    own, and the extremes are reached: hand cases and a sweep down to fp16 subnormals."""
    qmax = 2 ** bits - 1
    v = np.zeros((1, 128), np.float32)
    q, s, z = D.quantise32(v, bits)
    assert s[0, 0] == 1 and z[0, 0] == 0 and not q.any()
    v[0] = np.arange(128) % (qmax + 1)  # 0..qmax: step 1 exactly
    v[0, 0] = 0
    v[0, 1] = qmax
    q, s, z = D.quantise32(v, bits)
    assert s[0, 0] == 1 and z[0, 0] == 0 and (q == v).all()
    rng = np.random.default_rng(1)
    for mag in (3e4, 100.0, 1.0, 1e-3, 1e-5, 3e-7):
        for shift in (0.0, 3.0, -50.0):  # groups far from zero too
            v = ((rng.standard_normal((40, 128)) + shift) * mag).clip(-65504, 65504).astype(np.float16).astype(np.float32)
            q, s, z = D.quantise32(v, bits)
            assert np.isfinite(s).all() and (z >= 0).all() and (z <= qmax).all()
            got = s.astype(np.float64) * (q.astype(np.float64) - z.astype(np.float64))
            # half a step, and fp32 rounding of v / s + z (up to qmax + 1)
            assert (np.abs(got - v) <= s.astype(np.float64) * (0.5 + 2.0 ** -14 * 8) + 1e-12).all()


def test_oracle_non_finite_group_reads_as_nan():
    v = np.ones((3, 128), np.float32)
    v[0, 5], v[1, 5], v[2, 5] = np.nan, np.inf, -np.inf
    q, s, z = D.quantise32(v, 8)
    assert np.isnan(z).all() and (s == 1).all()


def test_oracle_cache_layout_by_hand():
    c = D.Cache(2, 16, 2, 128, 4, 8, fill=0xAA)
    k = np.zeros((1, 2, 128), np.float16)
    v = np.zeros((1, 2, 128), np.float16)
    k[0, 1, :16] = np.arange(16)
    v[0, 1, 3] = 255
    c.write(k, v, [16 + 5])
    blk = c.bytes[1, 1]
    assert blk.size == 16 * (64 + 128 + 8)
    assert blk[5 * 64:5 * 64 + 8].tolist() == [0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE]
    assert blk[16 * 64 + 5 * 128 + 3] == 255
    par = blk[16 * 192 + 5 * 8:16 * 192 + 5 * 8 + 8].view(np.float16)
    assert par[0] == 1 and par[1] == 0 and par[2] == 1 and par[3] == 0
    assert (c.bytes[0] == 0xAA).all() and (blk[6 * 64:16 * 64] == 0xAA).all()


def test_oracle_attention_special_cases():
    """Equal keys give the mean of the values; one dominating key gives its value; a
    page outside the pool and a length of zero leave tokens out."""
    rng = np.random.default_rng(2)
    c = D.Cache(3, 16, 1, 128, 16, 16)
    v = rng.standard_normal((48, 1, 128)).astype(np.float16)
    k = np.ones((48, 1, 128), np.float16)
    k[37] = 3
    c.write(k, v, np.arange(48))
    q = np.ones((2, 1, 128), np.float16)
    out, _ = D.attention64(c, q, np.array([[0, 1], [0, 1]]), [20, 0], 1.0)
    assert np.abs(out[0, 0] - v[:20, 0].astype(np.float64).mean(0)).max() < 1e-12 and not out[1].any()
    out, _ = D.attention64(c, q[:1], np.array([[2]]), [16], 1.0)
    assert np.abs(out[0, 0] - v[37, 0]).max() < 1e-12
    out, _ = D.attention64(c, q[:1], np.array([[7, 0]]), [32], 1.0)
    assert np.abs(out[0, 0] - v[:16, 0].astype(np.float64).mean(0)).max() < 1e-12


def test_oracle_rotated_attention_equals_plain():
    """Rotating q, k and the values and rotating back changes nothing but rounding."""
    rng = np.random.default_rng(3)
    sb = rng.integers(0, 2 ** 32, 4, dtype=np.uint64).astype(np.uint32)
    k, v = (rng.standard_normal((32, 2, 128)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((1, 4, 128)).astype(np.float16)
    outs = []
    for s in (None, sb):
        c = D.Cache(2, 16, 2, 128, 16, 16)
        c.write(k, v, np.arange(32), s)
        outs.append(D.attention64(c, q, np.array([[0, 1]]), [32], 0.1, s)[0])
    assert np.abs(outs[0] - outs[1]).max() < 5e-3
