"""The decode-step calls at the ends of what they accept: pages of many gigabytes, and values that are not finite."""
import numpy as np
import pytest
import torch

from dequant_gemv_packed_b200 import qlin as Q
from oracle import decode_oracle as D

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dequant_gemv_packed_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    Q.lib()
    yield
    torch.cuda.empty_cache()  # pools of gigabytes


@pytest.fixture(autouse=True)
def _clean_error_word():
    Q.qlin_device_error()
    yield
    assert Q.qlin_device_error() == 0


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


@pytest.mark.parametrize("kb,vb,size,log", [(8, 8, 1.0, 22), (4, 4, 1.0, 26), (4, 4, 60000.0, 22), (8, 4, 60000.0, 22)])
def test_millions_of_cleared_slots(kb, vb, size, log):
    """A sequence of 2^22 or 2^26 cleared slots (a page that its table names over and over) and 16 written tokens with
    scores near 12, so that both have a part of the weights; values of ordinary size, and with scales of 2^13.

    A cleared slot stands for k = v = 0: a weight of e^0 in the denominator.  The bound: a score's fp32 error
    twice, the denominator's fp32 sum in chains of at most 2^log / (148 * 4 * 8) additions and 400 joins, the exponentials,
    each as a share of sum p |v|; and the output's own rounding."""
    rng = np.random.default_rng(kb + vb)
    page, cleared = 256, 1 << log
    base = np.sign(rng.standard_normal(128))
    k = (base + 0.1 * rng.standard_normal((16, 1, 128))).astype(np.float16)
    v = (size * rng.uniform(-1, 1, (16, 1, 128))).astype(np.float16)
    q = (1.05 * base + 0.05 * rng.standard_normal((1, 4, 128))).astype(np.float16)
    c = D.Cache(2, page, 1, 128, kb, vb)
    c.write(k, v, range(page, page + 16))
    d = Q.KVDesc(2, page, 1, 128, kb, vb)
    table = np.zeros((1, cleared // page + 1), np.int32)
    table[0, -1] = 1
    got = Q.qlin_attn_decode(d, dev(c.bytes.reshape(-1)), dev(q), dev(table), dev(np.array([cleared + 16], np.int32)))
    kk, vv = (c.values(i, range(page, page + 16))[:, 0].astype(np.float64) for i in (0, 1))
    scale = float(np.float32(128 ** -0.5))
    par = c.par[1, 0, :16, 0].astype(np.float64)
    mag = np.abs(kk) + 2 * np.abs(par[:, :1] * par[:, 1:2])
    for h in range(4):
        x = q[0, h].astype(np.float64)
        s = scale * (kk @ x)
        assert 10 < s.min() and s.max() < 14
        e = scale * (mag @ np.abs(x)) * (128 + 64) * 2.0 ** -24 + 2.0 ** -22 * scale * np.abs(x).max() * np.abs(kk).sum(1)
        p = np.exp(s) / (cleared + np.exp(s).sum())
        ref = p @ vv
        chain = (cleared / (148 * 4 * 8) + 400) * 2.0 ** -24
        tol = (p * (2 * e + chain + 2.0 ** -18)) @ np.abs(vv) + np.abs(ref) * 2.0 ** -11 + 2.0 ** -25
        err = np.abs(got[0, h].double().cpu().numpy() - ref)
        assert (err <= tol).all(), f"worst error / bound {float((err / tol).max()):.3f}"


@pytest.mark.parametrize("page,dim,kb,vb", [(9_000_000, 256, 8, 8), (17_000_000, 256, 8, 4), (2 ** 27 + 16, 128, 4, 4)])
def test_attention_far_inside_one_page(page, dim, kb, vb):
    """The last tokens of a page of 4.8 to 18.3 GB: offsets from a tile's keys to its values and parameters pass 2^31,
    and the tile's place in the page 2^23 (2^27 tokens).

    The pool is cleared but for the last 40 tokens.  A cleared slot has a score of 0, those tokens have scores above
    50, so the others' share of the weights is below 2^28 e^-50 < 1e-13."""
    rng = np.random.default_rng(dim + kb)
    n = 40
    base = np.sign(rng.standard_normal(dim))
    k = (base + 0.3 * rng.standard_normal((n, 1, dim))).astype(np.float16)
    v = rng.standard_normal((n, 1, dim)).astype(np.float16)
    q = (6 * base + rng.standard_normal((1, 4, dim))).astype(np.float16)
    d = Q.KVDesc(1, page, 1, dim, kb, vb)
    pool = torch.zeros(Q.qlin_kv_cache_bytes(d), dtype=torch.uint8, device=DEV)
    slots = np.arange(page - n, page, dtype=np.int32)
    Q.qlin_kv_write(d, pool, dev(k), dev(v), dev(slots))
    small = D.Cache(3, 16, 1, dim, kb, vb)
    small.write(k, v, range(n))
    for got, ref in zip(Q.qlin_kv_read(d, pool, dev(slots)), small.read(range(n))):
        assert np.array_equal(got.cpu().numpy(), ref)
    scale = float(np.float32(dim ** -0.5))
    assert (small.values(0, range(n))[:, 0].astype(np.float64) @ q[0].T.astype(np.float64) * scale).min() > 50
    got = Q.qlin_attn_decode(d, pool, dev(q), dev(np.zeros((1, 1), np.int32)), dev(np.array([page], np.int32)))
    ref, tol = D.attention64(small, q, np.arange(3)[None], [n], scale)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"worst error / bound {float((err / tol).max()):.3f}"


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8), (4, 4)])
def test_infinities_and_nan(kb, vb, group, rotate):
    """One infinity or NaN in a query, a key or a value, in a sequence that is read whole and in one that is cut and
    joined: NaN in the outputs that it has a part in, and the same bits in all others; past the length it has
    no effect."""
    rng = np.random.default_rng(kb + group)
    heads, dim, page = 2, 256, 16
    lens = [40, 700]
    slots = [np.arange(48), np.arange(48, 48 + 704)]
    table = np.zeros((2, 44), np.int32)
    table[0, :3], table[1] = np.arange(3), np.arange(3, 47)
    sb = dev(rng.integers(0, 2 ** 32, dim // 32, dtype=np.uint64).astype(np.uint32).view(np.int32)) if rotate else None
    d = Q.KVDesc(47, page, heads, dim, kb, vb)
    at = dev(np.concatenate(slots).astype(np.int32))
    k, v = (rng.standard_normal((752, heads, dim)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((2, heads * group, dim)).astype(np.float16)

    def run(q, k, v):
        pool = torch.zeros(Q.qlin_kv_cache_bytes(d), dtype=torch.uint8, device=DEV)
        Q.qlin_kv_write(d, pool, dev(k), dev(v), at, sign_bits=sb)
        return Q.qlin_attn_decode(d, pool, dev(q), dev(table), dev(np.array(lens, np.int32)), sign_bits=sb).cpu().numpy()

    clean = run(q, k, v)
    assert np.isfinite(clean).all()
    for bad in (np.inf, -np.inf, np.nan):
        for b in (0, 1):
            for what in ("q", "k", "v", "past"):
                x = {"q": q.copy(), "k": k.copy(), "v": v.copy()}
                where = np.zeros(clean.shape, bool)
                if what == "q":
                    x["q"][b, group + 1, 130] = bad
                    where[b, group + 1] = True
                elif what == "past":
                    x["k"][slots[b][lens[b]], 1, 130] = x["v"][slots[b][lens[b]], 1, 130] = bad
                else:
                    x[what][slots[b][lens[b] // 2], 1, 130] = bad
                    where[b, group:, slice(0, 256) if what == "k" else 130 if kb == 16 and not rotate else slice(128, 256)] = True
                got = run(x["q"], x["k"], x["v"])
                assert np.array_equal(np.isnan(got), where), (what, bad, b)
                assert np.array_equal(got[~where], clean[~where]), (what, bad, b)


@pytest.mark.parametrize("scale", [2.0 ** 40, -2.0 ** 40])
@pytest.mark.parametrize("kb,vb", [(16, 16), (8, 8), (4, 4)])
def test_largest_scale(kb, vb, scale):
    """The token of the largest score has all the weight, whatever the scores' size and sign.  The bound: the output's
    rounding, and 2^-18 of s (q + |z|), at most twice the largest value, for the few fp32 steps of the quotient."""
    rng = np.random.default_rng(kb)
    c = D.Cache(2, 16, 1, 256, kb, vb)
    c.write(rng.standard_normal((20, 1, 256)).astype(np.float16), rng.standard_normal((20, 1, 256)).astype(np.float16),
            range(20))
    q = (1000 * rng.standard_normal((1, 4, 256))).astype(np.float16)
    d = Q.KVDesc(2, 16, 1, 256, kb, vb)
    got = Q.qlin_attn_decode(d, dev(c.bytes.reshape(-1)), dev(q), dev(np.array([[0, 1]], np.int32)),
                             dev(np.array([20], np.int32)), scale=scale).cpu().numpy()
    s = np.sign(scale) * (c.values(0, range(20))[:, 0].astype(np.float64) @ q[0].T.astype(np.float64))
    v = c.values(1, range(20))[:, 0].astype(np.float64)
    for h in range(4):
        ref = v[s[:, h].argmax()]
        assert (np.abs(got[0, h] - ref) <= np.abs(ref) * (2.0 ** -11 + 2.0 ** -17) + np.abs(v).max() * 2.0 ** -17).all()
