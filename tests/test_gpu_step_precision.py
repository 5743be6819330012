"""Decode attention where the precision of what enters its products shows: against the
definition in 64 bits, with bounds that count the roundings of fp32 and fp16."""
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


@pytest.fixture(autouse=True)
def _clean_error_word():
    Q.qlin_device_error()
    yield
    assert Q.qlin_device_error() == 0


def attend(c, q, table, lens, scale):
    d = Q.KVDesc(c.bytes.shape[0], c.page, c.heads, c.dim, *c.bits)
    pool = torch.from_numpy(c.bytes.reshape(-1).copy()).to(DEV)
    args = [torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
            for x in (q, table.astype(np.int32), np.asarray(lens, np.int32))]
    return Q.qlin_attn_decode(d, pool, *args, scale=scale).double().cpu().numpy()


def check(c, q, table, lens):
    scale = float(np.float32(c.dim ** -0.5))
    got = attend(c, q, table, lens, scale)
    ref, tol = D.attention64(c, q, table, lens, scale)
    err = np.abs(got - ref)
    assert (err <= tol).all(), f"worst error / bound {float((err / tol).max()):.3f}, worst error {err.max():.3g}"
    return ref


# Keys that are not negative have a grid that starts at zero (z = 0), so a zero key is exact and adds nothing to
# a score in any precision.  What is left of the score's error is the oracle's: fp32 sums, and the rounding of
# the query's small channels to 2^-22 of its largest.

@pytest.mark.parametrize("dim,group", [(128, 4), (128, 8), (256, 1), (256, 6)])
@pytest.mark.parametrize("kb,vb", [(8, 8), (4, 4), (8, 4), (4, 8)])
def test_small_query_channels_beside_a_large_one(kb, vb, dim, group):
    """A query channel 2^15 times the others, where every key is zero: the others make the scores and tell the
    tokens apart."""
    rng = np.random.default_rng(kb * 10 + vb + dim + group)
    heads, n = 2, 40
    c = D.Cache(3, 16, heads, dim, kb, vb)
    k = np.floor(rng.random((n, heads, dim)) * 2) * (15 * rng.permutation(n))[:, None, None]
    k[:, :, 7::128] = 0
    c.write(k.astype(np.float16), rng.standard_normal((n, heads, dim)).astype(np.float16), range(n))
    assert not c.values(0, range(n))[:, :, 7::128].any()
    q = (0.0015 + 0.002 * rng.random((1, heads * group, dim))).astype(np.float16)
    q[0, :, 7::128] = 100
    ref = check(c, q, np.arange(3)[None], [n])
    equal = c.values(1, range(n)).mean(0).repeat(group, 0)  # what equal weights would give
    assert np.abs(ref[0] - equal).max() > 0.5


@pytest.mark.parametrize("kb,vb", [(8, 8), (4, 4)])
@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("ratio", [2 ** 3, 2 ** 8, 2 ** 11, 2 ** 14])
def test_query_of_two_sizes(kb, vb, group, ratio):
    """Half of the query's channels larger than the others by a power of two, where the keys are zero; two tokens,
    so that no error of a score is averaged away."""
    rng = np.random.default_rng(ratio + group)
    c = D.Cache(1, 16, 1, 128, kb, vb)
    large = rng.permutation(128)[:64]
    k = 30 * np.abs(rng.standard_normal((2, 1, 128)))
    k[:, :, large] = 0
    c.write(k.astype(np.float16), rng.standard_normal((2, 1, 128)).astype(np.float16), range(2))
    q = 0.05 * np.abs(rng.standard_normal((1, group, 128)))
    q[:, :, large] = 0.06 * ratio
    check(c, q.astype(np.float16), np.zeros((1, 1), int), [2])


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (8, 4), (4, 8), (16, 16)])
@pytest.mark.parametrize("dim,group", [(128, 4), (128, 5), (128, 8), (256, 7), (128, 12)])
def test_weights_of_values_that_cancel(kb, vb, dim, group):
    """Three tokens whose large values cancel in the sum, so that a rounding of their weights is not hidden by the
    output's: a weight of 11 bits would be 2^-12 of the values away, one of 22 bits 2^-23."""
    rng = np.random.default_rng(kb + vb + dim + group)
    c = D.Cache(1, 16, 1, dim, kb, vb)
    k = 0.1 * rng.standard_normal((3, 1, dim))
    v = np.repeat(np.array([1000.0, -800.0, -100.0]).reshape(3, 1, 1), dim, 2) * (1 + 0.1 * rng.random((1, 1, dim)))
    c.write(k.astype(np.float16), v.astype(np.float16), range(3))
    q = rng.standard_normal((1, group, dim)).astype(np.float16)
    ref = check(c, q, np.zeros((1, 1), int), [3])
    assert np.abs(ref).max() < 200


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (8, 4), (4, 8)])
@pytest.mark.parametrize("dim,group", [(128, 4), (128, 5), (128, 8), (256, 8), (256, 12)])
def test_small_values_beside_a_large_one_elsewhere(kb, vb, dim, group):
    """One token whose values are 60,000 in half of a group's dimensions and zero in the others, among tokens with
    values near 0.001: in those others the output is theirs alone, their scales 2^-23 of the large token's."""
    rng = np.random.default_rng(kb + vb + dim + group)
    c = D.Cache(2, 16, 1, dim, kb, vb)
    v = 0.001 * rng.standard_normal((20, 1, dim))
    v[7] = np.where(np.arange(dim) % 128 < 64, 60000.0, 0.0)  # its grid starts at zero: a zero is exact
    k = 0.3 * rng.standard_normal((20, 1, dim))
    c.write(k.astype(np.float16), v.astype(np.float16), range(20))
    q = rng.standard_normal((1, group, dim)).astype(np.float16)
    ref = check(c, q, np.arange(2)[None], [20])
    assert np.abs(ref[..., np.arange(dim) % 128 >= 64]).max() < 0.002
