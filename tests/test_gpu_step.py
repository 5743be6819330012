"""GPU parity of the decode-step operators: the paged quantised key/value cache,
attention of one new token over it, and the residual norm, against
oracle/decode_oracle.py.  Stored bytes and values read back match bit for bit;
attention is held to the per-element bound that the oracle derives, the norm to
its own (in the test)."""
import numpy as np
import pytest
import torch

from dequant_gemv_packed_b200 import qlin as Q
from dequant_gemv_packed_b200 import workloads as W
from oracle import decode_oracle as D
from oracle import qlin_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDTHS = [(4, 4), (8, 8), (8, 4), (4, 8), (16, 16)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from dequant_gemv_packed_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    Q.lib()
    yield
    torch.cuda.empty_cache()  # some cases fill gigabytes, and some fill them with NaN


@pytest.fixture(autouse=True)
def _clean_error_word():
    Q.qlin_device_error()
    yield
    assert Q.qlin_device_error() == 0


def dev(x, dtype=None):
    if x is None:
        return None
    x = np.ascontiguousarray(x)
    x = x.view(np.int32) if x.dtype == np.uint32 else x
    return torch.from_numpy(x).to(DEV) if dtype is None else torch.from_numpy(x).to(DEV, dtype)


def signs(rng, dim, rotate=True):
    return rng.integers(0, 2 ** 32, dim // 32, dtype=np.uint64).astype(np.uint32) if rotate else None


def vectors(rng, t, heads, dim):
    x = rng.standard_normal((t, heads, dim)) * np.where(rng.random(dim) < 0.05, 8.0, 1.0)
    return x.astype(np.float16)


def pool_of(c):
    return dev(c.bytes.reshape(-1).copy())


def kv_desc(c):
    return Q.KVDesc(c.bytes.shape[0], c.page, c.heads, c.dim, *c.bits)


def filled(rng, pages, page, heads, dim, kb, vb, sb):
    """A cache whose every slot is written, by the oracle."""
    c = D.Cache(pages, page, heads, dim, kb, vb)
    n = pages * page
    c.write(vectors(rng, n, heads, dim), (0.5 * rng.standard_normal((n, heads, dim))).astype(np.float16), range(n), sb)
    return c


# ------------------------------------------------------------- write and read

@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("kb,vb", WIDTHS)
def test_write_and_read_bits(kb, vb, dim, rotate):
    """Bytes of written slots, untouched bytes elsewhere, skipped tokens, and the values read
    back: shuffled slots, token rows that are columns of a wider matrix."""
    rng = np.random.default_rng(kb * 100 + vb + dim)
    heads, page, pages, t = 3, 48, 3, 37
    sb = signs(rng, dim, rotate)
    c = D.Cache(pages, page, heads, dim, kb, vb, fill=0x5A)
    slots = rng.permutation(pages * page)[:t].astype(np.int32)
    slots[[3, 20]] = -1, -7
    k, v = vectors(rng, t, heads, dim), vectors(rng, t, heads, dim)
    v[5] = 0  # an empty group
    k[6] = k[6] * np.float16(2e-6)  # subnormal scales
    v[7] = np.abs(v[7]) + np.float16(100)  # far from zero
    d, pool = kv_desc(c), pool_of(c)
    wide = torch.zeros(t, 2 * heads * dim + 8, dtype=torch.float16, device=DEV)
    wide[:, 8:8 + heads * dim] = dev(k).flatten(1)
    wide[:, 8 + heads * dim:] = dev(v).flatten(1)
    Q.qlin_kv_write(d, pool, wide[:, 8:8 + heads * dim].unflatten(1, (heads, dim)),
                    wide[:, 8 + heads * dim:].unflatten(1, (heads, dim)), dev(slots), sign_bits=dev(sb))
    c.write(k, v, slots, sb)
    got = pool.cpu().numpy().reshape(c.bytes.shape)
    assert np.array_equal(got, c.bytes), int((got != c.bytes).sum())
    again = np.concatenate([slots, slots[:9], [-1]]).astype(np.int32)  # a slot may be read twice
    gk, gv = Q.qlin_kv_read(d, pool, dev(again), sign_bits=dev(sb))
    for g, r in zip((gk, gv), c.read(again, sb)):
        assert np.array_equal(g.cpu().numpy().view(np.uint16) & 0x7FFF, r.view(np.uint16) & 0x7FFF)
        assert np.array_equal(g.cpu().numpy(), r)


@pytest.mark.parametrize("kb,vb", WIDTHS)
def test_one_token_one_head(kb, vb):
    rng = np.random.default_rng(kb + vb)
    c = D.Cache(1, 16, 1, 128, kb, vb)
    d, pool = kv_desc(c), pool_of(c)
    k, v, sb = vectors(rng, 1, 1, 128), vectors(rng, 1, 1, 128), signs(rng, 128)
    slots = np.array([15], np.int32)
    Q.qlin_kv_write(d, pool, dev(k), dev(v), dev(slots), sign_bits=dev(sb))
    c.write(k, v, slots, sb)
    assert np.array_equal(pool.cpu().numpy().reshape(c.bytes.shape), c.bytes)


def test_slot_past_the_pool_is_skipped_and_reported():
    rng = np.random.default_rng(5)
    c = D.Cache(2, 16, 2, 128, 8, 8, fill=1)
    d, pool = kv_desc(c), pool_of(c)
    k = vectors(rng, 3, 2, 128)
    slots = np.array([32, 4, 2 ** 31 - 1], np.int32)
    Q.qlin_kv_write(d, pool, dev(k), dev(k), dev(slots))
    c.write(k, k, slots)
    assert np.array_equal(pool.cpu().numpy().reshape(c.bytes.shape), c.bytes)
    assert Q.qlin_device_error() == 1 << 24
    gk, _ = Q.qlin_kv_read(d, pool, dev(slots))
    assert np.array_equal(gk.cpu().numpy(), c.read(slots)[0])
    assert Q.qlin_device_error() == 1 << 24


@pytest.mark.parametrize("kb", [4, 8])
def test_non_finite_group_reads_as_nan(kb):
    rng = np.random.default_rng(6)
    k = vectors(rng, 4, 1, 256)
    k[0, 0, 3], k[1, 0, 130], k[2, 0, 7] = np.nan, np.inf, -np.inf
    c = D.Cache(1, 16, 1, 256, kb, 8)
    d, pool = kv_desc(c), pool_of(c)
    slots = np.arange(4, dtype=np.int32)
    Q.qlin_kv_write(d, pool, dev(k), dev(k), dev(slots))
    got = [x.cpu().numpy() for x in Q.qlin_kv_read(d, pool, dev(slots))]
    c.write(k, k, slots)
    for g, r in zip(got, c.read(slots)):
        assert np.array_equal(g, r, equal_nan=True)
        assert np.isnan(g[0, 0, :128]).all() and np.isfinite(g[0, 0, 128:]).all() and np.isnan(g[1, 0, 128:]).all()


def test_extreme_range_rotated():
    """The largest fp16 values in one direction: the 4-bit scale is cut at 65504, nothing overflows."""
    rng = np.random.default_rng(7)
    sb = signs(rng, 128)
    k = (65504 * D.sign_vector(sb, 128)).astype(np.float16).reshape(1, 1, 128)
    c = D.Cache(1, 16, 1, 128, 4, 8)
    d, pool = kv_desc(c), pool_of(c)
    Q.qlin_kv_write(d, pool, dev(k), dev(-k), dev(np.zeros(1, np.int32)), sign_bits=dev(sb))
    c.write(k, -k, [0], sb)
    assert np.array_equal(pool.cpu().numpy().reshape(c.bytes.shape), c.bytes)


# ------------------------------------------------------------------ attention

def run_attention(c, q, table, lens, scale=None, sb=None, pool=None, **kw):
    return Q.qlin_attn_decode(kv_desc(c), pool_of(c) if pool is None else pool, q if torch.is_tensor(q) else dev(q),
                              dev(table.astype(np.int32)), dev(np.asarray(lens, np.int32)), scale=scale,
                              sign_bits=dev(sb), **kw)


def check_attention(got, c, q, table, lens, scale=None, sb=None, what=""):
    scale = float(np.float32(c.dim ** -0.5 if scale is None else scale))
    ref, tol = D.attention64(c, q, table, lens, scale, sb)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.isfinite(err).all(), what
    assert (err <= tol).all(), f"{what}: worst error / bound {float((err / tol).max()):.3f}"


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("dim,heads,group", [(128, 2, 4), (128, 1, 1), (256, 2, 5), (128, 3, 8), (128, 1, 12)])
@pytest.mark.parametrize("kb,vb", WIDTHS)
def test_attention(kb, vb, dim, heads, group, rotate):
    """Every width, group size and rotation over lengths of none, one, a page's end and its
    neighbours, and several pages; shuffled pages; table entries past a length are junk."""
    rng = np.random.default_rng(kb * 7 + vb + dim + group)
    page, width = 32, 8
    lens = [0, 1, 31, 32, 33, 250, 17]
    sb = signs(rng, dim, rotate)
    c = filled(rng, len(lens) * width, page, heads, dim, kb, vb, sb)
    table = rng.permutation(len(lens) * width).reshape(len(lens), width)
    for b, n in enumerate(lens):
        table[b, -(-n // page):] = (-1, 2 ** 31 - 1, -2 ** 31)[b % 3]
    q = (1.5 * rng.standard_normal((len(lens), heads * group, dim))).astype(np.float16)
    got = run_attention(c, q, table, lens, sb=sb)
    check_attention(got, c, q, table, lens, sb=sb, what=f"{kb}/{vb} {dim} group {group}")
    assert not got[0].any()


@pytest.mark.parametrize("page,kb,vb", [(16, 4, 4), (256, 8, 4), (48, 16, 16), (64, 8, 8)])
def test_attention_long(page, kb, vb):
    """One long sequence (split over CTAs and joined) next to short and empty ones."""
    rng = np.random.default_rng(page)
    n = 3001
    width = -(-n // page)
    sb = signs(rng, 128)
    c = filled(rng, width + 9, page, 1, 128, kb, vb, sb)
    table = np.full((4, width), -5)
    order = rng.permutation(width + 9)
    table[1] = order[:width]
    table[0, 0], table[3, 0] = order[width], order[width + 1]
    lens = [page - 1, n, 0, 1]
    q = (2 * rng.standard_normal((4, 4, 128))).astype(np.float16)
    check_attention(run_attention(c, q, table, lens, sb=sb), c, q, table, lens, sb=sb, what=f"page {page}")


def test_attention_peaked_and_flat():
    """One token that takes all the weight (first, last, in the middle), scores that are all
    equal, a scale of zero and a negative one."""
    rng = np.random.default_rng(11)
    c = filled(rng, 40, 16, 1, 128, 8, 8, None)
    table = rng.permutation(40).reshape(1, 40)
    q = np.zeros((1, 2, 128), np.float16)
    for at in (0, 333, 639):
        slot = table[0, at // 16] * 16 + at % 16
        q[0, 0] = (10 * c.values(0, [slot])[0, 0]).astype(np.float16)
        check_attention(run_attention(c, q, table, [640], 1.0), c, q, table, [640], 1.0, what=f"peak {at}")
    q[0, 1] = 1
    for scale in (0.0, -0.7, 1e-30):
        check_attention(run_attention(c, q, table, [640], scale), c, q, table, [640], scale, what=f"scale {scale}")


def test_attention_growing_scores():
    """Scores that grow along the sequence by far more than the exponent range of fp16: the running
    maximum moves over and over; and the same falling."""
    rng = np.random.default_rng(12)
    for sign in (1, -1):
        c = D.Cache(40, 16, 1, 128, 16, 16)
        k = np.zeros((640, 1, 128), np.float16)
        k[:, 0, 0] = sign * np.arange(640)
        v = rng.standard_normal((640, 1, 128)).astype(np.float16)
        c.write(k, v, range(640))
        q = np.zeros((1, 2, 128), np.float16)
        q[0, 0, 0], q[0, 1, 0] = 1, 0.01
        table = np.arange(40).reshape(1, 40)
        check_attention(run_attention(c, q, table, [640], 1.0), c, q, table, [640], 1.0, what=f"sign {sign}")


@pytest.mark.parametrize("kb,vb", [(8, 8), (4, 4)])
def test_attention_value_scales_apart(kb, vb):
    """Values of very different sizes: scales 2^20 apart, the large ones on unlikely tokens."""
    rng = np.random.default_rng(13)
    c = D.Cache(8, 16, 1, 128, kb, vb)
    k = np.zeros((128, 1, 128), np.float16)
    v = rng.standard_normal((128, 1, 128)) * 1e-3
    k[::7, 0, 0], v[::7] = -60, v[::7] * 2.0 ** 20
    k[::5, 0, 1] = 3
    v = v.clip(-60000, 60000).astype(np.float16)
    c.write(k, v, range(128))
    q = np.zeros((1, 4, 128), np.float16)
    q[0, :, 0], q[0, :, 1] = (0.05, 0.1, 0.25, 0.3), 0.5
    table = np.arange(8).reshape(1, 8)
    check_attention(run_attention(c, q, table, [128], 1.0), c, q, table, [128], 1.0, what="scales apart")


@pytest.mark.parametrize("kb,vb,fill", [(8, 8, 0xFF), (4, 4, 0x7C), (16, 16, 0xFF), (16, 16, 0x7C), (8, 4, 0x7E)])
def test_masked_places_may_hold_anything(kb, vb, fill):
    """Slots past the length hold NaN and infinity patterns, in the last page's tail too."""
    rng = np.random.default_rng(14)
    c = D.Cache(6, 32, 2, 128, kb, vb, fill=fill)
    n = 71
    c.write(vectors(rng, n, 2, 128), vectors(rng, n, 2, 128), range(n))
    q = rng.standard_normal((2, 8, 128)).astype(np.float16)
    table = np.array([[0, 1, 2, 3], [1, 5, 4, 3]])
    for lens in ([71, 5], [65, 32], [1, 0]):
        check_attention(run_attention(c, q, table, lens), c, q, table, lens, what=f"{lens}")


@pytest.mark.parametrize("kb,vb", [(8, 8), (4, 4), (16, 16)])
def test_cleared_slots_inside_a_length_are_zero_vectors(kb, vb):
    """A slot of a zero-filled pool that was never written stands for k = v = 0: a score of 0, and a
    share of the weights; alone in the sequence, in the first tile, and among written tokens."""
    rng = np.random.default_rng(24)
    c = D.Cache(6, 16, 1, 128, kb, vb)
    n = 40
    c.write(vectors(rng, n, 1, 128), vectors(rng, n, 1, 128), range(20, 20 + n))
    q = (0.2 * rng.standard_normal((3, 4, 128))).astype(np.float16)
    table, lens = np.array([[0, 1, 2, 3], [5, 5, 5, 5], [4, 1, 2, 5]]), [50, 33, 64]
    got = run_attention(c, q, table, lens)
    check_attention(got, c, q, table, lens)
    assert not got[1].any()


def test_page_outside_the_pool_is_masked_and_reported():
    rng = np.random.default_rng(15)
    c = filled(rng, 4, 16, 1, 128, 8, 8, None)
    q = rng.standard_normal((3, 4, 128)).astype(np.float16)
    table = np.array([[0, 4, 1], [-1, 2, 3], [-3, 99, 2 ** 31 - 1]])
    lens = [48, 40, 48]
    got = run_attention(c, q, table, lens)
    assert Q.qlin_device_error() == 2 << 24
    check_attention(got, c, q, table, lens)
    assert not got[2].any()


def test_length_beyond_the_table_is_cut_and_reported():
    rng = np.random.default_rng(16)
    c = filled(rng, 4, 16, 1, 128, 8, 8, None)
    q = rng.standard_normal((2, 4, 128)).astype(np.float16)
    table = np.array([[0, 1], [2, 3]])
    got = run_attention(c, q, table, [1000, -4])
    assert Q.qlin_device_error() == 4 << 24
    check_attention(got, c, q, table, [32, 0])


def test_nan_query_gives_nan_for_its_head_only():
    rng = np.random.default_rng(17)
    c = filled(rng, 4, 16, 1, 128, 8, 8, None)
    q = rng.standard_normal((2, 4, 128)).astype(np.float16)
    table, lens = np.array([[0, 1], [2, 3]]), [32, 20]
    ref = run_attention(c, q, table, lens)
    bad = q.copy()
    bad[0, 2, 9] = np.nan
    got = run_attention(c, bad, table, lens)
    assert torch.isnan(got[0, 2]).all()
    keep = [(0, 0), (0, 1), (0, 3), (1, 0), (1, 1), (1, 2), (1, 3)]
    for b, h in keep:
        assert torch.equal(got[b, h], ref[b, h])


def test_pool_past_32_bits():
    """Offsets past 2^32 bytes: the last pages of a pool of 4.6 GB."""
    rng = np.random.default_rng(18)
    c = filled(rng, 3, 256, 8, 128, 16, 16, None)
    block = c.bytes.size // 3
    pages = 4_600_000_000 // block
    pool = torch.empty(pages * block, dtype=torch.uint8, device=DEV)
    pool[-3 * block:] = pool_of(c)
    d = Q.KVDesc(pages, 256, 8, 128, 16, 16)
    q = rng.standard_normal((1, 16, 128)).astype(np.float16)
    small = np.array([[2, 0, 1]])
    got = Q.qlin_attn_decode(d, pool, dev(q), dev((small + pages - 3).astype(np.int32)), dev(np.array([700], np.int32)))
    check_attention(got, c, q, small, [700])
    slots = np.array([5, 700, 300], np.int32)
    gk, gv = Q.qlin_kv_read(d, pool, dev(slots + (pages - 3) * 256))
    for g, r in zip((gk, gv), c.read(slots)):
        assert np.array_equal(g.cpu().numpy(), r)
    Q.qlin_kv_write(d, pool, gk * 2, gv, dev(slots + (pages - 3) * 256))
    assert torch.equal(Q.qlin_kv_read(d, pool, dev(slots + (pages - 3) * 256))[0], gk * 2)


def test_queries_may_be_columns_and_outputs_given():
    rng = np.random.default_rng(19)
    c = filled(rng, 6, 16, 2, 128, 8, 8, None)
    table, lens = np.array([[0, 1, 2], [3, 4, 5]]), [48, 33]
    wide = torch.randn(2, 12 * 128, device=DEV).half()
    q = wide[:, :8 * 128].unflatten(1, (8, 128))
    out = torch.full((2, 8, 128), float("nan"), dtype=torch.float16, device=DEV)
    got = run_attention(c, q, table, lens, out=out)
    assert got is out
    check_attention(out, c, q.cpu().numpy(), table, lens)


def long_case(seed, lens=(2500, 77, 1300), kb=8, vb=4):
    rng = np.random.default_rng(seed)
    width = -(-max(lens) // 32)
    sb = signs(rng, 128)
    c = filled(rng, len(lens) * width, 32, 2, 128, kb, vb, sb)
    table = rng.permutation(len(lens) * width).reshape(len(lens), width)
    q = rng.standard_normal((len(lens), 8, 128)).astype(np.float16)
    return c, q, table, list(lens), sb


def test_attention_is_deterministic():
    c, q, table, lens, sb = long_case(20)
    pool = pool_of(c)
    ref = run_attention(c, q, table, lens, sb=sb, pool=pool)
    for _ in range(5):
        assert torch.equal(run_attention(c, q, table, lens, sb=sb, pool=pool), ref)


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with its own workspace and output, repeated."""
    cases = [long_case(21), long_case(22, (600, 2100, 5, 900))]
    args = []
    for c, q, table, lens, sb in cases:
        ref = run_attention(c, q, table, lens, sb=sb)
        args.append((kv_desc(c), pool_of(c), dev(q), dev(table.astype(np.int32)), dev(np.asarray(lens, np.int32)),
                     dev(sb), ref))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for turn in range(20):
        for i, (d, pool, q, t, n, sb, _) in enumerate(args):
            s = streams[i] if turn % 2 else streams[i].cuda_stream  # a stream object, or its handle
            outs[i].append(Q.qlin_attn_decode(d, pool, q, t, n, sign_bits=sb, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, args[i][6]) for o in outs[i])


def test_captured_step_follows_new_inputs():
    """A captured write + attention replayed with new tokens, lengths and queries, against the
    calls made outside the graph; then a second graph of the same step beside it."""
    c, q, table, lens, sb = long_case(23)
    d, pool = kv_desc(c), pool_of(c)
    rng = np.random.default_rng(1)
    tq, tt, tl, ts = dev(q), dev(table.astype(np.int32)), dev(np.asarray(lens, np.int32)), dev(sb)
    k, v = dev(vectors(rng, 3, 2, 128)), dev(vectors(rng, 3, 2, 128))
    slots = dev(np.array([table[b, (n - 1) // 32] * 32 + (n - 1) % 32 for b, n in enumerate(lens)], np.int32))

    def step():
        Q.qlin_kv_write(d, pool, k, v, slots, sign_bits=ts)
        return Q.qlin_attn_decode(d, pool, tq, tt, tl, sign_bits=ts)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for new in ([2500, 77, 1300], [1, 0, 1299], [33, 2000, 2500]):
        tl.copy_(dev(np.asarray(new, np.int32)))
        tq.normal_()
        k.normal_()
        slots.copy_(dev(np.array([table[b, max(n - 1, 0) // 32] * 32 + max(n - 1, 0) % 32 if n else -1
                                  for b, n in enumerate(new)], np.int32)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        ref = step()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
        held = D.Cache(*[c.bytes.shape[0], 32, 2, 128, *c.bits])
        held.bytes[:] = pool.cpu().numpy().reshape(c.bytes.shape)
        check_attention(ref, held, tq.cpu().numpy(), table, new, sb=sb, what=str(new))


def test_many_sequences():
    """More sequences than a block keeps lengths of (512), empty ones among them, in small pages."""
    rng = np.random.default_rng(31)
    B = 700
    lens = rng.integers(0, 40, B)
    lens[[0, 5, 511, 512, 699]] = 0, 37, 16, 39, 0
    c = filled(rng, 60, 16, 1, 128, 8, 4, None)
    table = rng.integers(0, 60, (B, 3))  # sequences may share pages
    q = rng.standard_normal((B, 2, 128)).astype(np.float16)
    check_attention(run_attention(c, q, table, lens), c, q, table, lens)


@pytest.mark.parametrize("dim,heads,group,kb,vb", [(128, 5, 3, 4, 8), (256, 1, 16, 8, 8), (128, 2, 16, 16, 16),
                                                   (256, 3, 3, 16, 16), (128, 1, 7, 8, 8)])
def test_long_among_short(dim, heads, group, kb, vb):
    """Two long sequences cut over many teams, between scores of short ones of every tile count."""
    rng = np.random.default_rng(heads * group)
    lens = [3, 1900, 16, 17, 0, 1, 1000, 512, 513, 528] + list(range(1, 120, 7))
    width = 60
    c = filled(rng, 90, 32, heads, dim, kb, vb, None)
    table = rng.integers(0, 90, (len(lens), width))
    q = (1.5 * rng.standard_normal((len(lens), heads * group, dim))).astype(np.float16)
    check_attention(run_attention(c, q, table, lens), c, q, table, lens)


@pytest.mark.parametrize("n", [496, 511, 512, 513, 529])
def test_the_border_of_cutting(n):
    """Tables and lengths on both sides of the longest item that is not cut (512 tokens)."""
    rng = np.random.default_rng(n)
    c = filled(rng, 34, 16, 1, 128, 8, 8, None)
    q = rng.standard_normal((2, 4, 128)).astype(np.float16)
    for width in (32, 34):
        table = rng.permutation(34)[None, :width].repeat(2, 0)
        lens = [min(n, width * 16), 20]
        check_attention(run_attention(c, q, table, lens), c, q, table, lens, what=f"{n} in {width} pages")


@pytest.mark.parametrize("kb", [4, 8])
def test_query_with_an_outlying_channel(kb):
    """A query channel 2,000 times the others: their 16-bit integers are few, within the bound."""
    rng = np.random.default_rng(32)
    c = filled(rng, 8, 16, 1, 128, kb, 8, None)
    q = (0.05 * rng.standard_normal((1, 4, 128))).astype(np.float16)
    q[0, :, 7] = 100
    table = np.arange(8)[None]
    check_attention(run_attention(c, q, table, [128]), c, q, table, [128])


@pytest.mark.parametrize("dim,group,kb,vb", [(128, 3, 8, 4), (256, 2, 4, 8), (128, 12, 8, 8)])
def test_one_workspace_through_calls_of_every_size(dim, group, kb, vb):
    """1 to 66 (head, query block) pairs, on both sides of each count at which pieces are joined another
    way; cut and whole items and empty sequences by turns, in the same workspace, full of ones at first."""
    rng = np.random.default_rng(dim + group)
    c1, c2 = (filled(rng, 60, 32, h, dim, kb, vb, None) for h in (1, 2))
    blocks = -(-group // 8)
    ws = None
    for c in (c2, c1):
        pool = pool_of(c)
        for items in (66, 65, 64, 33, 32, 9, 8, 2, 1):
            B = items // (c.heads * blocks)
            if B * c.heads * blocks != items:
                continue
            table = rng.integers(0, 60, (B, 60))
            q = rng.standard_normal((B, c.heads * group, dim)).astype(np.float16)
            if ws is None:
                ws = torch.full((Q.qlin_attn_workspace_bytes(kv_desc(c), c.heads * group, B, 60),), 0xFF,
                                dtype=torch.uint8, device=DEV)
            for long in (1900, 40, 1000, 0):  # cut, whole, cut elsewhere, none
                lens = rng.integers(0, 60, B)
                lens[B // 2] = long
                lens[B - 1 if B > 2 else 0] = long // 2 if B > 2 else long
                got = run_attention(c, q, table, lens, pool=pool, workspace=ws)
                check_attention(got, c, q, table, lens, what=f"{items} of {long}")


def test_workspace_contents_do_not_matter():
    c, q, table, lens, sb = long_case(33)
    ref = run_attention(c, q, table, lens, sb=sb)
    size = Q.qlin_attn_workspace_bytes(kv_desc(c), 8, 3, table.shape[1])
    assert size > 0
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    pool = pool_of(c)
    for fill in (0xFF, 0x01, None):
        if fill is not None:
            ws.fill_(fill)
        assert torch.equal(run_attention(c, q, table, lens, sb=sb, pool=pool, workspace=ws), ref)
    with pytest.raises(Q.QlinError, match="WORKSPACE"):
        run_attention(c, q, table, lens, sb=sb, pool=pool, workspace=ws[:size - 16])


def test_captured_behind_copies_memsets_and_joins():
    """The calls wait for whatever precedes them: a host copy, a memset, and another stream's work
    that is joined, eagerly and in a graph; and what follows them waits for them."""
    c, q, table, lens, sb = long_case(36, (700, 90))
    d, pool = kv_desc(c), pool_of(c)
    tt, ts = dev(table.astype(np.int32)), dev(sb)
    host_n, tl = torch.tensor(lens, dtype=torch.int32).pin_memory(), torch.zeros(2, dtype=torch.int32, device=DEV)
    src, tq = dev(q), torch.zeros(2, 8, 128, dtype=torch.float16, device=DEV)
    w = torch.ones(1024, dtype=torch.float16, device=DEV)
    acc = torch.zeros(2, 1024, dtype=torch.float16, device=DEV)
    other = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            big = src.float().repeat(400, 1, 1)  # work that takes a while
            tq.copy_(big[:2])
        tl.copy_(host_n, non_blocking=True)
        here.wait_stream(other)
        o = Q.qlin_attn_decode(d, pool, tq, tt, tl, sign_bits=ts)
        acc.zero_()
        y, r = Q.qlin_rmsnorm(o.flatten(1), w, 1e-6, residual=acc)
        other.wait_stream(here)
        with torch.cuda.stream(other):
            z = r.clone()
        here.wait_stream(other)
        tq.zero_()
        tl.zero_()
        return o, y, z

    torch.cuda.synchronize()
    ref = [x.clone() for x in step()]
    torch.cuda.synchronize()
    check_attention(ref[0], c, q, table, lens, sb=sb)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(step(), ref))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for _ in range(20):
        for x in outs:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


@pytest.mark.parametrize("overlap", [False, True])
def test_beside_overlapping_layers(overlap):
    """norm -> GEMV -> norm -> GEMV -> attention -> GEMV chains with and without the GEMVs' overlap give
    the same bits, in a graph too."""
    rng = np.random.default_rng(37)
    c = filled(rng, 40, 16, 2, 128, 8, 8, None)
    d, pool = kv_desc(c), pool_of(c)
    table, n = dev(np.arange(40, dtype=np.int32).reshape(1, 40)), dev(np.array([630], np.int32))
    la, lb = linear(1024, 512, 4, 3), linear(512, 1024, 6, 4)
    x = dev(rng.standard_normal((1, 512)).astype(np.float16))
    w = dev((1 + 0.1 * rng.standard_normal(512)).astype(np.float16))

    def chain():
        h, r = x, x
        for _ in range(3):
            h, r = Q.qlin_rmsnorm(h, w, 1e-6, residual=r)
            q = Q.qlin_gemv(la[0], la[1], la[2].scales, la[2].zeros, la[3], h)
            o = Q.qlin_attn_decode(d, pool, q.view(1, 8, 128), table, n)
            h = Q.qlin_gemv(lb[0], lb[1], lb[2].scales, lb[2].zeros, lb[3], o.view(1, 1024))
        return h, r

    ref = [t.clone() for t in chain()]
    torch.cuda.synchronize()
    before = Q.qlin_set_overlap(overlap)
    try:
        for _ in range(30):
            assert all(torch.equal(a, b) for a, b in zip(chain(), ref))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = chain()
        for _ in range(10):
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    finally:
        Q.qlin_set_overlap(before)


def test_first_call_inside_a_capture():
    """A process whose first calls are captured: nothing is set up outside the graph."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = """
import torch
from dequant_gemv_packed_b200 import qlin as Q
d = Q.KVDesc(80, 16, 1, 128, 8, 4)
pool = torch.zeros(Q.qlin_kv_cache_bytes(d), dtype=torch.uint8, device="cuda")
k = torch.randn(900, 1, 128, device="cuda").half()
slots = torch.arange(900, device="cuda", dtype=torch.int32)
q = torch.randn(1, 4, 128, device="cuda").half()
table = torch.arange(80, device="cuda", dtype=torch.int32).view(1, 80)
n = torch.tensor([900], device="cuda", dtype=torch.int32)
w = torch.ones(512, device="cuda").half()
def step():
    Q.qlin_kv_write(d, pool, k, k, slots)
    o = Q.qlin_attn_decode(d, pool, q, table, n)
    return o, Q.qlin_rmsnorm(o.view(1, 512), w, 1e-6), Q.qlin_kv_read(d, pool, slots)[1]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    outs = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, step())) and outs[0].abs().max() > 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_binding_refuses_wrong_tensors():
    """Shapes, types and layouts that the binding checks before a call."""
    rng = np.random.default_rng(34)
    c = filled(rng, 4, 16, 2, 128, 8, 8, None)
    d, pool = kv_desc(c), pool_of(c)
    q = torch.zeros(2, 4, 128, device=DEV).half()
    table, lens = torch.zeros(2, 2, device=DEV, dtype=torch.int32), torch.zeros(2, device=DEV, dtype=torch.int32)
    k, slots = torch.zeros(3, 2, 128, device=DEV).half(), torch.zeros(3, device=DEV, dtype=torch.int32)
    sb = torch.zeros(8, device=DEV, dtype=torch.int32)
    bad = [(TypeError, lambda: Q.qlin_attn_decode(d, pool, q.float(), table, lens)),
           (TypeError, lambda: Q.qlin_attn_decode(d, pool, q, table.long(), lens)),
           (TypeError, lambda: Q.qlin_attn_decode(d, pool, q, table, lens.cpu())),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool, q, table[:1], lens)),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool, q, table, lens[:1])),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool, q[0], table, lens)),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool, q.transpose(1, 2).contiguous().transpose(1, 2), table, lens)),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool, q, table, lens, out=q[:1].clone())),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool, q, table, lens, sign_bits=sb)),
           (ValueError, lambda: Q.qlin_attn_decode(d, pool[:-16], q, table, lens)),
           (Q.QlinError, lambda: Q.qlin_attn_decode(d, pool, q[:, :3], table, lens)),
           (Q.QlinError, lambda: Q.qlin_attn_decode(d, pool, q, table, lens, out=q)),
           (Q.QlinError, lambda: Q.qlin_attn_decode(d, pool, q[:0], table[:0], lens[:0])),
           (TypeError, lambda: Q.qlin_kv_write(d, pool, k.float(), k, slots)),
           (ValueError, lambda: Q.qlin_kv_write(d, pool, k[:, :1], k, slots)),
           (ValueError, lambda: Q.qlin_kv_write(d, pool, k, k[:2], slots)),
           (ValueError, lambda: Q.qlin_kv_write(d, pool, k, k, slots[:2])),
           (Q.QlinError, lambda: Q.qlin_kv_write(d, pool, k[:1].expand(3, 2, 128), k, slots)),
           (TypeError, lambda: Q.qlin_kv_read(d, pool, slots.float())),
           (ValueError, lambda: Q.qlin_kv_read(d, pool, slots, k=k[:2])),
           (Q.QlinError, lambda: Q.qlin_kv_read(d, pool, slots, k=k, v=k)),
           (ValueError, lambda: Q.qlin_rmsnorm(k.view(3, 256), k.view(3, 256)[0, :128], 1e-6)),
           (ValueError, lambda: Q.qlin_rmsnorm(k.view(3, 256), k.view(3, 256)[0], 1e-6, residual_out=k.view(3, 256).clone())),
           (Q.QlinError, lambda: Q.qlin_rmsnorm(k.view(3, 256), k.view(3, 256)[0].clone(), -1.0))]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_write_and_read_many_tokens():
    """More units than the grid has lanes for: every block walks on; odd heads and two groups a head."""
    rng = np.random.default_rng(35)
    for heads, dim, t in ((3, 128, 4300), (1, 256, 5000)):
        c = D.Cache(-(-t // 48) + 1, 48, heads, dim, 8, 4)
        slots = rng.permutation(c.bytes.shape[0] * 48)[:t].astype(np.int32)
        slots[::97] = -1
        sb = signs(rng, dim)
        k, v = vectors(rng, t, heads, dim), vectors(rng, t, heads, dim)
        d, pool = kv_desc(c), pool_of(c)
        Q.qlin_kv_write(d, pool, dev(k), dev(v), dev(slots), sign_bits=dev(sb))
        c.write(k, v, slots, sb)
        assert np.array_equal(pool.cpu().numpy().reshape(c.bytes.shape), c.bytes)
        for g, r in zip(Q.qlin_kv_read(d, pool, dev(slots), sign_bits=dev(sb)), c.read(slots, sb)):
            assert np.array_equal(g.cpu().numpy(), r)


@pytest.mark.parametrize("dim,rotate", [(128, True), (256, False)])
@pytest.mark.parametrize("kb,vb", WIDTHS)
def test_write_and_read_a_prompt(kb, vb, dim, rotate):
    """So many groups (from 18,944 a side) that the kernels take four lanes a group."""
    rng = np.random.default_rng(kb + 3 * vb + dim)
    heads = 8 if dim == 128 else 5
    t = 2400 if dim == 128 else 1911
    c = D.Cache(t // 32 + 2, 32, heads, dim, kb, vb)
    slots = rng.permutation(c.bytes.shape[0] * 32)[:t].astype(np.int32)
    slots[5::89] = -2
    sb = signs(rng, dim, rotate)
    k, v = vectors(rng, t, heads, dim), vectors(rng, t, heads, dim)
    k[7, 0, 3], v[8, 1, 5], k[9] = np.nan, -np.inf, 0
    d, pool = kv_desc(c), pool_of(c)
    Q.qlin_kv_write(d, pool, dev(k), dev(v), dev(slots), sign_bits=dev(sb))
    c.write(k, v, slots, sb)
    got, ref = pool.cpu().numpy().reshape(c.bytes.shape), c.bytes
    if kb == 16:  # a NaN's payload is not part of the format
        got, ref = got.view(np.float16), ref.view(np.float16)
        assert np.array_equal(got, ref, equal_nan=True)
    else:
        assert np.array_equal(got, ref)
    for g, r in zip(Q.qlin_kv_read(d, pool, dev(slots), sign_bits=dev(sb)), c.read(slots, sb)):
        assert np.array_equal(g.cpu().numpy(), r, equal_nan=True)


# ----------------------------------------------------------------------- norm

def check_norm(x, w, eps, res=None, **kw):
    """One fp16 rounding (2^-11, 2^-25 for subnormals), and fp32: the mean's sum has chains of at most
    512 additions (2^-24 each, halved by the square root), quotient, root and products 8 roundings."""
    ref, h = D.rmsnorm64(x, w, eps, res)
    got = Q.qlin_rmsnorm(dev(x), dev(w), eps, residual=dev(res), **kw)
    y, r = got if res is not None else (got, None)
    if res is not None:
        assert np.array_equal(r.cpu().numpy(), h)
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err <= np.abs(ref) * (2.0 ** -11 + (256 + 8) * 2.0 ** -24) + 2.0 ** -25).all()
    return y


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("M,K", [(1, 8), (3, 136), (5, 1000), (1, 1024), (2, 1032), (1, 2560), (7, 2560), (300, 2568),
                                 (2, 8192), (3, 9728), (2, 16392), (2, 40000), (2, 65536), (1000, 128),
                                 (70001, 64)])
def test_norm(M, K, res):
    rng = np.random.default_rng(M + K)
    x = (rng.standard_normal((M, K)) * np.exp(rng.standard_normal((M, 1)))).astype(np.float16)
    w = (1 + 0.3 * rng.standard_normal(K)).astype(np.float16)
    check_norm(x, w, 1e-6, (3 * rng.standard_normal((M, K))).astype(np.float16) if res else None)


def test_norm_extremes():
    """A row of zeros (eps alone), the largest values (their squares' sum is far past fp16), subnormals."""
    x = np.zeros((4, 512), np.float16)
    x[1] = 65504
    x[2] = 2.0 ** -24
    x[3, 100] = -300
    w = np.ones(512, np.float16)
    y = check_norm(x, w, 1e-6)
    assert not y[0].any()
    assert not torch.isnan(Q.qlin_rmsnorm(dev(x[1:]), dev(w), 0.0)).any()


def test_norm_residual_in_place():
    rng = np.random.default_rng(3)
    x, r = rng.standard_normal((9, 2560)).astype(np.float16), rng.standard_normal((9, 2560)).astype(np.float16)
    w = np.ones(2560, np.float16)
    stream = dev(r)
    y, out = Q.qlin_rmsnorm(dev(x), dev(w), 1e-5, residual=stream, residual_out=stream)
    assert out is stream
    ref_y, ref_h = Q.qlin_rmsnorm(dev(x), dev(w), 1e-5, residual=dev(r))
    assert torch.equal(y, ref_y) and torch.equal(stream, ref_h)


# ------------------------------------------------------------ a run of them all

def linear(n, k, bits, index):
    w = W.draw_weight(n, k, bits, seed=3, index=index).to(DEV)
    a = W.draw_activation(1, k, seed=3, index=index).to(DEV)
    d = Q.Desc.of(w)
    return d, Q.qlin_pack(d, w.codes), w, a.sign_bits


@pytest.mark.parametrize("kb,vb,rotate", [(8, 8, True), (4, 4, True), (16, 16, False)])
def test_decode_step_between_the_layers(kb, vb, rotate):
    """norm -> q/k/v product -> cache -> attention -> output product -> norm, for a batch of new tokens
    over cached prompts, against the same steps in the oracle from each step's own inputs."""
    rng = np.random.default_rng(30)
    B, hidden, heads, group, dim, page = 5, 512, 2, 4, 128, 32
    lens = np.array([40, 1, 64, 200, 97])  # with the new token
    width = 7
    sb = signs(rng, dim, rotate)
    c = D.Cache(B * width, page, heads, dim, kb, vb)
    table = rng.permutation(B * width).reshape(B, width)
    d, pool = kv_desc(c), pool_of(c)
    for b, n in enumerate(lens):  # the prompts
        t = np.arange(n - 1)
        if not t.size:
            continue
        k, v = vectors(rng, n - 1, heads, dim), vectors(rng, n - 1, heads, dim)
        s = (table[b][t // page] * page + t % page).astype(np.int32)
        Q.qlin_kv_write(d, pool, dev(k), dev(v), dev(s), sign_bits=dev(sb))
        c.write(k, v, s, sb)
    x, r = (dev(rng.standard_normal((B, hidden)).astype(np.float16)) for _ in range(2))
    norm_w = dev((1 + 0.1 * rng.standard_normal(hidden)).astype(np.float16))
    qkv = linear((group + 2) * heads * dim, hidden, 4, 1)
    proj = linear(hidden, group * heads * dim, 6, 2)
    nq = group * heads * dim

    h, r1 = Q.qlin_rmsnorm(x, norm_w, 1e-6, residual=r)
    y = Q.qlin_linear(qkv[0], qkv[1], qkv[2].scales, qkv[2].zeros, qkv[3], h) * 4
    q, k, v = (y[:, a:b].unflatten(1, (-1, dim)) for a, b in ((0, nq), (nq, nq + heads * dim), (nq + heads * dim, None)))
    slots = np.array([table[b][(n - 1) // page] * page + (n - 1) % page for b, n in enumerate(lens)], np.int32)
    Q.qlin_kv_write(d, pool, k, v, dev(slots), sign_bits=dev(sb))
    o = Q.qlin_attn_decode(d, pool, q, dev(table.astype(np.int32)), dev(lens.astype(np.int32)), sign_bits=dev(sb))
    z = Q.qlin_linear(proj[0], proj[1], proj[2].scales, proj[2].zeros, proj[3], o.flatten(1))
    h2, r2 = Q.qlin_rmsnorm(z, norm_w, 1e-6, residual=r1)
    torch.cuda.synchronize()

    c.write(k.cpu().numpy(), v.cpu().numpy(), slots, sb)
    assert np.array_equal(pool.cpu().numpy().reshape(c.bytes.shape), c.bytes)
    check_attention(o, c, q.cpu().numpy(), table, lens, sb=sb)
    ref = O.linear64(o.flatten(1).cpu().numpy(), proj[2].codes.cpu().numpy(), proj[2].scales.cpu().numpy(),
                     proj[2].zeros.cpu().numpy(), proj[3].cpu().numpy().view(np.uint32))
    rel_max, rel_fro = O.parity_errors(z.float().cpu().numpy(), ref)
    assert rel_max <= 2e-3 and rel_fro <= 1e-3
    ref_h, ref_r = D.rmsnorm64(z.cpu().numpy(), norm_w.cpu().numpy(), 1e-6, r1.cpu().numpy())
    assert np.array_equal(r2.cpu().numpy(), ref_r)
    assert np.allclose(h2.cpu().numpy().astype(np.float64), ref_h, rtol=2.0 ** -10, atol=2.0 ** -24)
