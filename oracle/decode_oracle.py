"""Oracle of the decode-step operators in plain numpy: the paged quantised
key/value cache, attention of one new token over it, and the residual norm.

Stored bytes and values read back are defined step by step in IEEE fp32, so they
are computed in numpy float32 and compared bit for bit; attention and the norm
are computed in float64.  Shares no code with the library.
"""
import numpy as np

GROUP = 128
INV_SQRT128 = np.float32(0.0883883476483184405)


def sign_vector(sign_bits: np.ndarray, d: int) -> np.ndarray:
    """+1 / -1 per dimension from uint32 words."""
    k = np.arange(d)
    return np.where((sign_bits[k // 32] >> (k % 32).astype(np.uint32)) & 1, -1.0, 1.0)


def butterflies32(x: np.ndarray) -> np.ndarray:
    """Seven add/subtract stages (strides 1, 2, ..., 64) per block of 128, then the scaling, in fp32."""
    y = x.astype(np.float32).reshape(-1, GROUP).copy()
    h = 1
    while h < GROUP:
        for i in range(0, GROUP, 2 * h):
            a, b = y[:, i:i + h].copy(), y[:, i + h:i + 2 * h].copy()
            y[:, i:i + h], y[:, i + h:i + 2 * h] = a + b, a - b
        h *= 2
    return (y * INV_SQRT128).reshape(x.shape)


def rotate32(x: np.ndarray, sign_bits) -> np.ndarray:
    if sign_bits is None:
        return x.astype(np.float32)
    return butterflies32(x.astype(np.float32) * sign_vector(sign_bits, x.shape[-1]).astype(np.float32))


def unrotate32(x: np.ndarray, sign_bits) -> np.ndarray:
    if sign_bits is None:
        return x.astype(np.float32)
    return butterflies32(x) * sign_vector(sign_bits, x.shape[-1]).astype(np.float32)


def rotation64(sign_bits, d: int) -> np.ndarray:
    """R [d][d]: (1/sqrt(128)) H diag(signs) per block of 128, H from bit parity."""
    if sign_bits is None:
        return np.eye(d)
    i = np.arange(d)
    common = (i[:, None] & i[None, :]) & (GROUP - 1)
    parity = np.zeros_like(common)
    for b in range(7):
        parity ^= (common >> b) & 1
    same = (i[:, None] // GROUP) == (i[None, :] // GROUP)
    return np.where(same, 1.0 - 2.0 * parity, 0.0) / np.sqrt(128.0) * sign_vector(sign_bits, d)[None, :]


def half_up(x: np.ndarray) -> np.ndarray:
    """fp16 rounded towards +infinity of positive fp32 values up to 65504."""
    h = x.astype(np.float16)
    low = h.astype(np.float32) < x
    return np.where(low, np.nextafter(h, np.float16(np.inf)), h)


def quantise32(v: np.ndarray, bits: int):
    """(codes uint8 [..., d], scales, zeros fp16 [..., d/128]) of fp32 vectors."""
    f = np.float32
    y = v.reshape(*v.shape[:-1], -1, GROUP)
    qmax = f(2 ** bits - 1)
    with np.errstate(all="ignore"):
        lo, hi = np.minimum(y.min(-1), f(0)) + f(0), np.maximum(y.max(-1), f(0))
        span = (hi - lo) / qmax
        finite = span < np.inf
        s = np.where((span > 0) & finite, half_up(np.where(finite, np.minimum(span, f(65504)), f(1))), np.float16(1))
        z = np.where(finite, (-lo / s.astype(f)).astype(np.float16), np.array(0x7FFF, np.uint16).view(np.float16))
        t = y / s.astype(f)[..., None] + z.astype(f)[..., None]
        q = np.where(np.isnan(t), f(0), np.clip(np.rint(t), f(0), qmax))
    return q.astype(np.uint8).reshape(v.shape), s, z


def pack_row(codes: np.ndarray, bits: int) -> np.ndarray:
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


class Cache:
    """A pool of pages in host memory: `bytes` [pages][kv_heads][block], with typed views of it."""

    def __init__(self, pages, page, heads, dim, k_bits, v_bits, fill=0):
        self.page, self.heads, self.dim, self.bits = page, heads, dim, (k_bits, v_bits)
        kr, vr = dim * k_bits // 8, dim * v_bits // 8
        par = 0 if k_bits == 16 else 8 * (dim // GROUP)
        self.bytes = np.full((pages, heads, page * (kr + vr + par)), fill, np.uint8)
        self.k = np.lib.stride_tricks.as_strided(self.bytes, (pages, heads, page, kr), self.bytes.strides[:2] + (kr, 1))
        self.v = np.lib.stride_tricks.as_strided(self.bytes[:, :, page * kr:], (pages, heads, page, vr),
                                                 self.bytes.strides[:2] + (vr, 1))
        self.par = None
        if par:
            p = self.bytes[:, :, page * (kr + vr):].view(np.float16)
            self.par = np.lib.stride_tricks.as_strided(p, (pages, heads, page, dim // GROUP, 4),
                                                       p.strides[:2] + (par, 8, 2))

    def write(self, k, v, slots, sign_bits=None):
        """k, v [T, heads, dim] fp16; slots [T] (outside the pool: skipped)."""
        for t, s in enumerate(slots):
            if s < 0 or s >= self.bytes.shape[0] * self.page:
                continue
            p, o = divmod(int(s), self.page)
            for side, (rows, x) in enumerate(((self.k, k[t]), (self.v, v[t]))):
                bits = self.bits[side]
                y = rotate32(x, sign_bits)
                if bits == 16:
                    rows[p, :, o] = (x if sign_bits is None else y.astype(np.float16)).view(np.uint8)
                    continue
                q, sc, z = quantise32(y, bits)
                rows[p, :, o] = pack_row(q, bits)
                self.par[p, :, o, :, 2 * side], self.par[p, :, o, :, 2 * side + 1] = sc, z

    def values(self, side, slots):
        """fp32 values s (q - z), still rotated, [T, heads, dim]."""
        slots = np.asarray(slots)
        p, o = slots // self.page, slots % self.page
        bits, rows = self.bits[side], (self.k, self.v)[side][p, :, o]
        if bits == 16:
            return np.ascontiguousarray(rows).view(np.float16).astype(np.float32)
        codes = rows if bits == 8 else np.stack((rows & 15, rows >> 4), -1).reshape(*rows.shape[:-1], self.dim)
        par = self.par[p, :, o].astype(np.float32)
        with np.errstate(all="ignore"):
            q = codes.reshape(*codes.shape[:-1], -1, GROUP).astype(np.float32)
            return (par[..., 2 * side, None] * (q - par[..., 2 * side + 1, None])).reshape(*codes.shape[:-1], self.dim)

    def read(self, slots, sign_bits=None):
        """(k, v) fp16 [T, heads, dim]; zeros for slots outside the pool."""
        slots = np.asarray(slots)
        ok = (slots >= 0) & (slots < self.bytes.shape[0] * self.page)
        at = np.where(ok, slots, 0)
        out = []
        for side in range(2):
            x = self.values(side, at)
            with np.errstate(all="ignore"):
                x = (x if sign_bits is None else unrotate32(x, sign_bits)).astype(np.float16)
            out.append(np.where(ok[:, None, None], x, np.float16(0)))
        return out


def attention64(cache: Cache, q, table, lens, scale, sign_bits=None):
    """(out, tolerance) [B, q_heads, dim] in float64, before the final rounding to fp16.

    The tolerance bounds what fp32 scores and 22-bit softmax weights may do:
      * a weight, times the value's scale, enters the value sums as two fp16 digits:
        2^-21 relative (within the last item's), or, where digits are subnormal, 2^-40
        of the sequence's largest such product (16 bits, without scales: 2^-32 of the
        largest weight).  For each token that moves the output by as much of q - z
        (at 16 bits of the value);
      * a score is 128 or 256 products summed in fp32 (a rounding of 2^-24 of the
        magnitudes per step, sums of code products and of the zero's share apart);
      * for 4- and 8-bit keys x is rounded to 24-bit integers of unit 2^(E-21), E the
        exponent of the group's largest |x|: at most 2^-22 max|x| a value, that is
        2^-22 max|x| sum |k| a score;
        a score's error e enters as p e |v - out|, twice that with the exponential's own;
      * the value sums are len products in fp32 over s (q + |z|);
      * everything else (rotation, quotient, joins) is some 64 fp32 steps.
    The inverse rotation mixes a group's errors with weights 1/sqrt(128)."""
    B, Hq, D = q.shape
    R = rotation64(sign_bits, D)
    out, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    g = Hq // cache.heads
    coded = cache.par is not None
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * cache.page)
        t = np.arange(n)
        pages = table[b][t // cache.page]
        t = t[(pages >= 0) & (pages < cache.bytes.shape[0])]
        if not t.size:
            continue
        slots = table[b][t // cache.page].astype(np.int64) * cache.page + t % cache.page
        k, v = cache.values(0, slots).astype(np.float64), cache.values(1, slots).astype(np.float64)
        mag, par = [], None
        for side, x in ((0, k), (1, v)):  # s (q + |z|) at most: |value| + 2 s |z|
            m = np.abs(x)
            if coded:
                par = cache.par[slots // cache.page, :, slots % cache.page].astype(np.float64)
                m = m + 2 * np.repeat(np.abs(par[..., 2 * side] * par[..., 2 * side + 1]), GROUP, -1)
            mag.append(m)
        for h in range(Hq):
            x = q[b, h].astype(np.float64)
            if sign_bits is not None:
                x = rotate32(q[b, h], sign_bits).astype(np.float16).astype(np.float64)
            kh, vh = k[:, h // g], v[:, h // g]
            s = scale * (kh @ x)
            e = abs(scale) * (mag[0][:, h // g] @ np.abs(x)) * (D + 64) * 2.0 ** -24 + np.abs(s) * 2.0 ** -22
            if coded:
                for c in range(0, D, GROUP):
                    e = e + abs(scale) * 2.0 ** -22 * np.abs(x[c:c + GROUP]).max() * np.abs(kh[:, c:c + GROUP]).sum(1)
            p = np.exp(s - s.max())
            p /= p.sum()
            o = p @ vh
            far = np.abs(vh - o)
            d = (p * (2 * e + 2.0 ** -20)) @ far
            if coded:
                for c in range(0, D, GROUP):
                    sv = par[:, h // g, c // GROUP, 2]  # scales of the values
                    steps = np.abs(vh[:, c:c + GROUP]) / np.where(sv > 0, sv, 1)[:, None]
                    d[c:c + GROUP] += 2.0 ** -40 * (p * sv).max() * steps.sum(0)
            else:
                d = d + 2.0 ** -32 * p.max() * np.abs(vh).sum(0)
            d = d + (t.size + 64) * 2.0 ** -24 * (p @ mag[1][:, h // g]) + 2.0 ** -18 * np.abs(o)
            out[b, h] = R.T @ o
            tol[b, h] = np.abs(R.T) @ d
    return out, tol + np.abs(out) * 2.0 ** -11 + 2.0 ** -25


def rmsnorm64(x, weight, eps, residual=None):
    """(y in float64, h fp16): h = fp16(x + residual), y = h / sqrt(mean h^2 + eps) * weight."""
    h = x if residual is None else (x.astype(np.float64) + residual.astype(np.float64)).astype(np.float16)
    w = h.astype(np.float64)
    return w / np.sqrt((w * w).mean(-1, keepdims=True) + eps) * weight.astype(np.float64), h
