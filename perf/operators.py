"""Timed cases of the decode-step operators around the quantised linear layers.

The linear layers of a decoder step are joined by three things: the norm in
front of them, the key/value cache that the step writes, and the attention of
the new token over that cache.  This file holds cases of each (``listed``,
``draw``), their inputs (``prepare``), one pass in plain torch operations or
through the library (``run``, by the module's ``own``), the definition in 64
bits (``exact``) and what a pass cannot do without (``work``).

Cache layout (one pool of pages, ``uint8 [pages][kv_heads][block]``); the block
of one page and one head holds, for its ``page`` tokens,

    K rows [page][head_dim * k_bits / 8], V rows [page][head_dim * v_bits / 8],
    and below 16 bits the parameters fp16 [page][head_dim / 128][4] = (ks, kz, vs, vz).

A row is a little-endian bit stream of codes, as ``qlin_pack`` writes it; at 16
bits it is the fp16 vector.  A vector is rotated (random signs, block-128
Walsh-Hadamard, 1/sqrt(128)) if the cache has signs, then quantised per group
of 128 on a grid that contains zero:

    lo = min(v, 0), hi = max(v, 0), qmax = 2^bits - 1,
    s = fp16 rounded up of (hi - lo) / qmax (1 if that is 0, at most 65504),
    z = fp16(-lo / s), q = clamp(rint(v / s + z), 0, qmax),  value = s (q - z).
"""
import math

import torch

own = False

GROUP = 128
INV_SQRT = 0.0883883476483184405  # 1 / sqrt(128)
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def _attention(name, batch, longest, q_heads=32, kv_heads=8, head_dim=128, page=64, k_bits=8, v_bits=8, rotate=False,
               ragged=True):
    return {"name": name, "op": "attention", "batch": batch, "longest": longest, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "k_bits": k_bits, "v_bits": v_bits,
            "rotate": rotate, "ragged": ragged}


def _cache(name, tokens, kv_heads=8, head_dim=128, page=64, k_bits=8, v_bits=8, rotate=True, padded=False, write=True):
    return {"name": name, "op": "cache" if write else "read", "tokens": tokens, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "k_bits": k_bits, "v_bits": v_bits, "rotate": rotate, "padded": padded}


def _norm(name, rows, width, residual=True):
    return {"name": name, "op": "norm", "rows": rows, "width": width, "residual": residual}


def listed():
    return [
        # one user, a short chat: a call whose latency counts
        _attention("attention 1 x 131, 8 bit", 1, 131, page=16, ragged=False),
        # one user, a long document, in 4 bits after the rotation
        _attention("attention 1 x 32773, 4 bit", 1, 32773, k_bits=4, v_bits=4, rotate=True, ragged=False),
        # a serving batch of mixed lengths, one slot of it empty
        _attention("attention 16 ragged, 8 bit", 16, 8190, page=32, rotate=True),
        # a full batch of short requests in small pages
        _attention("attention 200 short, 4 bit", 200, 509, page=16, k_bits=4, v_bits=4, rotate=True),
        # a cache that is not quantised, moderately long requests
        _attention("attention 48 x 2500, 16 bit", 48, 2500, k_bits=16, v_bits=16, ragged=False),
        # wide heads, eight queries a key, finer keys than values
        _attention("attention 7 ragged, wide 8/4", 7, 20011, q_heads=32, kv_heads=4, head_dim=256, page=128, v_bits=4),
        # the new tokens of a padded decode batch
        _cache("cache 16 padded, 8 bit", 16, page=16, padded=True),
        # a prompt
        _cache("cache 4099, 4 bit", 4099, k_bits=4, v_bits=4),
        # a long prompt with wide heads, not rotated
        _cache("cache 16384, wide 8/4", 16384, kv_heads=4, head_dim=256, page=128, v_bits=4, rotate=False),
        # a cached prefix read back for the next chunk of a prompt
        _cache("read 30001, 4/8 bit", 30001, page=32, k_bits=4, write=False),
        # one token in front of a layer
        _norm("norm 1 x 2560", 1, 2560),
        # a prompt in front of a layer
        _norm("norm 8191 x 2560", 8191, 2560),
    ]


def _about(rng, low, high):
    """Spread over the logarithm of the range, odd sizes among it."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("attention", "attention", "cache", "read", "norm"))
    if op == "norm":
        width = 8 * _about(rng, 8, 2048)
        c = _norm("", _about(rng, 1, max(1, min(8192, 20_000_000 // width))), width, rng.random() < 0.7)
        del c["name"]
        return c
    head_dim = rng.choice((128, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8, 8, 10))
    page = rng.choice((16, 32, 64, 128, 256))
    k_bits, v_bits = rng.choice(((4, 4), (8, 8), (8, 4), (4, 8), (16, 16)))
    rotate = rng.random() < 0.6
    if op == "attention":
        batch = _about(rng, 1, 200)
        longest = _about(rng, 1, max(2, min(32773, 120_000_000 // (batch * kv_heads * head_dim))))
        c = _attention("", batch, longest, kv_heads * rng.choice((1, 2, 4, 4, 5, 8, 16)), kv_heads, head_dim, page,
                       k_bits, v_bits, rotate, rng.random() < 0.7)
    else:
        tokens = _about(rng, 1, max(2, min(30001, 30_000_000 // (kv_heads * head_dim))))
        c = _cache("", tokens, kv_heads, head_dim, page, k_bits, v_bits, rotate, rng.random() < 0.3, op == "cache")
    del c["name"]
    return c


def _lengths(case):
    """Tokens of each sequence: all `longest`, or spread below it with the longest
    first and, in a batch of 8 or more, an empty slot second."""
    b, top = case["batch"], case["longest"]
    if not case["ragged"]:
        return [top] * b
    spread = [max(1, int(top ** (((i * 61) % 97) / 96.0))) for i in range(b)]
    mixed = [(n if i % 2 else 1 + (top - 1) * ((i * 37) % 101) // 101) for i, n in enumerate(spread)]
    mixed[0] = top
    if b >= 8:
        mixed[1] = 0
    return mixed


def _block(case):
    """Bytes of a K row, a V row, a token's parameters, and one (page, head) block."""
    d, kb, vb = case["head_dim"], case["k_bits"], case["v_bits"]
    k_row, v_row, par = d * kb // 8, d * vb // 8, 0 if kb == 16 else 8 * (d // GROUP)
    return k_row, v_row, par, case["page"] * (k_row + v_row + par)


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        return {"bytes": 2 * n * (4 if case["residual"] else 2) + 2 * case["width"], "flops": 6 * n}
    k_row, v_row, par, _ = _block(case)
    d, h = case["head_dim"], case["kv_heads"]
    stages = int(math.log2(GROUP)) if case["rotate"] else 0
    if case["op"] == "attention":
        tokens, rows = sum(_lengths(case)), case["batch"] * case["q_heads"]
        return {"bytes": tokens * h * (k_row + v_row + par) + 4 * rows * d + 4 * sum(-(-n // case["page"]) + 1 for n in _lengths(case)),
                "flops": 4 * tokens * case["q_heads"] * d + 2 * rows * d * stages}
    n = case["tokens"] * h
    stored, plain = n * (k_row + v_row + par), 4 * n * d
    passes = 2 if case["op"] == "cache" else 1  # written and read back, or read alone
    return {"bytes": passes * (stored + plain) + 4 * case["tokens"], "flops": passes * 2 * n * d * (stages + 4)}


# ------------------------------------------------- plain torch: the arithmetic

def _stage(x, h):
    """One butterfly stage of stride h along the last dimension (of 128 values)."""
    y = x.unflatten(-1, (-1, 2, h))
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack((a + b, a - b), -2).flatten(-3)


def _hadamard(x):
    """Walsh-Hadamard transform of each block of 128 in 32 bits, strides 1 to 64, times 1/sqrt(128)."""
    y = x.unflatten(-1, (-1, GROUP))
    y = _stage(_stage(_stage(_stage(_stage(_stage(_stage(y, 1), 2), 4), 8), 16), 32), 64)
    return (y * torch.tensor(INV_SQRT, dtype=torch.float32, device=x.device)).flatten(-2)


def _flip(x, signs):
    """x with the sign of element k changed where bit k of signs is set."""
    bits = (signs.unsqueeze(-1) >> torch.arange(32, device=signs.device, dtype=torch.int32)) & 1
    return torch.where(bits.flatten().bool(), -x, x)


def _rotate(x, signs):
    return x if signs is None else _hadamard(_flip(x, signs))


def _unrotate(x, signs):
    return x if signs is None else _flip(_hadamard(x), signs)


def _half_up(x):
    """fp16, rounded up, of positive 32-bit values."""
    h = x.half()
    return torch.where(h.float() < x, (h.view(torch.int16) + 1).view(torch.float16), h)


def _quantise(v, bits):
    """Codes, scales and zeros of 32-bit vectors, per group of 128."""
    y = v.unflatten(-1, (-1, GROUP))
    qmax = float(2 ** bits - 1)
    zero = torch.zeros((), dtype=torch.float32, device=v.device)
    lo, hi = torch.minimum(y.amin(-1), zero), torch.maximum(y.amax(-1), zero)
    span = (hi - lo) / torch.full_like(hi, qmax)  # a quotient: division by a number multiplies by its reciprocal
    s = torch.where(span > 0, _half_up(torch.clamp(span, max=65504.0)), torch.ones_like(span).half())
    z = (-lo / s.float()).half()
    q = torch.clamp(torch.round(y / s.float().unsqueeze(-1) + z.float().unsqueeze(-1)), 0.0, qmax)
    return q.flatten(-2).to(torch.uint8), s, z


def _bytes_of(codes, bits):
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _codes_of(rows, bits):
    return rows if bits == 8 else torch.stack((rows & 15, rows >> 4), -1).flatten(-2)


def _sections(case, pool):
    """Views of the pool: K rows, V rows [pages][heads][page][bytes], parameters [pages][heads][page][groups][4]."""
    k_row, v_row, par, _ = _block(case)
    p = case["page"]
    k = pool[:, :, :p * k_row].unflatten(2, (p, k_row))
    v = pool[:, :, p * k_row:p * (k_row + v_row)].unflatten(2, (p, v_row))
    if not par:
        return k, v, None
    return k, v, pool[:, :, p * (k_row + v_row):].view(torch.float16).unflatten(2, (p, case["head_dim"] // GROUP, 4))


def _stored(case, k, v, signs):
    """What the cache holds for fp16 vectors k, v [..., head_dim]: rows as bytes, and parameters."""
    k, v = _rotate(k.float(), signs), _rotate(v.float(), signs)
    if case["k_bits"] == 16:
        return k.half().view(torch.uint8), v.half().view(torch.uint8), None
    (kq, ks, kz), (vq, vs, vz) = _quantise(k, case["k_bits"]), _quantise(v, case["v_bits"])
    return _bytes_of(kq, case["k_bits"]), _bytes_of(vq, case["v_bits"]), torch.stack((ks, kz, vs, vz), -1)


def _values(rows, bits, s, z):
    """32-bit values (still rotated) of stored rows [..., bytes] with scales and zeros [..., groups]."""
    if bits == 16:
        return rows.contiguous().view(torch.float16).float()
    q = _codes_of(rows, bits).unflatten(-1, (-1, GROUP)).float()
    return (s.float().unsqueeze(-1) * (q - z.float().unsqueeze(-1))).flatten(-2)


# --------------------------------------------------------------- the inputs

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, *shape):
    """Keys with a few channels that stand out, as keys have."""
    d = shape[-1]
    gain = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.03, 6.0, 1.0)
    return (_randn(gen, *shape) * gain).half()


def _pool(case, gen, pages, signs):
    """A pool of that many pages, every slot of it written."""
    p, h, d = case["page"], case["kv_heads"], case["head_dim"]
    k = _keys(gen, pages, h, p, d)
    v = (0.5 * _randn(gen, pages, h, p, d)).half()
    pool = torch.zeros(pages, h, _block(case)[3], dtype=torch.uint8, device="cuda")
    for part, data in zip(_sections(case, pool), _stored(case, k, v, signs)):
        if data is not None:
            part.copy_(data)
    return pool


def _describe(case, pages):
    if not own:
        return None
    from dequant_gemv_packed_b200 import qlin
    return qlin.KVDesc(pages, case["page"], case["kv_heads"], case["head_dim"], case["k_bits"], case["v_bits"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "norm":
        m, k = case["rows"], case["width"]
        return {"case": case, "x": _randn(gen, m, k).half(), "weight": (1.0 + 0.2 * _randn(gen, k)).half(),
                "residual": (4.0 * _randn(gen, m, k)).half() if case["residual"] else None}
    signs = None
    if case["rotate"]:
        signs = torch.randint(-2 ** 31, 2 ** 31, (case["head_dim"] // 32,), generator=gen, device="cuda").to(torch.int32)
    p, h, d = case["page"], case["kv_heads"], case["head_dim"]
    if case["op"] == "attention":
        lens = _lengths(case)
        need = [-(-n // p) for n in lens]
        width, total = max(1, max(need)), sum(need)
        pages = total + 3
        order = torch.randperm(pages, generator=gen, device="cuda")[:total].to(torch.int32)
        # each sequence's pages are the next ones of the shuffled list; entries past its length are not looked at
        start = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda").unsqueeze(1)
        count = torch.tensor(need, device="cuda").unsqueeze(1)
        at = torch.arange(width, device="cuda").unsqueeze(0)
        picked = order[(start + at).clamp(max=max(total - 1, 0))] if total else torch.zeros_like(start + at, dtype=torch.int32)
        table = torch.where(at < count, picked, torch.full_like(picked, -1)).contiguous()
        # the queries are the first columns of the rows that one product for q, k and v gives
        fused = (2.0 * _randn(gen, case["batch"], (case["q_heads"] + 2 * h) * d)).half()
        return {"case": case, "pages": pages, "cache": _pool(case, gen, pages, signs), "signs": signs, "table": table,
                "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
                "q": fused[:, :case["q_heads"] * d].unflatten(1, (case["q_heads"], d))}
    t = case["tokens"]
    pages = -(-t // p) + 2
    # consecutive tokens of shuffled pages
    order = torch.randperm(pages, generator=gen, device="cuda")[:-(-t // p)]
    at = torch.arange(t, device="cuda")
    slots = order[at // p] * p + at % p
    if case["padded"]:
        slots = torch.where(at % 5 == 3, torch.full_like(slots, -1), slots)
    slots = slots.to(torch.int32)
    if case["op"] == "read":
        return {"case": case, "pages": pages, "cache": _pool(case, gen, pages, signs), "signs": signs, "slots": slots}
    # keys and values are the last columns of the rows that one product for q, k and v gives
    fused = torch.empty(t, (4 * h + 2 * h) * d, dtype=torch.float16, device="cuda")
    fused[:, 4 * h * d:5 * h * d] = _keys(gen, t, h, d).flatten(1)
    fused[:, 5 * h * d:] = (0.5 * _randn(gen, t, h * d)).half()
    return {"case": case, "pages": pages, "signs": signs, "slots": slots,
            "cache": torch.zeros(pages, h, _block(case)[3], dtype=torch.uint8, device="cuda"),
            "k": fused[:, 4 * h * d:5 * h * d].unflatten(1, (h, d)), "v": fused[:, 5 * h * d:].unflatten(1, (h, d))}


# ------------------------------------------------------------------ the passes

def _plain_norm(s):
    h = s["x"].float() if s["residual"] is None else (s["x"].float() + s["residual"].float()).half().float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    return {"y": y.half()} if s["residual"] is None else {"y": y.half(), "residual": h.half()}


def _plain_write(s):
    case, p = s["case"], s["case"]["page"]
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    for part, data in zip(_sections(case, s["cache"]), _stored(case, s["k"], s["v"], s["signs"])):
        if data is not None:
            part[at // p, :, at % p] = data[live]


def _plain_read(s):
    case, p = s["case"], s["case"]["page"]
    live = (s["slots"] >= 0).view(-1, 1, 1)
    at = s["slots"].clamp(min=0).long()
    k, v, par = _sections(case, s["cache"])
    q = (None,) * 4 if par is None else par[at // p, :, at % p].unbind(-1)
    k = _unrotate(_values(k[at // p, :, at % p], case["k_bits"], q[0], q[1]), s["signs"]).half()
    v = _unrotate(_values(v[at // p, :, at % p], case["v_bits"], q[2], q[3]), s["signs"]).half()
    return {"k": torch.where(live, k, torch.zeros_like(k)), "v": torch.where(live, v, torch.zeros_like(v))}


def _plain_attention(s):
    case = s["case"]
    h, d, b = case["kv_heads"], case["head_dim"], case["batch"]
    table = s["table"].clamp(min=0).long()
    # [batch][width][heads][page][...] -> [batch][heads][tokens][...]
    k, v, par = (None if x is None else x[table].transpose(1, 2).flatten(2, 3) for x in _sections(case, s["cache"]))
    q4 = (None,) * 4 if par is None else par.unbind(-1)
    k = _values(k, case["k_bits"], q4[0], q4[1])
    x = _rotate(s["q"].float(), s["signs"])
    x = (x.half() if s["signs"] is not None else x).float().unflatten(1, (h, -1))
    score = torch.matmul(x, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))  # [batch][heads][group][tokens]
    live = torch.arange(score.shape[-1], device=score.device) < s["lens"].view(b, 1, 1, 1)
    score = torch.where(live, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    v = _values(v, case["v_bits"], q4[2], q4[3])
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return _unrotate(o, s["signs"]).half().flatten(1, 2)


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "norm":
            return _plain_norm(state)
        if case["op"] == "attention":
            return {"out": _plain_attention(state)}
        if case["op"] == "cache":
            _plain_write(state)
        return _plain_read(state)
    from dequant_gemv_packed_b200 import qlin
    if case["op"] == "norm":
        if state["residual"] is None:
            return {"y": qlin.qlin_rmsnorm(state["x"], state["weight"], EPS)}
        y, h = qlin.qlin_rmsnorm(state["x"], state["weight"], EPS, residual=state["residual"])
        return {"y": y, "residual": h}
    desc = state.get("desc")
    if desc is None:  # the handle that a program keeps with its cache
        desc = state["desc"] = _describe(case, state["pages"])
    if case["op"] == "attention":
        return {"out": qlin.qlin_attn_decode(desc, state["cache"], state["q"], state["table"], state["lens"],
                                             sign_bits=state["signs"])}
    if case["op"] == "cache":
        qlin.qlin_kv_write(desc, state["cache"], state["k"], state["v"], state["slots"], sign_bits=state["signs"])
    k, v = qlin.qlin_kv_read(desc, state["cache"], state["slots"], sign_bits=state["signs"])
    return {"k": k, "v": v}


# ------------------------------------------------- the definition in 64 bits

def _matrix64(signs, d):
    """Rotation as a matrix R [d][d], R x = (H diag(signs) x) / sqrt(128) per block of 128."""
    if signs is None:
        return torch.eye(d, dtype=torch.float64, device="cuda")
    i = torch.arange(d, device="cuda")
    common = (i.view(-1, 1) & i.view(1, -1)) & (GROUP - 1)
    odd = sum((common >> k) & 1 for k in range(7)) & 1
    m = (1.0 - 2.0 * odd.double()) * (i.view(-1, 1) // GROUP == i.view(1, -1) // GROUP) / math.sqrt(float(GROUP))
    sign = 1.0 - 2.0 * ((signs.long()[i // 32] >> (i % 32)) & 1).double()
    return m * sign.view(1, -1)


def _grid64(v, bits):
    """Quantised values of 64-bit vectors, by the definition (scale and zero in fp16, the rest in 64 bits)."""
    top = 2.0 ** bits - 1.0
    out = torch.empty_like(v)
    for g in range(v.shape[-1] // GROUP):
        x = v[..., g * GROUP:(g + 1) * GROUP]
        lo, hi = x.amin(-1, keepdim=True).clamp(max=0.0), x.amax(-1, keepdim=True).clamp(min=0.0)
        want = ((hi - lo) / top).clamp(max=65504.0)
        step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -14))) - 10.0)
        s = torch.ceil(want / step) * step
        s = torch.where(s == 0, torch.ones_like(s), s)
        z = (-lo / s).half().double()
        out[..., g * GROUP:(g + 1) * GROUP] = s * (torch.round(x / s + z).clamp(0.0, top) - z)
    return out


def _held64(case, pool, pages, offsets, what):
    """64-bit values (still rotated) that the cache holds at (page, offset) pairs: [...][heads][head_dim]."""
    k_row, v_row, par, _ = _block(case)
    p, d = case["page"], case["head_dim"]
    bits, row, base = (case["k_bits"], k_row, 0) if what == "k" else (case["v_bits"], v_row, p * k_row)
    flat = pool.view(pool.shape[0], pool.shape[1], -1)
    heads = torch.arange(pool.shape[1], device="cuda")
    at = (base + offsets * row).unsqueeze(-1) + torch.arange(row, device="cuda")
    raw = flat[pages[..., None, None], heads[:, None], at.unsqueeze(-2)]
    if bits == 16:
        return raw.contiguous().view(torch.float16).double()
    codes = raw.double() if bits == 8 else torch.empty(*raw.shape[:-1], d, dtype=torch.float64, device="cuda")
    if bits == 4:
        codes[..., 0::2] = (raw % 16).double()
        codes[..., 1::2] = (raw // 16).double()
    at = (p * (k_row + v_row) + offsets * par).unsqueeze(-1) + torch.arange(par, device="cuda")
    four = flat[pages[..., None, None], heads[:, None], at.unsqueeze(-2)].contiguous().view(torch.float16).double()
    i = torch.arange(d, device="cuda") // GROUP * 4 + (0 if what == "k" else 2)
    return four[..., i] * (codes - four[..., i + 1])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = (h + s["residual"].double()).half().double()
        mean = torch.einsum("mk,mk->m", h, h) / case["width"]
        y = torch.einsum("mk,m,k->mk", h, 1.0 / torch.sqrt(mean + EPS), s["weight"].double())
        return {"y": y} if s["residual"] is None else {"y": y, "residual": h}
    turn = _matrix64(s["signs"], case["head_dim"])
    p = case["page"]
    if case["op"] != "attention":
        slots = s["slots"].long()
        ok = (slots >= 0).double().view(-1, 1, 1)
        if case["op"] == "read":
            at = slots.clamp(min=0)
            return {w: ok * (_held64(case, s["cache"], at // p, at % p, w) @ turn) for w in ("k", "v")}
        out = {}
        for w in ("k", "v"):
            x, bits = s[w].double() @ turn.T, case[w + "_bits"]
            out[w] = ok * ((x.half().double() if bits == 16 else _grid64(x, bits)) @ turn)
        return out
    lens, h, d = s["lens"].tolist(), case["kv_heads"], case["head_dim"]
    out = torch.zeros(case["batch"], case["q_heads"], d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):  # one sequence at a time
        if not n:
            continue
        t = torch.arange(n, device="cuda")
        pages = s["table"][b].long()[t // p]
        k = _held64(case, s["cache"], pages, t % p, "k")
        v = _held64(case, s["cache"], pages, t % p, "v")
        x = s["q"][b].double()
        if s["signs"] is not None:
            x = (x @ turn.T).half().double()
        x = x.view(h, -1, d)
        w = torch.softmax(torch.einsum("hgd,thd->hgt", x, k) / math.sqrt(float(d)), -1)
        out[b] = (torch.einsum("hgt,thd->hgd", w, v) @ turn).reshape(case["q_heads"], d)
    return {"out": out}
