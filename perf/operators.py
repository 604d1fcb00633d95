"""Cases and plain forms of the operators around decode: rotary positions (and
their gradient), a paged key/value cache held in 4 bits (append, read back,
attention over it), the attention weight that each cached key has gathered,
and the eviction of the keys that gathered least.

``run(state)`` computes one pass in elementary torch operations where ``own``
is false, and with the calls a user makes of io_aware_attention_gb300 where it
is true.  ``exact(case, seed)`` is the definition in 64 bits, written apart.

The cache.  A pool is uint8 (pages, kv heads, 72 * D): a page holds 64 keys of
one kv head, D = 64 or 128 stored channels (a head size in between is padded
with zeros).  A stored value is e2m1 * e4m3 * (the tensor's scale): a sign, two
exponent bits and one mantissa bit a value, one e4m3 scale for 16 channels.
Within a page's block, with key x = 0 .. 63, channel c, block of channels b:
  K codes   at 0:      byte x*D/2 + c/2, low nibble the even channel;
  K scales  at 32*D:   byte ((x%8)*4 + b/p)*8*p + (x/8)*p + b%p, p = D/64;
  V codes   at 36*D:   byte (x/2)*D + c, low nibble the even key;
  V scales  at 68*D:   byte (((x/2)%4)*D/16 + b)*16 + (x/8)*2 + x%2.
Key j of sequence s lies in page table[s][j / 64], row j % 64.
"""
import math

import torch

own = False

PAGE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One generated token of four sequences far into a long context, grouped heads.
        {"name": "rope_token", "op": "rope", "B": 4, "H": 32, "Hkv": 8, "N": 1, "d": 128, "rot": 128, "layout": "half",
         "stretch": 8.0, "first": 100000, "bwd": False},
        # A training step's queries and keys (this repository's headline shape), forward and gradient.
        {"name": "rope_train", "op": "rope", "B": 8, "H": 32, "Hkv": 32, "N": 4096, "d": 128, "rot": 128,
         "layout": "half", "stretch": 1.0, "first": 0, "bwd": True},
        # An odd length, an in-between head size and part of the head rotated in neighbouring pairs.
        {"name": "rope_part", "op": "rope", "B": 3, "H": 10, "Hkv": 2, "N": 1021, "d": 80, "rot": 40,
         "layout": "interleaved", "stretch": 1.0, "first": 17, "bwd": True},
        # One generated token of 64 sequences of unequal lengths goes into the cache.
        {"name": "append_token", "op": "append", "B": 64, "Hkv": 8, "N": 1, "d": 128, "most": 4096, "least": 1},
        # Prompts of unequal lengths, right-aligned in one batch, go into an empty cache.
        {"name": "append_prompt", "op": "append", "B": 4, "Hkv": 8, "N": 4096, "d": 128, "most": 4096, "least": 700},
        # The smallest decode call: one sequence, one token, grouped heads.
        {"name": "decode_one", "op": "decode", "B": 1, "H": 32, "Hkv": 8, "Nq": 1, "d": 128, "most": 1000, "least": 1000,
         "causal": False},
        # A batch of unequal lengths, from no key at all, with four new tokens each.
        {"name": "decode_ragged", "op": "decode", "B": 48, "H": 16, "Hkv": 4, "Nq": 4, "d": 64, "most": 5000, "least": 0,
         "causal": True},
        # The decode bench's shape: 8 sequences of 32768 keys, every head with keys of its own.
        {"name": "decode_long", "op": "decode", "B": 8, "H": 32, "Hkv": 32, "Nq": 1, "d": 128, "most": 32768,
         "least": 32768, "causal": False},
        # The weight that one new token gives to a middling cache.
        {"name": "weights_one", "op": "weights", "B": 1, "H": 32, "Hkv": 8, "Nq": 1, "d": 128, "most": 4097, "least": 4097,
         "causal": False},
        # The same for eight long sequences.
        {"name": "weights_long", "op": "weights", "B": 8, "H": 32, "Hkv": 8, "Nq": 2, "d": 128, "most": 32768,
         "least": 30000, "causal": True},
        # Two short sequences cut back to 512 keys.
        {"name": "evict_short", "op": "evict", "B": 2, "Hkv": 8, "d": 64, "most": 1500, "least": 300, "keep": 512,
         "sink": 4, "recent": 64},
        # Eight long sequences cut back to an eighth.
        {"name": "evict_long", "op": "evict", "B": 8, "Hkv": 8, "d": 128, "most": 32768, "least": 30001, "keep": 4096,
         "sink": 16, "recent": 512},
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "weights", "evict"])
    hkv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    if op == "rope":
        d = 8 * rng.randint(2, 16)
        heads = hkv * rng.choice([1, 2, 4])
        n = _spread(rng, 1, 8192)
        most = max(1, min(64, (8 * 32 * 4096 * 128) // (heads * n * d)))
        return {"op": op, "B": _spread(rng, 1, most), "H": heads, "Hkv": hkv, "N": n, "d": d,
                "rot": d if rng.random() < 0.4 else 2 * rng.randint(1, d // 2),
                "layout": rng.choice(["half", "interleaved"]), "stretch": rng.choice([1.0, 2.0, 8.0]),
                "first": rng.choice([0, rng.randint(0, 1000000)]), "bwd": rng.random() < 0.6}
    d = rng.choice([64, 128, 128, 8 * rng.randint(2, 16)])
    if op == "append":
        n = rng.choice([1, _spread(rng, 1, 8192)])
        most = max(n, _spread(rng, 1, 8192))
        batch = _spread(rng, 1, max(1, min(64, (1 << 19) // (hkv * most))))
        return {"op": op, "B": batch, "Hkv": hkv, "N": n, "d": d, "most": most, "least": rng.randint(0, most)}
    most = _spread(rng, 1 if op != "evict" else 16, 40000)
    batch = _spread(rng, 1, max(1, min(256, (1 << 22) // (hkv * (most + PAGE)))))
    least = rng.choice([most, rng.randint(0, most)])
    if op == "evict":
        keep = _spread(rng, 1, most)
        recent = rng.randint(0, keep)
        return {"op": op, "B": batch, "Hkv": hkv, "d": d, "most": most, "least": least, "keep": keep,
                "sink": rng.randint(0, min(16, keep - recent)), "recent": recent}
    return {"op": op, "B": batch, "H": hkv * rng.choice([1, 2, 4, 7, 8]), "Hkv": hkv, "Nq": rng.choice([1, 1, 2, 3, 8]),
            "d": d, "most": most, "least": least, "causal": rng.random() < 0.5}


# ------------------------------------------------------------- what is in hand

def _stored(d):
    return 64 if d <= 64 else 128


def _turns(inv_freq):
    """Rotation per position in units of 2^-64 of a turn, as the 64 bits of an int64."""
    out = []
    for f in inv_freq:
        u = int(round(f / (2.0 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1)
        out.append(u - 2 ** 64 if u >= 2 ** 63 else u)
    return out


def _inv_freq(rot, stretch):
    return [10000.0 ** (-2.0 * i / rot) / stretch for i in range(rot // 2)]


def _lens(case, gen):
    low, high = case["least"], case["most"]
    n = torch.randint(low, high + 1, (case["B"],), generator=gen, device="cuda", dtype=torch.int32)
    n[0] = high
    n[-1] = low if case["B"] > 1 else high
    return n


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _pages(case, gen, spare):
    """A page table over a pool with spare pages, in no order."""
    most = (case["most"] + PAGE - 1) // PAGE
    count = case["B"] * most + spare
    order = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    return count, order[:case["B"] * most].reshape(case["B"], most).contiguous(), order[case["B"] * most:]


def _filled(case, gen, spare=3):
    """A pool holding the keys and values of random sequences: what earlier
    appends left.  Places of no key hold junk."""
    B, Hkv, d, D = case["B"], case["Hkv"], case["d"], _stored(case["d"])
    count, table, rest = _pages(case, gen, spare)
    lens = _lens(case, gen)
    pool = torch.randint(0, 256, (count, Hkv, 72 * D), generator=gen, device="cuda", dtype=torch.uint8)
    most = table.shape[1]
    if most:
        real = (torch.arange(most * PAGE, device="cuda")[None] < lens[:, None]).reshape(B, 1, most, PAGE)
        old = pool[table.long()].permute(0, 2, 1, 3)
        gain = torch.exp(0.5 * _randn(gen, Hkv, 1, D))
        new = []
        for plane in range(2):
            x = _randn(gen, B, Hkv, most * PAGE, D)
            x = x * gain if plane == 0 else x
            x[..., d:] = 0
            new.append(_quantise(x))
            del x
        packed = _pack(new[0], new[1], B, Hkv, most, D)
        # Rows behind a sequence's end keep the junk.
        keep = _row_masks(real, D)
        mixed = (packed & keep) | (old & ~keep)
        pool[table.long()] = mixed.permute(0, 2, 1, 3)
    return pool, table, lens, rest


def _row_masks(real, D):
    """0xff (or a nibble's bits) where a byte of a page's block belongs to a real key: real is (B, 1, pages, 64)."""
    B, _, P, _ = real.shape
    nb, p = D // 16, D // 64
    full = real.to(torch.uint8) * 255
    kc = full[..., None].expand(B, 1, P, 64, D // 2).reshape(B, 1, P, -1)
    ks = full.reshape(B, 1, P, 8, 8).transpose(-1, -2)[:, :, :, :, None, :, None].expand(B, 1, P, 8, 4, 8, p).reshape(B, 1, P, -1)
    pair = real.reshape(B, 1, P, 32, 2)
    nib = pair[..., 0].to(torch.uint8) * 15 + pair[..., 1].to(torch.uint8) * 240
    vc = nib[..., None].expand(B, 1, P, 32, D).reshape(B, 1, P, -1)
    vs = full.reshape(B, 1, P, 8, 4, 2).permute(0, 1, 2, 4, 3, 5)[:, :, :, :, None].expand(B, 1, P, 4, nb, 8, 2).reshape(B, 1, P, -1)
    return torch.cat([kc, ks, vc, vs], -1)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": dict(case)}
    op = case["op"]
    if op == "rope":
        B, N, d = case["B"], case["N"], case["d"]
        s["q"] = _randn(gen, B, case["H"], N, d).to(torch.bfloat16)
        s["k"] = _randn(gen, B, case["Hkv"], N, d).to(torch.bfloat16)
        if case["bwd"]:
            s["dq"] = _randn(gen, B, case["H"], N, d).to(torch.bfloat16)
            s["dk"] = _randn(gen, B, case["Hkv"], N, d).to(torch.bfloat16)
        inv = _inv_freq(case["rot"], case["stretch"])
        s["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device="cuda")
        s["freqs"] = torch.tensor(_turns(inv), dtype=torch.int64, device="cuda")
        s["factor"] = 0.1 * math.log(case["stretch"]) + 1.0
        shift = torch.randint(0, 1 + case["first"] // 8, (B, 1), generator=gen, device="cuda")
        s["positions"] = (case["first"] - shift + torch.arange(N, device="cuda")[None]).to(torch.int32).contiguous()
        return s
    if op == "append":
        B, D = case["B"], _stored(case["d"])
        count, s["table"], _ = _pages(case, gen, 3)
        s["lens"] = _lens(case, gen)
        s["pool"] = torch.randint(0, 256, (count, case["Hkv"], 72 * D), generator=gen, device="cuda", dtype=torch.uint8)
        gain = torch.exp(0.5 * _randn(gen, case["Hkv"], 1, case["d"]))
        s["k"] = (_randn(gen, B, case["Hkv"], case["N"], case["d"]) * gain).to(torch.bfloat16)
        s["v"] = _randn(gen, B, case["Hkv"], case["N"], case["d"]).to(torch.bfloat16)
        return s
    # Twice the pages of the kept keys lie free where keys are evicted into them.
    kept_pages = -(-case["keep"] // PAGE) if op == "evict" else 0
    s["pool"], s["table"], s["lens"], rest = _filled(case, gen, 3 + case["B"] * kept_pages)
    if op == "evict":
        s["table_out"] = rest[:case["B"] * kept_pages].reshape(case["B"], kept_pages).contiguous()
        # Weights gathered over many tokens: a few keys hold most, many hold the same nothing.
        w = torch.exp(2.0 * _randn(gen, case["B"], case["Hkv"], case["most"]))
        s["weights"] = torch.where(w < 0.3, torch.zeros_like(w), w)
        return s
    s["q"] = _randn(gen, case["B"], case["H"], case["Nq"], case["d"]).to(torch.bfloat16)
    s["scale"] = 1.0 / math.sqrt(case["d"])
    if op == "weights":
        s["weights"] = torch.rand((case["B"], case["Hkv"], case["most"]), generator=gen, device="cuda")
        s["lse"] = _attend(s)[1]
    return s


# ---------------------------------------------------------------- plain forms

def _quantise(x):
    """(codes, scale bytes) of fp32 rows (..., D): one e4m3 scale for 16 channels."""
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    scale = (blocks.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = scale.float()[..., None]
    y = torch.where(sf > 0, blocks / sf, 0.0 * blocks)
    a = y.abs()
    # Nearest of 0 .5 1 1.5 2 3 4 6; halfway goes to the even code.
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + torch.signbit(y).to(torch.uint8) * 8
    return code.reshape(x.shape), scale.view(torch.uint8)


def _pack(k, v, B, Hkv, P, D):
    """Pages (B, Hkv, P, 72 * D) of quantised keys and values (B, Hkv, P * 64, ...)."""
    nb, p = D // 16, D // 64
    kc = k[0].reshape(B, Hkv, P, 64, D // 2, 2)
    kc = (kc[..., 0] | (kc[..., 1] << 4)).reshape(B, Hkv, P, -1)
    ks = k[1].reshape(B, Hkv, P, 8, 8, 4, p).permute(0, 1, 2, 4, 5, 3, 6).reshape(B, Hkv, P, -1)
    vc = v[0].reshape(B, Hkv, P, 32, 2, D)
    vc = (vc[:, :, :, :, 0] | (vc[:, :, :, :, 1] << 4)).reshape(B, Hkv, P, -1)
    vs = v[1].reshape(B, Hkv, P, 8, 4, 2, nb).permute(0, 1, 2, 4, 6, 3, 5).reshape(B, Hkv, P, -1)
    return torch.cat([kc, ks, vc, vs], -1)


def _grid(device):
    return torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=device)


def _read(pool, table, at, real, d):
    """bf16 (k, v) of the places at (B, Hkv, n), (B, Hkv, n, d); 0 where real is false."""
    Hkv, D = pool.shape[1], pool.shape[2] // 72
    nb, p = D // 16, D // 64
    at = torch.where(real, at, 0)
    page = table.long()[:, None].expand(-1, Hkv, -1).gather(2, at // PAGE)
    start = ((page * Hkv + torch.arange(Hkv, device=pool.device)[None, :, None]) * 72 * D)[..., None]
    flat, grid, x = pool.view(-1), _grid(pool.device), (at % PAGE)[..., None]
    ch, bl = torch.arange(d, device=pool.device), torch.arange(nb, device=pool.device)

    def rows(codes, scales):
        y = grid[codes.int()] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)[..., :d]
        return torch.where(real[..., None], y, 0.0).to(torch.bfloat16)

    k = rows(flat[start + x * (D // 2) + ch // 2] >> (ch % 2 * 4).to(torch.uint8) & 15,
             flat[start + 32 * D + ((x % 8) * 4 + bl // p) * 8 * p + x // 8 * p + bl % p])
    v = rows(flat[start + 36 * D + x // 2 * D + ch] >> (x % 2 * 4).to(torch.uint8) & 15,
             flat[start + 68 * D + ((x // 2 % 4) * nb + bl) * 16 + x // 8 * 2 + x % 2])
    return k, v


def _unpack(pool, table, lens, d, values=True):
    """fp32 (k, v) of every place of the table, (B, Hkv, pages * 64, d); 0 where there is no key."""
    B, P = table.shape
    Hkv, D = pool.shape[1], pool.shape[2] // 72
    nb, p = D // 16, D // 64
    real = torch.arange(P * PAGE, device=pool.device)[None] < lens[:, None]
    blocks = pool[table.long()].permute(0, 2, 1, 3)
    grid = _grid(pool.device)

    def rows(codes, scales):
        x = grid[codes.int()].reshape(B, Hkv, P * PAGE, nb, 16)
        x = x * scales.contiguous().view(torch.float8_e4m3fn).float().reshape(B, Hkv, P * PAGE, nb, 1)
        return torch.where(real[:, None, :, None], x.reshape(B, Hkv, P * PAGE, D), 0.0)[..., :d]

    kc = blocks[..., :32 * D]
    kc = torch.stack([kc & 15, kc >> 4], -1)
    ks = blocks[..., 32 * D:36 * D].reshape(B, Hkv, P, 8, 4, 8, p).permute(0, 1, 2, 5, 3, 4, 6)
    k = rows(kc, ks)
    if not values:
        return k, None
    vc = blocks[..., 36 * D:68 * D].reshape(B, Hkv, P, 32, 1, D)
    vc = torch.cat([vc & 15, vc >> 4], 4)
    vs = blocks[..., 68 * D:].reshape(B, Hkv, P, 4, nb, 8, 2).permute(0, 1, 2, 5, 3, 6, 4)
    return k, rows(vc, vs)


def _scores(s, values):
    """Masked fp32 scores (B, Hkv, G * Nq, places) and the values."""
    c = s["case"]
    k, v = _unpack(s["pool"], s["table"], s["lens"], c["d"], values)
    rows = c["H"] // c["Hkv"] * c["Nq"]
    q = s["q"].float().reshape(c["B"], c["Hkv"], rows, c["d"])
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    seen = s["lens"][:, None].expand(c["B"], c["Nq"])
    if c["causal"]:
        seen = seen - c["Nq"] + 1 + torch.arange(c["Nq"], device=x.device)[None]
    seen = seen[:, None, :, None].expand(c["B"], c["H"], c["Nq"], 1).reshape(c["B"], c["Hkv"], rows, 1)
    place = torch.arange(x.shape[-1], device=x.device)
    return torch.where(place < seen, x, -math.inf), v


def _attend(s, out=False):
    c = s["case"]
    x, v = _scores(s, out)
    if not x.shape[-1]:
        x = torch.full((*x.shape[:-1], 1), -math.inf, device=x.device)
        v = v if v is None else torch.zeros((*v.shape[:2], 1, v.shape[3]), device=x.device)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).reshape(c["B"], c["H"], c["Nq"])
    if not out:
        return None, lse
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.reshape(c["B"], c["H"], c["Nq"], c["d"]).to(torch.bfloat16), lse


def _rotate(x, cos, sin, rot, layout):
    y = x.float()
    r, rest = y[..., :rot], y[..., rot:]
    if layout == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).reshape(r.shape)
    return torch.cat([r, rest], -1).to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    # Angles of far positions in 64 bits.
    angle = s["positions"].double()[:, None, :, None] * s["inv_freq"]
    cos, sin = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()
    out = {n: _rotate(s[n], cos, sin, c["rot"], c["layout"]) for n in ("q", "k")}
    if c["bwd"]:
        out.update({n: _rotate(s[n], cos, -sin, c["rot"], c["layout"]) for n in ("dq", "dk")})
    return out


def _plain_append(s):
    c = s["case"]
    B, Hkv, N, d, D = c["B"], c["Hkv"], c["N"], c["d"], _stored(c["d"])
    pad = torch.nn.functional.pad
    at = s["lens"].long()[:, None] - N + torch.arange(N, device="cuda")
    real = at >= 0
    # Each new row's values, quantised, and its bytes at their places in the pool.
    kc, ks = _quantise(pad(s["k"].float(), (0, D - d)))
    vc, vs = _quantise(pad(s["v"].float(), (0, D - d)))
    b, i = torch.nonzero(real, as_tuple=True)
    x = at[b, i]
    page, x = s["table"][b, x // PAGE].long(), x % PAGE
    p = D // 64
    at0 = (page * Hkv * 72 * D)[:, None, None] + (torch.arange(Hkv, device="cuda") * 72 * D)[None, :, None]
    x = x[:, None, None]
    ch, bl = torch.arange(D, device="cuda")[None, None], torch.arange(D // 16, device="cuda")[None, None]
    flat = s["pool"].view(-1)
    kc, ks, vc, vs = (t[b, :, i] for t in (kc, ks, vc, vs))

    def put(where, new):
        flat.scatter_(0, where.reshape(-1), new.reshape(-1))

    put(at0 + x * (D // 2) + ch[..., :D // 2], kc[..., 0::2] | (kc[..., 1::2] << 4))
    put(at0 + 32 * D + ((x % 8) * 4 + bl // p) * 8 * p + x // 8 * p + bl % p, ks)
    put(at0 + 68 * D + ((x // 2 % 4) * (D // 16) + bl) * 16 + x // 8 * 2 + x % 2, vs)
    # Two keys share a byte: the new row's half of it, and the other half from
    # the row beside it where that is new too (the next one of the same
    # sequence for an even key, the one before for an odd key).
    where, odd = at0 + 36 * D + x // 2 * D + ch, x % 2 == 1
    low = torch.where(odd, flat[where] & 15, vc)
    high = torch.where(odd, vc, flat[where] >> 4)
    if N > 1:
        after, before = torch.roll(vc, -1, 0), torch.roll(vc, 1, 0)
        low = torch.where(odd & (i > 0)[:, None, None] & real[b, (i - 1).clamp(min=0)][:, None, None], before, low)
        high = torch.where(~odd & (i < N - 1)[:, None, None], after, high)
    put(where, low | (high << 4))
    k, v = _read(s["pool"], s["table"], at[:, None].expand(B, Hkv, N), real[:, None].expand(B, Hkv, N), d)
    return {"k": k, "v": v}


def _plain_weights(s):
    c = s["case"]
    x, _ = _scores(s, False)
    lse = s["lse"].reshape(c["B"], c["Hkv"], -1, 1)
    p = torch.exp(x - torch.where(lse == -math.inf, torch.zeros_like(lse), lse))
    return {"weights": s["weights"] + p.sum(-2)[..., :c["most"]]}


def _plain_evict(s):
    c = s["case"]
    B, Hkv, keep, most = c["B"], c["Hkv"], c["keep"], c["most"]
    lens = s["lens"][:, None, None]
    place = torch.arange(most, device="cuda")[None, None]
    new = torch.clamp(s["lens"], max=keep)
    held = (place < c["sink"]) | (place >= lens - c["recent"]) | (lens <= keep)
    rank = torch.where(held, math.inf, s["weights"])
    rank = torch.where(place < lens, rank, -math.inf)
    # Stable, so that of equal weights the lowest places come first.
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :keep]
    count = torch.arange(keep, device="cuda")[None, None] < new[:, None, None]
    kept = torch.sort(torch.where(count, order, most), dim=-1)[0]
    take = torch.where(count, kept, 0)
    k, v = _read(s["pool"], s["table"], take, count.expand(B, Hkv, keep), c["d"])
    weights = torch.zeros_like(s["weights"])
    weights[..., :keep] = torch.where(count, s["weights"].gather(2, take), 0.0)
    return {"kept": torch.where(count, kept, -1).to(torch.int32), "lens": new.to(torch.int32), "weights": weights, "k": k, "v": v}


# ------------------------------------------------------------------- one pass

def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if own:
        import io_aware_attention_gb300 as fa

        if op == "rope":
            how = {"positions": s["positions"], "layout": c["layout"], "factor": s["factor"]}
            q, k = fa.rope(s["q"], s["k"], s["freqs"], **how)
            out = {"q": q, "k": k}
            if c["bwd"]:
                out["dq"], out["dk"] = fa.rope_bwd(s["dq"], s["dk"], s["freqs"], **how)
            return out
        if op == "append":
            fa.qcache_append(s["k"], s["v"], s["pool"], s["table"], s["lens"])
            k, v = fa.qcache_read(s["pool"], s["table"], s["lens"], c["N"], c["d"], newest=True)
            return {"k": k, "v": v}
        if op == "decode":
            o, lse = fa.qcache_decode(s["q"], s["pool"], s["table"], s["lens"], causal=c["causal"], scale=s["scale"])
            return {"o": o, "lse": lse}
        if op == "weights":
            return {"weights": fa.qcache_weights(s["q"], s["lse"], s["pool"], s["table"], s["lens"], s["weights"],
                                                 causal=c["causal"], scale=s["scale"])}
        kept, lens, weights = fa.qcache_evict(s["pool"], s["table"], s["lens"], s["weights"], c["keep"], sink=c["sink"],
                                              recent=c["recent"], table_out=s["table_out"])
        k, v = fa.qcache_read(s["pool"], s["table_out"], lens, c["keep"], c["d"])
        return {"kept": kept, "lens": lens, "weights": weights, "k": k, "v": v}
    if op == "rope":
        return _plain_rope(s)
    if op == "append":
        return _plain_append(s)
    if op == "decode":
        o, lse = _attend(s, out=True)
        return {"o": o, "lse": lse}
    if op == "weights":
        return _plain_weights(s)
    return _plain_evict(s)


def work(case):
    """Bytes: every input once and every output once; lengths at their mean."""
    c, op, d = case, case["op"], case["d"]
    if op == "rope":
        n = c["B"] * (c["H"] + c["Hkv"]) * c["N"] * d * (2 if c["bwd"] else 1)
        return {"bytes": 4 * n + 4 * c["B"] * c["N"], "flops": 3 * n}
    mean = c["most"] if c["B"] == 1 else (c["least"] + c["most"]) / 2
    row = 9 * _stored(d) // 16  # bytes of one stored key, and of one stored value
    if op == "append":
        n = c["B"] * c["Hkv"] * min(c["N"], max(mean, 1))
        full = c["B"] * c["Hkv"] * c["N"] * d * 4
        return {"bytes": int(n * (4 * d + 2 * row)) + full, "flops": int(n * d * 8)}
    keys = c["B"] * c["Hkv"] * mean
    if op == "evict":
        rows = c["B"] * c["Hkv"] * min(c["keep"], mean)
        values = c["B"] * c["Hkv"] * c["keep"] * 4 * (d + 1)
        return {"bytes": int(4 * keys + rows * 4 * row + values + 4 * c["B"] * c["Hkv"] * c["most"]), "flops": int(keys)}
    rows = c["B"] * c["H"] * c["Nq"]
    pairs = rows * mean
    if op == "decode":
        return {"bytes": int(keys * 2 * row + rows * (4 * d + 4)), "flops": int(pairs * 4 * d)}
    return {"bytes": int(keys * row + 8 * c["B"] * c["Hkv"] * c["most"] + rows * (2 * d + 4)), "flops": int(pairs * (2 * d + 1))}


# --------------------------------------------------------- the definition in 64 bits

def _value(pool, page, head, x, c, D, plane):
    """Stored values in 64 bits, straight from the bytes' places; page, x: rows, c: channels."""
    at = (page * pool.shape[1] + head) * (72 * D)
    flat, b, p = pool.view(-1), c // 16, D // 64
    if plane == "k":
        byte, high = at + x * (D // 2) + c // 2, c % 2
        sc = at + 32 * D + ((x % 8) * 4 + b // p) * (8 * p) + (x // 8) * p + b % p
    else:
        byte, high = at + 36 * D + (x // 2) * D + c, x % 2
        sc = at + 68 * D + (((x // 2) % 4) * (D // 16) + b) * 16 + (x // 8) * 2 + x % 2
    code = (flat[byte].long() >> (4 * high)) & 15
    mant, e = (code & 1).double(), (code >> 1) & 3
    mag = torch.where(e == 0, 0.5 * mant, (1.0 + 0.5 * mant) * torch.pow(2.0, (e - 1).double()))
    s = flat[sc].long()
    se, sm = (s >> 3) & 15, (s & 7).double()
    scale = torch.where(se == 0, sm * 2.0 ** -9, (1.0 + sm / 8.0) * torch.pow(2.0, (se - 7).double()))
    return torch.where(code >= 8, -mag, mag) * scale


def _exact_rows(s, b, head, n, plane, src=None):
    """Rows src (or the first n) of one head of one sequence."""
    D = _stored(s["case"]["d"])
    j = torch.arange(n, device="cuda") if src is None else src
    page = s["table"][b].long()[j // PAGE]
    return _value(s["pool"], page[:, None], head, (j % PAGE)[:, None], torch.arange(s["case"]["d"], device="cuda")[None], D, plane)


def _exact_round(x):
    """The stored value of each entry of x (..., d) in 64 bits."""
    d = x.shape[-1]
    y = torch.nn.functional.pad(x.double(), (0, -d % 16)).unflatten(-1, (-1, 16))
    top = (y.abs().amax(-1, keepdim=True) / 6.0).clamp(max=448.0)
    # e4m3: 8 steps to each power of two, steps of 2^-9 below 2^-6; halves to even.
    step = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -6))) - 3)
    scale = torch.round(top / step) * step
    z = torch.where(scale > 0, y / torch.where(scale > 0, scale, 1.0), 0.0).clamp(-6.0, 6.0)
    a = z.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return (torch.round(a / step) * step * torch.sign(z) * scale).flatten(-2)[..., :d]


def exact(case, seed):
    s, c = prepare(case, seed), case
    op = c["op"]
    if op == "rope":
        rot, lead = c["rot"], s["positions"].double()[:, None, :, None]
        turn = torch.complex(torch.cos(lead * s["inv_freq"]), torch.sin(lead * s["inv_freq"])) * s["factor"]

        def rotated(x, turn):
            x = x.double()
            if c["layout"] == "half":
                z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
                r = torch.cat([z.real, z.imag], -1)
            else:
                z = torch.view_as_complex(x[..., :rot].contiguous().reshape(*x.shape[:-1], rot // 2, 2)) * turn
                r = torch.view_as_real(z).flatten(-2)
            return torch.cat([r, x[..., rot:]], -1)

        out = {n: rotated(s[n], turn) for n in ("q", "k")}
        if c["bwd"]:
            out.update({n: rotated(s[n], turn.conj()) for n in ("dq", "dk")})
        return out
    lens = s["lens"].tolist()
    if op == "append":
        k, v = _exact_round(s["k"]), _exact_round(s["v"])
        for b, n in enumerate(lens):
            k[b, :, :max(0, c["N"] - n)] = 0
            v[b, :, :max(0, c["N"] - n)] = 0
        return {"k": k, "v": v}
    if op == "evict":
        shape = (c["B"], c["Hkv"], c["keep"])
        kept = torch.full(shape, -1, dtype=torch.int32, device="cuda")
        w = torch.zeros_like(s["weights"])
        k, v = (torch.zeros((*shape, c["d"]), dtype=torch.float64, device="cuda") for _ in range(2))
        for b, n in enumerate(lens):
            m = min(n, c["keep"])
            if m == 0:
                continue
            for h in range(c["Hkv"]):
                src = torch.arange(n, device="cuda")
                if n > c["keep"]:
                    low, high = c["sink"], n - c["recent"]
                    more = c["keep"] - c["sink"] - c["recent"]
                    mid = torch.sort(-s["weights"][b, h, low:high].double(), stable=True)[1][:more] + low
                    src = torch.cat([src[:low], torch.sort(mid)[0], src[high:]])
                kept[b, h, :m] = src
                w[b, h, :m] = s["weights"][b, h, src]
                k[b, h, :m] = _exact_rows(s, b, h, m, "k", src)
                v[b, h, :m] = _exact_rows(s, b, h, m, "v", src)
        return {"kept": kept, "lens": torch.clamp(s["lens"], max=c["keep"]), "weights": w.double(), "k": k, "v": v}
    if c["B"] * c["Hkv"] > 2048:
        return None
    G, Nq = c["H"] // c["Hkv"], c["Nq"]
    o = torch.zeros((c["B"], c["H"], Nq, c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["H"], Nq), -math.inf, dtype=torch.float64, device="cuda")
    w = s["weights"].double() if op == "weights" else None
    for b, n in enumerate(lens):
        if n == 0:
            continue
        for h in range(c["Hkv"]):
            k = _exact_rows(s, b, h, n, "k")
            x = torch.einsum("gqd,nd->gqn", s["q"][b, h * G:(h + 1) * G].double(), k) * s["scale"]
            if c["causal"]:
                i = torch.arange(Nq, device="cuda")[:, None]
                x = x.masked_fill(torch.arange(n, device="cuda")[None] > n - Nq + i, -math.inf)
            if op == "weights":
                given = s["lse"][b, h * G:(h + 1) * G].double()[..., None]
                w[b, h, :n] += torch.where(x == -math.inf, 0.0, torch.exp(x - given)).sum((0, 1))
                continue
            lse[b, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[b, h * G:(h + 1) * G] = torch.nan_to_num(torch.softmax(x, -1)) @ _exact_rows(s, b, h, n, "v")
    return {"weights": w} if op == "weights" else {"o": o, "lse": lse}
