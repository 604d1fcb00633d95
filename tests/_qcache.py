"""The 4-bit cache from its definition, in 64 bits on the CPU (numpy): rounding,
the bytes' places, and attention over the stored values.  Written from
include/fa.h's description; shares no code with the library."""
import numpy as np
import torch

PAGE = 64
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# e4m3 without sign: 8 steps to a power of two, steps of 2^-9 below 2^-6; 127 is NaN.
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def stored_channels(d):
    return 64 if d <= 64 else 128


def nearest_even(x, grid):
    """Index of the grid value nearest to each x >= 0; half way goes to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x, scale=1.0):
    """(codes, scale bytes) of rows x (..., d), d padded to the stored channels."""
    x = np.asarray(x, np.float64)
    D = stored_channels(x.shape[-1])
    x = np.concatenate([x, np.zeros((*x.shape[:-1], D - x.shape[-1]))], -1)
    blocks = x.reshape(*x.shape[:-1], D // 16, 16)
    top = np.minimum(np.nanmax(np.abs(np.where(np.isnan(blocks), 0, blocks)), -1) / (6.0 * scale), 448.0)
    byte = nearest_even(top, E4M3[:127])
    s = E4M3[byte][..., None] * scale
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s > 0, blocks / np.where(s > 0, s, 1.0), 0.0 * np.where(np.isfinite(blocks), blocks, 0.0))
    y = np.where(np.isnan(blocks), 6.0, y)
    code = nearest_even(np.minimum(np.abs(y), 6.0), MAGNITUDES) + 8 * ((y < 0) & (np.abs(y) > 0.25))
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def value(code, byte, scale=1.0):
    s = np.repeat(E4M3[byte & 127], 16, -1)
    return np.where(code >= 8, -1.0, 1.0) * MAGNITUDES[code & 7] * s * scale


def places(D):
    """Byte indexes in a page's block of (K code, K scale, V code, V scale)
    for key x and channel c (codes) or channel block b (scales)."""
    x = np.arange(PAGE)[:, None]
    c, b, p = np.arange(D)[None], np.arange(D // 16)[None], D // 64
    kc = x * (D // 2) + c // 2
    ks = 32 * D + ((x % 8) * 4 + b // p) * 8 * p + (x // 8) * p + b % p
    vc = 36 * D + (x // 2) * D + c + 0 * x
    vs = 68 * D + (((x // 2) % 4) * (D // 16) + b) * 16 + (x // 8) * 2 + x % 2
    return kc, ks, vc, vs


def unpack(pool, table, lens, d, k_scale=1.0, v_scale=1.0):
    """Lists over sequences of the stored k and v, (Hkv, len, d) in 64 bits."""
    pool, table, lens = (t.cpu().numpy() for t in (pool, table, lens))
    D = stored_channels(d)
    kc, ks, vc, vs = places(D)
    ks_out, vs_out = [], []
    odd_c, odd_x = (np.arange(D) % 2 == 1)[None], (np.arange(PAGE) % 2 == 1)[:, None]
    for b, n in enumerate(lens):
        rows_k, rows_v = [], []
        for slot in range(-(-int(n) // PAGE)):
            blk = pool[table[b, slot]]  # (Hkv, bytes)
            codes = np.where(odd_c, blk[:, kc] >> 4, blk[:, kc] & 15)
            rows_k.append(value(codes, blk[:, ks], k_scale))
            codes = np.where(odd_x, blk[:, vc] >> 4, blk[:, vc] & 15)
            rows_v.append(value(codes, blk[:, vs], v_scale))
        empty = np.zeros((pool.shape[1], 0, D))
        ks_out.append(np.concatenate(rows_k + [empty], 1)[:, :n, :d])
        vs_out.append(np.concatenate(rows_v + [empty], 1)[:, :n, :d])
    return ks_out, vs_out


def make_cache(lens, Hkv, d, seed, max_pages=None, spare=2, gain=1.0, k_scale=1.0, v_scale=1.0):
    """A pool on the CPU filled by the definition: pages in random order, junk
    (0xff: NaN scales) in every byte that belongs to no key.  Returns (pool,
    table, lens) tensors."""
    rng = np.random.default_rng(seed)
    D = stored_channels(d)
    pages = [-(-n // PAGE) for n in lens]
    max_pages = max(1, max(pages)) if max_pages is None else max_pages
    order = rng.permutation(sum(pages) + spare)
    pool = np.full((len(order), Hkv, 72 * D), 0xFF, np.uint8)
    table = np.full((len(lens), max_pages), -7, np.int32)  # entries past the last page are not read
    kc, ks, vc, vs = places(D)
    at = 0
    for b, n in enumerate(lens):
        for slot in range(pages[b]):
            page = order[at]
            at += 1
            table[b, slot] = page
            m = min(PAGE, n - slot * PAGE)
            for plane, scale in (("k", k_scale), ("v", v_scale)):
                x = rng.standard_normal((Hkv, m, d)) * gain * scale
                x = torch.tensor(x).to(torch.bfloat16).double().numpy()
                code, byte = quantise(x, scale)
                blk = pool[page]
                if plane == "k":
                    blk[:, kc[:m, 0::2]] = code[..., 0::2] | (code[..., 1::2] << 4)
                    blk[:, ks[:m]] = byte
                else:
                    for r in range(m):
                        old = blk[:, vc[r]]
                        blk[:, vc[r]] = (old & 0xF0 | code[:, r]) if r % 2 == 0 else (old & 0x0F | (code[:, r] << 4))
                    blk[:, vs[:m]] = byte
    return torch.from_numpy(pool), torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32)


def attention(q, ks, vs, causal, scale):
    """o, lse, and what bounds the kernels' errors, per query row in 64 bits:
    sum |p v| (like o) and the largest scale * sum |q k| of a row."""
    q = q.double().cpu().numpy()
    B, H, Nq, d = q.shape
    o, mag = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full((B, H, Nq), -np.inf), np.zeros((B, H, Nq))
    for b in range(B):
        Hkv, n, _ = ks[b].shape
        for h in range(H):
            k, v = ks[b][h * Hkv // H], vs[b][h * Hkv // H]
            for i in range(Nq):
                m = max(0, n - Nq + i + 1) if causal else n
                if m == 0:
                    continue
                s = scale * (k[:m] @ q[b, h, i])
                top = s.max()
                e = np.exp(s - top)
                lse[b, h, i] = top + np.log(e.sum())
                p = e / e.sum()
                o[b, h, i], mag[b, h, i] = p @ v[:m], p @ np.abs(v[:m])
                big[b, h, i] = scale * (np.abs(k[:m]) @ np.abs(q[b, h, i])).max()
    return o, lse, mag, big


def gathered(q, lse, ks, causal, scale, W):
    """The weight each key receives, (B, Hkv, W), and a bound on its relative error's driver."""
    q, lse = q.double().cpu().numpy(), lse.double().cpu().numpy()
    B, H, Nq, d = q.shape
    Hkv = ks[0].shape[0]
    w, err = np.zeros((B, Hkv, W)), np.zeros((B, Hkv, W))
    for b in range(B):
        n = ks[b].shape[1]
        for h in range(H):
            k = ks[b][h * Hkv // H]
            for i in range(Nq):
                m = min(W, max(0, n - Nq + i + 1) if causal else n)
                if m <= 0 or lse[b, h, i] == -np.inf:
                    continue
                e = np.exp(scale * (k[:m] @ q[b, h, i]) - lse[b, h, i])
                w[b, h * Hkv // H, :m] += e
                err[b, h * Hkv // H, :m] += e * (scale * (np.abs(k[:m]) @ np.abs(q[b, h, i])) + abs(lse[b, h, i]) + 1)
    return w, err
