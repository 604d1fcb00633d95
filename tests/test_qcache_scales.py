"""Rounding into the 4-bit cache with tensor scales that are no powers of two: every block's
scale is the nearest e4m3 and every code the nearest, with values placed beside the borders.

A quotient x / (e4m3 * scale) next to a border between two codes is made by taking x, a bf16 number, and the scale
as the fp32 number nearest to x / (border * e4m3) and its neighbours: the quotient then lies within 2^-23 of the border, on
either side.  The expected codes are found with whole numbers, so nothing is rounded on the way."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
from test_serve_abi import append, decode, lib, needs_lib, read, weights  # noqa: F401  (lib is a fixture)

GRID = [Fraction(m) for m in ref.MAGNITUDES.tolist()]
E4M3 = [Fraction(m) for m in ref.E4M3[:127].tolist()]


def nearest(x, grid):
    """Index of the grid value nearest to x >= 0, half way to the even index, above the last to the last."""
    lo = max(i for i, g in enumerate(grid) if g <= x)
    if lo + 1 == len(grid):
        return lo
    down, up = x - grid[lo], grid[lo + 1] - x
    return lo if down < up or (down == up and lo % 2 == 0) else lo + 1


def expected(row, scale):
    """(signed codes' values, scale byte) of one block of 16 numbers with the tensor's scale (a float32)."""
    xs, s = [Fraction(float(x)) for x in row], Fraction(float(scale))
    byte = nearest(min(max(abs(x) for x in xs) / (6 * s), E4M3[-1]), E4M3)
    unit = E4M3[byte] * s
    codes = [0 if unit == 0 else (-1 if x < 0 else 1) * GRID[nearest(min(abs(x) / unit, 6), GRID)] for x in xs]
    return [float(c) for c in codes], byte


def test_expected_codes_on_the_cpu():
    codes, byte = expected([6, -6, 4, 3, 2, 1.5, 1, 0.5, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25], 1.0)
    assert codes == [6, -6, 4, 3, 2, 1.5, 1, 0.5, 0, 1, 1, 2, 2, 4, 4, 0] and ref.E4M3[byte] == 1.0


def bf16(x):
    return float(torch.tensor(x).to(torch.bfloat16))


def beside_borders(seed):
    """(scale, block of 16) pairs: the scale puts one of the block's numbers within fp32's last place of a border."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(40):
        base = bf16(float(rng.uniform(0.5, 4.0)))
        border = float(rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]))
        unit = float(ref.E4M3[rng.integers(40, 80)])
        near = np.float32(base / (border * unit))
        for step in (-2, -1, 0, 1, 2):
            scale = near
            for _ in range(abs(step)):
                scale = np.nextafter(scale, np.float32(np.inf if step > 0 else 0), dtype=np.float32)
            block = [base, -base] + [bf16(float(rng.standard_normal()) * unit * float(scale)) for _ in range(13)]
            block.append(bf16(6 * unit * float(scale)))  # the largest: this unit, or one beside it
            out.append((scale, block))
        # A border of the block's own scale: the largest number is 6 * scale * (half way between two e4m3 numbers).
        i = int(rng.integers(30, 90))
        half = (float(ref.E4M3[i]) + float(ref.E4M3[i + 1])) / 2
        near = np.float32(base / (6 * half))
        for step in (-1, 0, 1):
            scale = near if step == 0 else np.nextafter(near, np.float32(np.inf if step > 0 else 0), dtype=np.float32)
            out.append((scale, [base] + [bf16(float(rng.uniform(-base, base))) for _ in range(15)]))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_every_code_is_the_nearest(seed):
    d, pool, table = 16, fa.qcache_pool(1, 1, 16), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    kc, ks, vc, vs = ref.places(64)
    for scale, block in beside_borders(seed):
        x = torch.tensor(block).to(torch.bfloat16).reshape(1, 1, 1, d)
        fa.qcache_append(x.cuda(), x.flip(3).contiguous().cuda(), pool, table, lens, scale, scale)
        blk = pool[0, 0].cpu().numpy()
        codes, byte = expected(x.flatten().tolist(), scale)
        k = np.where(np.arange(d) % 2 == 1, blk[kc[0, :d]] >> 4, blk[kc[0, :d]] & 15)
        v = (blk[vc[0, :d]] & 15)[::-1]
        for name, got, at in (("k", k, ks), ("v", v, vs)):
            assert blk[at[0, 0]] == byte, (name, scale, block)
            values = np.where(got >= 8, -1.0, 1.0) * ref.MAGNITUDES[got & 7]
            assert (values == np.array(codes)).all(), (name, scale, block)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.013, 7.3, 1 / 3, 2.0 ** -5, 1e-9, 3e9])
@pytest.mark.parametrize("d", [64, 104])
def test_random_rows(scale, d):
    """Many rows at once; the 64-bit quotients of random bf16 numbers decide (none lies on a border unless exactly)."""
    B, Hkv, N = 2, 2, 150
    g = torch.Generator("cpu").manual_seed(d)
    scale = float(np.float32(scale))
    k, v = ((torch.randn((B, Hkv, N, d), generator=g) * torch.exp(torch.randn((B, Hkv, N, 1), generator=g)) * scale * 3).to(torch.bfloat16)
            for _ in range(2))
    pool, table = fa.qcache_pool(B * 3, Hkv, d), torch.arange(B * 3, dtype=torch.int32, device="cuda").reshape(B, 3)
    lens = torch.full((B,), N, dtype=torch.int32, device="cuda")
    fa.qcache_append(k.cuda(), v.cuda(), pool, table, lens, scale, scale)
    got_k, got_v = ref.unpack(pool, table, lens, d, scale, scale)
    for b in range(B):
        for x, got in ((k, got_k), (v, got_v)):
            assert np.array_equal(got[b], ref.value(*ref.quantise(x[b].double().numpy(), scale), scale)[..., :d])


@needs_lib
@pytest.mark.parametrize("scale, refused", [(2.0 ** -61, True), (2.0 ** 61, True), (1e-45, True), (3e38, True), (2.0 ** -60, False),
                                            (2.0 ** 60, False)])
def test_scales_out_of_range_are_refused(lib, scale, refused):  # noqa: F811
    if torch.cuda.is_available() and not refused:
        pytest.skip("a GPU is present: the call would run on fake addresses")
    ok = (1,) if refused else (2, 3)  # (2, 3: no device)
    for which in ("k_scale", "v_scale"):
        assert append(lib, **{which: scale}) in ok and read(lib, **{which: scale}) in ok
        assert decode(lib, **{which: scale}) in ok
    assert weights(lib, k_scale=scale) in ok
