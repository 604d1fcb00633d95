"""Rotary positions (fa_rope) and their gradient against the formula in 64 bits.

Tolerance: results are rounded to bf16 once (2^-8 of the result), and before
that carry fp32 errors: cosine and sine good to 2^-21.1 (what CUDA documents for
__sinf and __cosf on [-pi, pi]), an angle of at most pi rounded twice to 24 bits
(2 pi 2^-25 = 2^-22.3), and the roundings of two products and a sum (3 * 2^-24 =
2^-22.4): 0.45 + 0.20 + 0.18 = 0.83 of 2^-20 times factor * (|a| + |b|).
"""
import math

import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

gpu = pytest.mark.gpu


def reference(x, inv_freq, pos, layout, factor, inverse=False):
    """x (B, H, N, d) and pos (B, N) -> the turned rows and |a| + |b| of each channel's pair, float64."""
    x = x.double().cpu()
    rot = 2 * len(inv_freq)
    angle = pos.double().cpu()[:, None, :, None] * torch.tensor(inv_freq, dtype=torch.float64)
    c, s = torch.cos(angle) * factor, torch.sin(angle) * factor * (-1 if inverse else 1)
    y, mag = x.clone(), x.abs()
    one, two = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = a * c - b * s, b * c + a * s
    mag[..., one] = mag[..., two] = (a.abs() + b.abs()) * abs(factor)
    return y, mag


def check(got, want, mag, what=""):
    err = (got.double().cpu() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * mag).all(), f"{what}: {err.max().item()}"


def freqs_of(inv_freq):
    out = []
    for f in inv_freq:
        u = int(round(f / (2 * math.pi) * 2 ** 64)) & (2 ** 64 - 1)
        out.append(u - 2 ** 64 if u >= 2 ** 63 else u)
    return torch.tensor(out, dtype=torch.int64)


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)).to(torch.bfloat16)


# ------------------------------------------------------------------ frequencies

def turns(freqs):
    return (freqs.numpy().astype(np.uint64).astype(np.float64) / 2.0 ** 64)


def test_frequencies_on_the_cpu():
    plain, f = fa.rope_frequencies(64, base=10000.0, device="cpu")
    assert f == 1.0 and plain.dtype == torch.int64 and plain.shape == (32,)
    want = 10000.0 ** (-np.arange(32) / 32) / (2 * np.pi)
    assert np.allclose(turns(plain), want, rtol=1e-14, atol=0)
    linear, f = fa.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert f == 1.0 and np.allclose(turns(linear), want / 4, rtol=1e-14, atol=0)
    base, f = fa.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert f == 1.0 and np.isclose(turns(base)[0], want[0]) and np.isclose(turns(base)[-1], want[-1] / 4)
    parts, f = fa.rope_frequencies(64, scaling="parts", factor=4.0, original_length=4096, device="cpu")
    assert np.isclose(f, 0.1 * math.log(4.0) + 1)
    made = 4096 * want
    assert np.allclose(turns(parts)[made >= 32], want[made >= 32], rtol=1e-14)
    assert np.allclose(turns(parts)[made <= 1], want[made <= 1] / 4, rtol=1e-14)
    between = (made > 1) & (made < 32)
    assert between.any() and (turns(parts)[between] < want[between]).all() and (turns(parts)[between] > want[between] / 4).all()


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=64, base=0.5), dict(rot=64, scaling="no"),
                                dict(rot=64, scaling="linear", factor=0.5), dict(rot=64, scaling="parts", factor=2.0)])
def test_bad_frequencies_are_refused(kw):
    with pytest.raises(ValueError):
        fa.rope_frequencies(device="cpu", **kw)


# ------------------------------------------------------------------------- GPU

@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d, rot", [(128, 128), (64, 64), (128, 32), (80, 40), (80, 48), (96, 96), (72, 72), (8, 8), (8, 2),
                                    (128, 126), (40, 24), (24, 16), (80, 36), (80, 38)])
@pytest.mark.parametrize("B, H, Hk, N", [(1, 1, 1, 1), (2, 5, 3, 37), (3, 16, 2, 130)])
def test_rope_and_gradient(layout, d, rot, B, H, Hk, N):
    inv = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    g = torch.Generator("cpu").manual_seed(d + rot + N)
    pos = torch.randint(0, 300000, (B, N), generator=g, dtype=torch.int32)
    q, k = rand((B, H, N, d), 1), rand((B, Hk, N, d), 2)
    factor = 1.2
    how = dict(positions=pos.cuda(), layout=layout, factor=factor)
    for inverse in (False, True):
        call = fa.rope_bwd if inverse else fa.rope
        qo, ko = call(q.cuda(), k.cuda(), freqs_of(inv).cuda(), **how)
        torch.cuda.synchronize()
        for got, x in ((qo, q), (ko, k)):
            check(got, *reference(x, inv, pos, layout, factor, inverse), f"d{d} rot{rot} inverse {inverse}")
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])  # channels past rot are copied


@gpu
def test_gradient_by_differences():
    """The map is linear: <dq', rope(x + h e) - rope(x - h e)> / 2h = <rope_bwd(dq'), e>, on values whose
    steps are exact, within the roundings of the two results (2^-8 of each entry)."""
    B, H, N, d = 1, 2, 5, 16
    freqs, _ = fa.rope_frequencies(d, base=100.0)
    x = (torch.randint(-8, 9, (B, H, N, d), generator=torch.Generator().manual_seed(3)) / 8).to(torch.bfloat16)
    up = rand((B, H, N, d), 4)
    grad, _ = fa.rope_bwd(up.cuda(), None, freqs)
    h = 0.5
    for c in range(d):
        e = torch.zeros(d)
        e[c] = h
        hi, _ = fa.rope((x + e).to(torch.bfloat16).cuda(), None, freqs)
        lo, _ = fa.rope((x - e).to(torch.bfloat16).cuda(), None, freqs)
        diff = ((hi.double() - lo.double()).cpu() * up.double()).sum(-1) / (2 * h)
        slack = 2.0 ** -8 * ((hi.double().abs() + lo.double().abs()).cpu() * up.double().abs()).sum(-1) / (2 * h)
        got = grad[..., c].double().cpu()
        assert ((diff - got).abs() <= slack + 2.0 ** -8 * got.abs() + 1e-6).all()


@gpu
def test_positions_forms_agree():
    """int32, int64, shared, and lengths give the same turn; without either, rows stand at 0, 1, ...; far and
    negative positions keep their angles."""
    B, H, N, d = 3, 4, 9, 64
    inv = [10000.0 ** (-2 * i / d) for i in range(d // 2)]
    f = freqs_of(inv).cuda()
    q = rand((B, H, N, d), 5)
    lens = torch.tensor([9, 100, 4], dtype=torch.int32)
    pos = lens[:, None].long() - N + torch.arange(N)[None]
    a, _ = fa.rope(q.cuda(), None, f, lens=lens.cuda())
    b, _ = fa.rope(q.cuda(), None, f, positions=pos.cuda())
    c, _ = fa.rope(q.cuda(), None, f, positions=pos.to(torch.int32).cuda())
    assert torch.equal(a, b) and torch.equal(a, c)
    check(a, *reference(q, inv, pos, "half", 1.0))
    one = torch.arange(N)
    d0, _ = fa.rope(q.cuda(), None, f)
    d1, _ = fa.rope(q.cuda(), None, f, positions=one.cuda())
    d2, _ = fa.rope(q.cuda(), None, f, positions=one[None].expand(B, N).cuda())
    assert torch.equal(d0, d1) and torch.equal(d0, d2)
    far = torch.tensor([2 ** 31 - 1, 10 ** 7, -(10 ** 6)], dtype=torch.int64)[:, None] + torch.zeros(N, dtype=torch.int64)
    got, _ = fa.rope(q.cuda(), None, f, positions=far.cuda())
    # The reference's own angle t * f is rounded to 53 bits: 2^31 * 2^-53 is far below the tolerance.
    check(got, *reference(q, inv, far, "half", 1.0))


@gpu
@pytest.mark.parametrize("rot, layout", [(64, "half"), (40, "interleaved"), (36, "half")])
def test_views_of_a_fused_projection_and_in_place(rot, layout):
    """q and k as strided views of one (B, N, 3, H, d) tensor, into new tensors and in place; v is not touched."""
    B, N, H, d = 2, 33, 6, 64
    qkv = rand((B, N, 3, H, d), 6).cuda()
    f = freqs_of([100.0 ** (-2 * i / rot) for i in range(rot // 2)]).cuda()
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    qo, ko = fa.rope(q, k, f, layout=layout)
    q2, k2 = fa.rope(q.contiguous(), k.contiguous(), f, layout=layout)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    before = qkv.clone()
    fa.rope_into(q, k, q, k, f, layout=layout)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, :, 2], before[:, :, 2])


@gpu
def test_unaligned_rows_and_repeated_inputs():
    """Rows that start off 16 bytes, and an input expanded over heads (stride 0)."""
    B, H, N, d = 2, 3, 17, 64
    f, _ = fa.rope_frequencies(d)
    for off in (1, 2, 3, 4):
        buf = rand((B * H * N * d + off,), 7).cuda()
        q = buf[off:].view(B, H, N, d)
        got, _ = fa.rope(q, None, f)
        want, _ = fa.rope(q.clone(), None, f)
        assert torch.equal(got, want)
    one = rand((B, 1, N, d), 8).cuda()
    got, _ = fa.rope(one.expand(B, H, N, d), None, f)
    want, _ = fa.rope(one.expand(B, H, N, d).contiguous(), None, f)
    assert torch.equal(got, want)
    with pytest.raises(fa.FaError):  # an output may not repeat a place
        fa.rope_into(q, None, one.expand(B, H, N, d), None, f)


@gpu
def test_forward_then_gradient_is_the_identity_times_factor_squared():
    B, H, N, d = 1, 3, 64, 128
    f, factor = fa.rope_frequencies(d, scaling="parts", factor=8.0, original_length=512)
    q = rand((B, H, N, d), 9)
    y, _ = fa.rope(q.cuda(), None, f, factor=factor)
    z, _ = fa.rope_bwd(y, None, f, factor=factor)
    want = q.double() * factor ** 2
    mag = (q.double().abs() + torch.roll(q.double().abs(), d // 2, -1)) * factor ** 2
    # y's rounding (2^-8 of |y| <= factor (|a| + |b|)) passes through the second turn by both its terms.
    assert ((z.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 2 * 2.0 ** -8 * mag + 1e-6).all()


@gpu
def test_infinities_and_nan_stay_in_their_pair():
    d = 64
    f, _ = fa.rope_frequencies(d)
    q = torch.ones((1, 1, 3, d), dtype=torch.bfloat16)
    q[0, 0, 1, 5], q[0, 0, 2, 40] = float("inf"), float("nan")
    got, _ = fa.rope(q.cuda(), None, f)
    bad = ~torch.isfinite(got[0, 0].cpu())
    assert not bad[0].any()
    assert bad[1].nonzero().flatten().tolist() == [5, 37] and bad[2].nonzero().flatten().tolist() == [8, 40]
