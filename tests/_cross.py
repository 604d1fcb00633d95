"""Cross attention in 64 bits, with bounds on what the kernels' roundings may add.

The kernels round each probability (and each entry of dS) to bf16 once before it
meets a matrix product, and each result once: a half step of bf16 is 2^-8 of the
value.  Scores are fp32 sums of d products (an error of at most d 2^-24 of the
sum of magnitudes, and as much again for the order), their exponentials good to
2^-21 and a few units in the argument's last place; ETA covers these per unit
of the largest sum of magnitudes.
"""
import math

import torch

HALF = 2.0 ** -8


def slack(q, k, scale):
    """A bound on a probability's relative error before its rounding, (B, H, Nq, 1)."""
    d = q.shape[-1]
    g = q.shape[1] // k.shape[1]
    big = torch.einsum("bhnd,bhmd->bhnm", q.abs(), k.abs().repeat_interleave(g, 1)).amax(-1, keepdim=True)
    return (2 * d + 8) * 2.0 ** -24 * scale * big + 2.0 ** -19


def reference(q, k, v, lens, scale, do=None):
    """fp64 (o, lse) and, given do, (dq, dk, dv); with them bounds on the kernels' errors.

    lens: a list of key counts.  Rows of k and v from there on are not read."""
    q, k, v = (t.double() for t in (q, k, v))
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1:3]
    g = H // Hkv
    real = torch.arange(Nk, device=q.device)[None] < torch.tensor(lens, device=q.device)[:, None]
    k, v = (torch.where(real[:, None, :, None], t, 0.0) for t in (k, v))
    kk, vv = (t.repeat_interleave(g, 1) for t in (k, v))
    s = scale * torch.einsum("bhnd,bhmd->bhnm", q, kk)
    s = s.masked_fill(~real[:, None, None], -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(real[:, None, None], torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    o = p @ vv
    eta = slack(q, k, scale)
    a = p @ vv.abs()
    # sum p~ v / sum p~ is off by at most sum p |eps| |v - o|, then one rounding.
    tol_o = (HALF + 2 * eta) * (a + o.abs()) + HALF * o.abs() + 1e-30
    tol_lse = eta[..., 0] + 2.0 ** -20 * (1 + lse.abs().nan_to_num(posinf=0.0))
    out = {"o": (o, tol_o), "lse": (lse, tol_lse)}
    if do is None:
        return out
    do = do.double()
    dp = do @ vv.transpose(-1, -2)
    dd = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - dd)
    # D comes from the rounded o; dP is an fp32 sum.
    off_d = (do.abs() * tol_o).sum(-1, keepdim=True) + 2.0 ** -20 * (do.abs() * o.abs()).sum(-1, keepdim=True)
    off_dp = 2.0 ** -20 * (do.abs() @ vv.abs().transpose(-1, -2))
    off_p = HALF + 2 * eta + tol_lse[..., None]
    off_s = off_p * ds.abs() + p * (off_d + off_dp) * (1 + HALF)

    def grouped(t):
        return t.reshape(B, Hkv, g, *t.shape[2:]).sum(2)

    dv = grouped(p.transpose(-1, -2) @ do)
    dv_off = grouped((off_p * p).transpose(-1, -2) @ do.abs())
    dk = grouped(scale * ds.transpose(-1, -2) @ q)
    dk_off = grouped(scale * off_s.transpose(-1, -2) @ q.abs())
    dq = scale * ds @ kk
    dq_off = scale * off_s @ kk.abs()
    # fp32 sums over the rows (or keys) on top.
    for name, x, off in (("dq", dq, dq_off), ("dk", dk, dk_off), ("dv", dv, dv_off)):
        out[name] = (x, 1.02 * off + HALF * x.abs() + 1e-30)
    return out


def check(got, want, what=""):
    x, tol = want
    got = got.double()
    assert torch.equal(torch.isinf(got), torch.isinf(x)), f"{what}: infinities differ"
    bad = torch.where(torch.isinf(x), 0.0, (got - x).abs() / tol)
    worst = bad.max().item()
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound at {divmod(int(bad.argmax()), x.shape[-1])}"
    return worst


def fused_states(B, Hkv, Nk, d, gen, device="cuda"):
    """k and v as views of one buffer (B, Nk, 2, Hkv, d)."""
    kv = torch.randn((B, Nk, 2, Hkv, d), generator=gen, device=device).to(torch.bfloat16)
    return kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
