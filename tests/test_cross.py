"""Cross attention (fa_cross_fwd, fa_cross_bwd) against 64 bits: lengths from one
row to many tiles on either side, grouped heads, padding that holds NaN,
sequences without keys, views, split key ranges, more sequences than a launch
holds, streams and graphs."""
import math

import pytest
import torch

import io_aware_attention_gb300 as fa

from _cross import check, fused_states, reference

pytestmark = pytest.mark.gpu


def draw(B, H, Hkv, Nq, Nk, d, lens, seed, fused=True, mult=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    q = (torch.randn((B, H, Nq, d), generator=gen, device="cuda") * mult).to(torch.bfloat16)
    k, v = fused_states(B, Hkv, Nk, d, gen)
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    do = torch.randn((B, H, Nq, d), generator=gen, device="cuda").to(torch.bfloat16)
    if lens is not None:
        pad = torch.arange(Nk, device="cuda")[None] >= torch.tensor(lens, device="cuda")[:, None]
        k.masked_fill_(pad[:, None, :, None], math.nan)
        v.masked_fill_(pad[:, None, :, None], math.inf)
    return q, k, v, do


def device_lens(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")


def run_all(q, k, v, do, lens, scale=None):
    n = device_lens(lens)
    o, lse = fa.cross_fwd(q, k, v, n, scale)
    dq, dk, dv = fa.cross_bwd(q, k, v, o, lse, do, n, scale)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def compare(q, k, v, do, lens, got, scale=None):
    B, Nk = q.shape[0], k.shape[2]
    want = reference(q, k, v, lens or [Nk] * B, scale or q.shape[-1] ** -0.5, do)
    for name in got:
        check(got[name], want[name], name)


@pytest.mark.parametrize("d", [64, 128, 8, 40, 72, 120])
@pytest.mark.parametrize("Nq, Nk", [(1, 1), (1, 300), (2, 127), (63, 129), (64, 64), (129, 1), (128, 257), (300, 520)])
def test_lengths(d, Nq, Nk):
    args = draw(2, 4, 2, Nq, Nk, d, None, Nq * 1000 + Nk + d)
    compare(*args, None, run_all(*args, None))


# Key counts around every border that the kernels treat apart: products of 16 keys,
# halves of 64, tiles of 128, and none at all.
@pytest.mark.parametrize("d", [64, 128, 48, 88])
@pytest.mark.parametrize("lens", [[0, 1, 15], [16, 17, 63], [64, 65, 79], [80, 81, 111], [127, 128, 129], [191, 192, 193],
                                  [0, 0, 0], [208, 255, 256], [257, 300, 0]])
def test_padding(d, lens):
    args = draw(3, 6, 2, 70, 300, d, lens, sum(lens) + d)
    compare(*args, lens, run_all(*args, lens))


@pytest.mark.parametrize("H, Hkv", [(1, 1), (5, 5), (6, 1), (8, 2), (14, 2)])
@pytest.mark.parametrize("fused", [False, True])
def test_groups(H, Hkv, fused):
    lens = [200, 77]
    args = draw(2, H, Hkv, 90, 200, 64, lens, H * 10 + Hkv, fused)
    compare(*args, lens, run_all(*args, lens))


# One query row against long keys: the key range is split, parts of short sequences hold nothing.
@pytest.mark.parametrize("d", [64, 128, 80])
@pytest.mark.parametrize("B, H, Hkv, Nq, Nk, lens", [
    (1, 1, 1, 1, 20000, None), (2, 8, 2, 1, 5000, [5000, 3]), (4, 4, 4, 3, 3001, [0, 1, 128, 3001]),
    (1, 16, 16, 1, 1500, [1400]), (3, 8, 1, 16, 4097, [4097, 129, 0])])
def test_split_keys(d, B, H, Hkv, Nq, Nk, lens):
    args = draw(B, H, Hkv, Nq, Nk, d, lens, Nk + d)
    assert fa.cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d) > 0
    compare(*args, lens, run_all(*args, lens))


# Many queries against few keys: the query blocks of a key block are cut into parts.
@pytest.mark.parametrize("d", [64, 128, 40])
@pytest.mark.parametrize("B, H, Hkv, Nq, Nk, lens", [
    (1, 1, 1, 2000, 1, None), (1, 8, 1, 300, 77, [70]), (2, 6, 2, 700, 200, [200, 5]), (3, 4, 4, 513, 130, [0, 129, 128]),
    (2, 14, 2, 111, 90, [0, 0])])
def test_queries_in_parts(d, B, H, Hkv, Nq, Nk, lens):
    args = draw(B, H, Hkv, Nq, Nk, d, lens, Nq + d)
    rows = B * H * -(-Nq // 64) * 64
    assert fa.cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d) > rows * ((64 if d <= 64 else 128) + 2) * 4
    compare(*args, lens, run_all(*args, lens))
    apart = (args[0].transpose(1, 2).contiguous().transpose(1, 2), *args[1:])  # heads that do not run as one
    compare(*args, lens, run_all(*apart, lens))


def test_more_sequences_than_a_launch_holds():
    B = 600
    lens = [(7 * b) % 41 for b in range(B)]
    args = draw(B, 2, 1, 3, 40, 64, lens, 5)
    compare(*args, lens, run_all(*args, lens))


def test_unequal_lengths_over_many_rounds():
    lens = [1000, 3, 517, 999, 0, 640, 128, 129, 1, 831]
    args = draw(10, 12, 4, 700, 1000, 128, lens, 6)
    compare(*args, lens, run_all(*args, lens))


# Large scores: one key takes nearly all the weight, maxima rise from tile to tile.
@pytest.mark.parametrize("d", [64, 128])
def test_rising_scores(d):
    q, k, v, do = draw(1, 2, 2, 130, 900, d, None, 8, False, 4.0)
    k = (k.float() * torch.linspace(0.1, 3.0, 900, device="cuda")[:, None]).to(torch.bfloat16)
    compare(q, k, v, do, None, run_all(q, k, v, do, None))


def test_views_of_queries_and_results():
    """(B, N, H, d) tensors, their transposes taken as they are and written as they are."""
    B, H, Hkv, Nq, Nk, d = 2, 6, 2, 37, 150, 64
    lens = [150, 90]
    q, k, v, do = draw(B, H, Hkv, Nq, Nk, d, lens, 9)
    want = run_all(q, k, v, do, lens)
    turn = lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    qt, dot = turn(q), turn(do)
    o, dq = (torch.full((B, Nq, H, d), math.nan, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    lse = torch.full((B, H, Nq), math.nan, device="cuda")
    dkv = torch.full((B, Nk, 2, Hkv, d), math.nan, dtype=torch.bfloat16, device="cuda")
    dk, dv = dkv[:, :, 0].transpose(1, 2), dkv[:, :, 1].transpose(1, 2)
    n = device_lens(lens)
    ws = torch.empty(max(16, fa.cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)), dtype=torch.uint8, device="cuda")
    fa.cross_fwd_into(qt, k, v, o, lse, ws, n)
    ws = torch.empty(fa.cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d), dtype=torch.uint8, device="cuda")
    fa.cross_bwd_into(qt, k, v, o, lse, dot, dq, dk, dv, ws, n)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    compare(q, k, v, do, lens, {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv})
    assert torch.equal(o, want["o"]) and torch.equal(lse, want["lse"])


def test_one_row_views():
    """One row of every head of a fused projection (B, 1, H d): heads are rows at one stride."""
    B, H, Hkv, Nk, d = 3, 8, 2, 260, 128
    q, k, v, do = draw(B, H, Hkv, 1, Nk, d, None, 10)
    qv = q.transpose(1, 2).reshape(B, 1, H * d).reshape(B, 1, H, d).transpose(1, 2)
    compare(q, k, v, do, None, run_all(qv, k, v, do, None))


def test_places_beyond_32_bits():
    """Batches 2^31 elements apart, in what is read and in what is written."""
    B, H, Hkv, Nq, Nk, d = 2, 4, 2, 40, 150, 64
    lens = [150, 77]
    q, k, v, do = draw(B, H, Hkv, Nq, Nk, d, lens, 31)
    want = run_all(q, k, v, do, lens)
    wide = [torch.empty((1 << 31) + (1 << 20), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    at = [0] * 4  # (an output shares a buffer with no other tensor, but dk with dv)

    def far(side, like, fill):
        """A view of one of the wide buffers, its batches 2^31 elements apart."""
        b, h, n, c = like.shape
        t = wide[side][at[side]:].as_strided((b, h, n, c), (1 << 31, n * c, c, 1))
        at[side] += h * n * c
        if fill:
            t.copy_(like)
        return t

    n = device_lens(lens)
    q2, k2, v2, do2 = (far(0, t, True) for t in (q, k, v, do))
    o2, dq2, dk2, dv2 = (far(side, t, False) for side, t in ((1, q), (2, q), (3, k), (3, v)))
    lse = torch.empty((B, H, Nq), device="cuda")
    ws = torch.empty(max(16, fa.cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)), dtype=torch.uint8, device="cuda")
    fa.cross_fwd_into(q2, k2, v2, o2, lse, ws, n)
    ws = torch.empty(fa.cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d), dtype=torch.uint8, device="cuda")
    fa.cross_bwd_into(q2, k2, v2, o2, lse, do2, dq2, dk2, dv2, ws, n)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    assert torch.equal(o2, want["o"]) and torch.equal(lse, want["lse"])
    compare(q, k, v, do, lens, {"o": o2, "lse": lse, "dq": dq2, "dk": dk2, "dv": dv2})


def test_expanded_states():
    """Beams share one encoder's states: batch stride 0; a shared head: head stride 0."""
    gen = torch.Generator("cuda").manual_seed(11)
    k, v = fused_states(1, 2, 333, 64, gen)
    k, v = k.expand(4, 2, 333, 64), v[:, :1].expand(4, 2, 333, 64)
    q, do = (torch.randn((4, 4, 20, 64), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    lens = [333, 1, 200, 128]
    compare(q, k, v, do, lens, run_all(q, k, v, do, lens))


def test_expanded_gradient():
    """The gradient of a sum: dO is one row, expanded over heads and batches."""
    q, k, v, _ = draw(2, 4, 2, 50, 80, 128, None, 12)
    do = torch.randn((1, 1, 50, 128), device="cuda").to(torch.bfloat16).expand(2, 4, 50, 128)
    compare(q, k, v, do, None, run_all(q, k, v, do, None))


def test_differences():
    """The gradient against differences of the 64-bit loss along random directions."""
    lens = [60, 33]
    q, k, v, do = draw(2, 4, 2, 40, 60, 64, lens, 13)
    got = run_all(q, k, v, do, lens)
    scale = 64 ** -0.5
    real = (torch.arange(60, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None])[:, None, :, None]
    base = {"q": q.double(), "k": torch.where(real, k.double(), 0.0), "v": torch.where(real, v.double(), 0.0)}
    want = reference(q, k, v, lens, scale, do)

    def loss(x):
        return (reference(x["q"], x["k"], x["v"], lens, scale)["o"][0] * do.double()).sum()

    gen = torch.Generator("cuda").manual_seed(14)
    for name in base:
        u = torch.randn(base[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        if name != "q":
            u = torch.where(real, u, 0.0)
        h = 1e-5
        diff = (loss({**base, name: base[name] + h * u}) - loss({**base, name: base[name] - h * u})) / (2 * h)
        tol = (want["d" + name][1] * u.abs()).sum() + 1e-6 * diff.abs() + 1e-6
        assert (diff - (got["d" + name].double() * u).sum()).abs() <= tol, name


def test_runs_agree():
    """The forward, dk and dv do not depend on timing; nor does the forward on what else the batch holds."""
    lens = [700, 300, 0, 128]
    args = draw(4, 8, 2, 65, 700, 128, lens, 15)
    a, b = run_all(*args, lens), run_all(*args, lens)
    for name in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[name], b[name]), name


def test_length_beyond_the_states_is_reported():
    q, k, v, do = draw(2, 2, 2, 5, 50, 64, None, 16)
    n = torch.tensor([51, -3], dtype=torch.int32, device="cuda")
    o, lse = fa.cross_fwd(q, k, v, n)
    assert fa.check_device_status() == 1
    grads = fa.cross_bwd(q, k, v, o, lse, do, n)
    assert fa.check_device_status() == 1
    compare(q, k, v, do, [50, 0], dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *grads))))


def test_streams():
    lens = [400, 150]
    args = draw(2, 4, 2, 33, 400, 64, lens, 17)
    want = run_all(*args, lens)
    q, k, v, do = args
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = device_lens(lens)
    side.wait_stream(torch.cuda.current_stream())
    o, lse = fa.cross_fwd(q, k, v, n, stream=side)
    dq, dk, dv = fa.cross_bwd(q, k, v, o, lse, do, n, stream=side)
    side.synchronize()
    assert torch.equal(o, want["o"]) and torch.equal(dk, want["dk"]) and torch.equal(dv, want["dv"])
    compare(q, k, v, do, lens, {"dq": dq})


def test_graph_follows_lengths():
    q, k, v, do = draw(2, 4, 4, 1, 900, 128, None, 18)
    n = device_lens([900, 900])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fa.cross_bwd(q, k, v, *fa.cross_fwd(q, k, v, n), do, n)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.cross_fwd(q, k, v, n)
        dq, dk, dv = fa.cross_bwd(q, k, v, o, lse, do, n)
    for lens in ([900, 900], [0, 5], [640, 128]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        compare(q, k, v, do, lens, {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv})
    assert fa.check_device_status() == 0


def test_guards():
    """Nothing outside the results is written."""
    B, H, Hkv, Nq, Nk, d = 2, 4, 2, 45, 140, 72
    lens = [139, 0]
    q, k, v, do = draw(B, H, Hkv, Nq, Nk, d, lens, 19)
    sizes = {"o": q.shape, "lse": q.shape[:3], "dq": q.shape, "dk": k.shape, "dv": k.shape}
    bufs, outs = {}, {}
    for name, shape in sizes.items():
        n = math.prod(shape)
        bufs[name] = torch.full((n + 128,), -77.0, dtype=torch.float32 if name == "lse" else torch.bfloat16, device="cuda")
        outs[name] = bufs[name][64:64 + n].view(shape)
    n = device_lens(lens)
    need = fa.cross_fwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)
    ws = torch.full((need + 128,), 77, dtype=torch.uint8, device="cuda")
    fa.cross_fwd_into(q, k, v, outs["o"], outs["lse"], ws[64:64 + need] if need else None, n)
    need2 = fa.cross_bwd_workspace_bytes(B, H, Hkv, Nq, Nk, d)
    ws2 = torch.full((need2 + 128,), 77, dtype=torch.uint8, device="cuda")
    fa.cross_bwd_into(q, k, v, outs["o"], outs["lse"], do, outs["dq"], outs["dk"], outs["dv"], ws2[64:64 + need2], n)
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
    compare(q, k, v, do, lens, outs)
    for name, b in bufs.items():
        assert (b[:64] == -77.0).all() and (b[-64:] == -77.0).all(), name
    for b, m in ((ws, need), (ws2, need2)):
        assert (b[:64] == 77).all() and (b[64 + m:] == 77).all()


def test_a_wait_that_runs_out_is_reported():
    """A K tile (a Q tile) that is never loaded: the status tells, and the next call is right."""
    q, k, v, do = draw(1, 2, 2, 200, 500, 128, None, 20)
    good = run_all(q, k, v, do, None)
    fa.set_wait_limit_ns(20_000_000)
    try:
        for tile in (0, 2):
            fa.debug_skip_k_tile(tile)
            fa.cross_fwd(q, k, v)
            assert fa.check_device_status() == 4
            fa.cross_bwd(q, k, v, good["o"], good["lse"], do)
            assert fa.check_device_status() == 4
    finally:
        fa.debug_skip_k_tile(-1)
        fa.set_wait_limit_ns(0)
    compare(q, k, v, do, None, run_all(q, k, v, do, None))
