"""The decode-time operators together, as a serving loop runs them: rotary
positions, append to the 4-bit cache, attention over it, the weights that
keys gather, eviction -- eagerly, captured in a CUDA graph and replayed, on
two streams at once, and against the forward kernel.
"""
import math
import threading
import types

import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
from test_qcache import check_attention

pytestmark = pytest.mark.gpu


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator("cpu").manual_seed(seed)).to(torch.bfloat16).cuda()


class Loop:
    """A batch of sequences with a cache, stepped a token (or a prompt) at a time."""

    def __init__(self, B, H, Hkv, d, max_pages, seed):
        self.B, self.H, self.Hkv, self.d = B, H, Hkv, d
        g = torch.Generator("cpu").manual_seed(seed)
        self.pool = torch.randint(0, 256, (B * max_pages, Hkv, fa.qcache_pool(1, 1, d).shape[2]), generator=g, dtype=torch.uint8).cuda()
        self.table = torch.randperm(B * max_pages, generator=g).to(torch.int32).reshape(B, max_pages).cuda()
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.weights = torch.zeros((B, Hkv, max_pages * 64), device="cuda")
        self.freqs, self.factor = fa.rope_frequencies(d, scaling="parts", factor=4.0, original_length=256)

    def step(self, q, k, v, positions):
        """Keys stand where they were produced (positions), not at their place after an eviction."""
        q, k = fa.rope(q, k, self.freqs, positions=positions, factor=self.factor)
        self.lens += k.shape[2]
        fa.qcache_append(k, v, self.pool, self.table, self.lens)
        o, lse = fa.qcache_decode(q, self.pool, self.table, self.lens, causal=True)
        fa.qcache_weights(q, lse, self.pool, self.table, self.lens, self.weights, causal=True, out=self.weights)
        return q, o, lse

    def evict(self, keep, sink, recent):
        kept, lens, weights = fa.qcache_evict(self.pool, self.table, self.lens, self.weights, keep, sink=sink, recent=recent)
        self.lens.copy_(lens)
        self.weights.copy_(weights)
        return kept


@pytest.mark.parametrize("B, H, Hkv, d", [(2, 8, 2, 128), (3, 4, 4, 64), (1, 7, 1, 80)])
def test_loop_matches_the_definition_and_a_captured_graph(B, H, Hkv, d):
    prompt, steps, keep = 150, 5, 100
    loops = [Loop(B, H, Hkv, d, 6, seed=d) for _ in range(2)]
    # The prompt's keys go in 8 rows of queries at a time being enough for the test's attention.
    k0, v0, q0 = rand((B, Hkv, prompt, d), 1), rand((B, Hkv, prompt, d), 2), rand((B, H, 8, d), 3)
    for loop in loops:
        _, k = fa.rope(k0, k0, loop.freqs, factor=loop.factor)
        loop.lens += prompt
        fa.qcache_append(k, v0, loop.pool, loop.table, loop.lens)
        o, lse = fa.qcache_decode(q0, loop.pool, loop.table, loop.lens)
        fa.qcache_weights(q0, lse, loop.pool, loop.table, loop.lens, loop.weights, out=loop.weights)
    eager, graphed = loops
    kept = eager.evict(keep, 4, 20)
    kept2 = graphed.evict(keep, 4, 20)
    assert torch.equal(kept, kept2) and eager.lens.tolist() == [keep] * B
    assert kept[..., :4].tolist() == [[[0, 1, 2, 3]] * Hkv] * B
    assert kept[..., -20:].tolist() == [[list(range(130, 150))] * Hkv] * B

    def inputs(i):
        pos = torch.full((B, 1), prompt + i, dtype=torch.int64, device="cuda")
        return rand((B, H, 1, d), 10 + i), rand((B, Hkv, 1, d), 30 + i), rand((B, Hkv, 1, d), 50 + i), pos

    held = [t.clone() for t in inputs(0)]
    # Warm-up (on a loop of its own) and capture.
    spare = Loop(B, H, Hkv, d, 6, seed=d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        spare.step(*held)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    saved = [t.clone() for t in (graphed.pool, graphed.lens, graphed.weights)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = graphed.step(*held)
    assert all(torch.equal(a, b) for a, b in zip(saved, (graphed.pool, graphed.lens, graphed.weights)))  # captured, not run
    for i in range(steps):
        new = inputs(i)
        for t, x in zip(held, new):
            t.copy_(x)
        graph.replay()
        q, o, lse = eager.step(*new)
        torch.cuda.synchronize()
        assert fa.check_device_status() == 0
        for a, b in zip(out, (q, o, lse)):
            assert torch.equal(a, b), i
        assert torch.equal(graphed.pool, eager.pool) and torch.equal(graphed.weights, eager.weights)
        check_attention(o, lse, q.cpu(), (eager.pool, eager.table, eager.lens), True, 1 / math.sqrt(d), f"step {i}")
    assert eager.lens.tolist() == [keep + steps] * B
    # Every sequence's weights grew by one for each query head and step.
    total = eager.weights.double().sum(-1).cpu()
    assert total.shape == (B, Hkv) and torch.isfinite(total).all()


def test_two_streams_at_once():
    """Two loops on two streams and two threads, interleaved at will, give what each gives alone."""
    B, H, Hkv, d = 2, 8, 2, 128

    def run(seed, stream):
        out = []
        with torch.cuda.stream(stream):
            loop = Loop(B, H, Hkv, d, 4, seed)
            for i in range(20):
                pos = torch.full((B, 3), i, dtype=torch.int32, device="cuda")
                out.append(loop.step(rand((B, H, 3, d), seed + i), rand((B, Hkv, 3, d), seed + 50 + i),
                                     rand((B, Hkv, 3, d), seed + 90 + i), pos))
            loop.evict(30, 2, 5)
            out.append(loop.step(rand((B, H, 1, d), 7), rand((B, Hkv, 1, d), 8), rand((B, Hkv, 1, d), 9), pos[:, :1].contiguous()))
        stream.synchronize()
        return out

    alone = [run(s, torch.cuda.Stream()) for s in (100, 300)]
    both = [None, None]

    def work(i, s):
        both[i] = run(s, torch.cuda.Stream())

    threads = [threading.Thread(target=work, args=(i, s)) for i, s in enumerate((100, 300))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert fa.check_device_status() == 0
    for a, b in zip(alone, both):
        assert b is not None
        for x, y in zip(a, b):
            assert all(torch.equal(u, w) for u, w in zip(x, y))


def test_against_the_forward_and_the_bf16_decode():
    """What is read back from the cache, through fa.fwd and fa.decode, gives what the cache's own attention gives
    (both within bf16's rounding of the same values; probabilities of the forward are rounded to bf16)."""
    B, H, d, n = 2, 3, 128, 333
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    pool = fa.qcache_pool(B * 6, H, d)
    table = torch.arange(B * 6, dtype=torch.int32, device="cuda").reshape(B, 6)
    q, k, v = rand((B, H, n, d), 1), rand((B, H, n, d), 2), rand((B, H, n, d), 3)
    fa.qcache_append(k, v, pool, table, lens)
    k4, v4 = fa.qcache_read(pool, table, lens, n, d)
    o1, l1 = fa.fwd(q, k4, v4, causal=True)
    last = q[:, :, -8:].contiguous()
    o2, l2 = fa.qcache_decode(last, pool, table, lens, causal=True)
    o3, l3 = fa.decode(last, k4, v4, causal=True)
    torch.cuda.synchronize()
    assert (o1[:, :, -8:].float() - o2.float()).abs().max() <= 1e-2 and (l1[:, :, -8:] - l2).abs().max() <= 1e-3
    assert (o3.float() - o2.float()).abs().max() <= 1e-2 and (l3 - l2).abs().max() <= 1e-3


def test_lengths_and_tables_are_read_when_the_call_runs():
    """One captured decode serves other lengths and pages at replay."""
    d = 64
    pool, table, lens = (t.cuda() for t in ref.make_cache([300, 100, 0], 2, d, seed=8))
    q = rand((3, 4, 1, d), 4)
    fa.qcache_decode(q, pool, table, lens)  # set-up outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa.qcache_decode(q, pool, table, lens)
    for new in ([300, 100, 0], [1, 0, 0], [299, 64, 0], [0, 0, 0], [128, 99, 0]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        a, b = fa.qcache_decode(q, pool, table, lens)
        assert torch.equal(o, a) and torch.equal(lse, b), new
        check_attention(o, lse, q.cpu(), (pool, table, lens), False, 1 / math.sqrt(d), str(new))
    assert fa.check_device_status() == 0


def test_an_explicit_stream():
    """stream= runs the call, and gives its workspace and results, on that stream: while the current stream is busy
    and reuses the memory it frees, the results stay right."""
    B, H, Hkv, d, n = 2, 8, 2, 128, 300
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    pool = fa.qcache_pool(B * 8, Hkv, d)
    table = torch.arange(B * 8, dtype=torch.int32, device="cuda").reshape(B, 8)
    q, k, v = rand((B, H, 1, d), 1), rand((B, Hkv, n, d), 2), rand((B, Hkv, n, d), 3)
    freqs, _ = fa.rope_frequencies(d)
    zero = torch.zeros((B, Hkv, 512), device="cuda")
    table_out = table[:, 4:].contiguous()

    def calls(stream):
        q2, _ = fa.rope(q, None, freqs, lens=lens, stream=stream)
        fa.qcache_append(k, v, pool, table, lens, stream=stream)
        o, lse = fa.qcache_decode(q2, pool, table, lens, stream=stream)
        w = fa.qcache_weights(q2, lse, pool, table, lens, zero, stream=stream)
        kept, new, w2 = fa.qcache_evict(pool, table, lens, w, 100, table_out=table_out, stream=stream)
        return [q2, o, lse, w, kept, new, w2, *fa.qcache_read(pool, table_out, new, 100, d, stream=stream)]

    want = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        a = torch.randn((2048, 2048), device="cuda")
        for _ in range(10):  # keeps the current stream busy, allocating and freeing
            a = (a @ a).clamp(-1, 1)
        got = calls(side)
        junk = [torch.full_like(t, 7) for t in got]
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        del junk
    assert fa.check_device_status() == 0


def test_a_stream_of_another_device_is_refused():
    """A stream that the tensors' device does not have is an error, not a call on some other stream."""
    other = types.SimpleNamespace(device=torch.device("cuda", torch.cuda.current_device() + 1), cuda_stream=0)
    pool, table = fa.qcache_pool(2, 1, 64), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens, q = torch.ones(1, dtype=torch.int32, device="cuda"), rand((1, 1, 1, 64), 1)
    w, lse = torch.zeros((1, 1, 64), device="cuda"), torch.zeros((1, 1, 1), device="cuda")
    freqs, _ = fa.rope_frequencies(64)
    for call in (lambda: fa.rope(q, None, freqs, stream=other), lambda: fa.qcache_read(pool, table, lens, 1, 64, stream=other),
                 lambda: fa.qcache_decode(q, pool, table, lens, stream=other),
                 lambda: fa.qcache_weights(q, lse, pool, table, lens, w, stream=other),
                 lambda: fa.qcache_evict(pool, table, lens, w, 1, stream=other)):
        with pytest.raises(ValueError, match="stream is on"):
            call()
