"""The serving loop as the package's documentation prints it, run over two evictions: every
token attends by the true positions of the keys that are left, not by their places in the cache.

The loop's code is taken from the package's docstring.  Beside it a second cache takes every key,
turned by its position in the text, and drops none; the keys that the loop should still hold are picked
from that one, and attention over them is computed in 64 bits.
"""
import math
import textwrap

import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
from test_qcache import check_attention

pytestmark = pytest.mark.gpu


def printed_loop():
    """(a step's code, the eviction's code) of the package's docstring."""
    blocks = [b for b in fa.__doc__.split("\n\n") if b.startswith("    ")]
    block = next(b for b in blocks if "qcache_append(" in b)
    lines = textwrap.dedent(block).splitlines()
    cut = next(i for i, line in enumerate(lines) if "qcache_evict(" in line)
    return "\n".join(line for line in lines[:cut] if "qcache_pool(" not in line), "\n".join(lines[cut:])


class Picked:
    """Attention's reference over keys picked per kv head, with check_attention's interface."""

    def __init__(self, ks, vs):
        self.ks, self.vs = ks, vs

    def unpack(self, *_):
        return self.ks, self.vs


@pytest.mark.parametrize("B, H, Hkv, d", [(2, 4, 2, 64), (1, 6, 3, 128)])
def test_the_printed_loop_over_two_evictions(monkeypatch, B, H, Hkv, d):
    step, evict = printed_loop()
    g = torch.Generator("cpu").manual_seed(d)
    rand = lambda *shape: torch.randn(shape, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    prompt, keep, total = 60, 50, 150
    freqs, factor = fa.rope_frequencies(d, base=100.0)
    pages = -(-total // 64)
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").reshape(B, pages)
    all_pool, all_lens = fa.qcache_pool(B * pages, Hkv, d), torch.zeros(B, dtype=torch.int32, device="cuda")

    def remember(k, v, first):
        """The cache that drops nothing: keys turned by where they stand in the text."""
        at = torch.arange(first, first + k.shape[2], device="cuda")
        _, turned = fa.rope(k, k, freqs, positions=at, factor=factor)
        all_lens.add_(k.shape[2])
        fa.qcache_append(turned, v, all_pool, table, all_lens)
        return turned

    loop = {"io_aware_attention_gb300": fa, "freqs": freqs, "factor": factor, "table": table, "keep": keep,
            "pool": fa.qcache_pool(B * pages, Hkv, d), "lens": torch.full((B,), prompt, dtype=torch.int32, device="cuda"),
            "weights": torch.zeros((B, Hkv, total), device="cuda"),
            "positions": torch.full((B, 1), prompt, dtype=torch.int64, device="cuda")}
    k, v = rand(B, Hkv, prompt, d), rand(B, Hkv, prompt, d)
    fa.qcache_append(remember(k, v, 0), v, loop["pool"], table, loop["lens"])
    held = torch.arange(prompt).expand(B, Hkv, prompt)  # the position in the text of each place of the loop's cache
    t = prompt
    for steps in (20, 15, 8):
        for _ in range(steps):
            q, k, v = rand(B, H, 1, d), rand(B, Hkv, 1, d), rand(B, Hkv, 1, d)
            remember(k, v, t)
            held = torch.cat([held, torch.full((B, Hkv, 1), t)], -1)
            loop.update(q=q, k=k, v=v)
            exec(step, loop)
            torch.cuda.synchronize()
            assert fa.check_device_status() == 0 and loop["lens"].tolist() == [held.shape[-1]] * B
            want_q, _ = fa.rope(q, None, freqs, positions=torch.tensor([t], device="cuda"), factor=factor)
            ks, vs = ref.unpack(all_pool, table, all_lens, d)
            at = held.numpy()
            pick = lambda x: [x[b][[[h] for h in range(Hkv)], at[b]] for b in range(B)]  # noqa: E731
            with monkeypatch.context() as m:
                m.setattr(ref, "unpack", Picked(pick(ks), pick(vs)).unpack)
                check_attention(loop["o"], loop["lse"], want_q.cpu(), (None, None, None), False, 1 / math.sqrt(d), f"token {t}")
            t += 1
        exec(evict, loop)
        held = held.gather(2, loop["kept"].long().cpu())
