"""The words of drafted trees: parents of any layout."""
import numpy as np
import pytest
import torch

import io_aware_attention_gb300 as fa

import _qcache as ref
import _tree

gpu = pytest.mark.gpu


def layouts(parents, device):
    """The same parents in other layouts and types."""
    t = torch.from_numpy(parents).to(device)
    wide = torch.zeros((parents.shape[0], 2 * parents.shape[1]), dtype=torch.int64, device=device)
    wide[:, ::2] = t
    return {"turned": t.t().contiguous().t(), "every other": wide[:, ::2], "int32": t.to(torch.int32), "int8, turned": t.to(torch.int8).t().contiguous().t()}


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=gpu)])
@pytest.mark.parametrize("B, T", [(1, 1), (3, 1), (1, 7), (4, 7), (64, 64)])
def test_any_layout(device, B, T):
    """Words and depths come contiguous, as the calls that take them want them."""
    parents = _tree.random_parents(B, T, np.random.default_rng(T))
    want = torch.from_numpy(_tree.ancestors(parents))
    for name, t in layouts(parents, device).items():
        words, depths = fa.tree_words(t)
        assert words.is_contiguous() and depths.is_contiguous(), name
        assert words.dtype == depths.dtype == torch.int64 and torch.equal(words.cpu(), want), name
    shared = torch.from_numpy(parents[:1]).to(device).expand(B, T)
    words, _ = fa.tree_words(shared)
    assert words.is_contiguous() and torch.equal(words.cpu(), want[:1].expand(B, T))


@gpu
def test_turned_parents_reach_the_tree():
    """Parents kept draft by draft, (T, B), turned for the call."""
    T, lens = 6, [90, 70, 64]
    parents = _tree.random_parents(3, T, np.random.default_rng(2))
    kept = torch.from_numpy(parents.T.copy()).cuda()
    cache = [t.cuda() for t in ref.make_cache(lens, 2, 64, seed=1)]
    q = torch.randn((3, 4, T, 64), device="cuda").to(torch.bfloat16)
    words, _ = fa.tree_words(kept.t())
    want = fa.qcache_tree(q, torch.from_numpy(_tree.ancestors(parents)).cuda(), *cache)
    for a, b in zip(fa.qcache_tree(q, words, *cache), want):
        assert torch.equal(a, b)
