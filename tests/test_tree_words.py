"""The words of drafted trees: parents of any layout, and parents that do not come before their children."""
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


@gpu
@pytest.mark.parametrize("T", [1, 2, 9, 64])
def test_wrong_parents_on_the_gpu_are_marked(T):
    """The word 0 and the depth -1 for a draft whose parent is itself or a later one, and its bit in no
    word; the rest of the tree as if that draft were a root that no one sees."""
    rng = np.random.default_rng(T)
    parents = _tree.random_parents(40, T, rng)
    at = rng.integers(0, T, 40)
    parents[np.arange(40), at] = rng.integers(at, T + 3)  # (T and above: no draft at all)
    parents[-1] = _tree.random_parents(1, T, rng)[0]
    chain = np.arange(T) - 1  # the last draft of a chain of 64 has all bits set
    parents[0], parents[1] = chain, chain
    parents[1, T - 1] = T - 1
    parents[2] = chain
    parents[2, 0] = 2 ** 40
    wrong = parents >= np.arange(T)
    words, depths = fa.tree_words(torch.from_numpy(parents).cuda())
    with pytest.raises(ValueError):
        fa.tree_words(torch.from_numpy(parents))
    bits = np.array([sum(1 << i for i in range(T) if row[i]) for row in wrong], np.uint64)[:, None]
    want = _tree.ancestors(np.where(wrong, -1, parents)).view(np.uint64) & ~bits
    assert np.array_equal(words.cpu().numpy(), want.view(np.int64))
    assert np.array_equal(depths.cpu().numpy(), [[bin(int(w)).count("1") - 1 for w in row] for row in want])
    assert (depths.cpu().numpy()[wrong] == -1).all() and (depths.cpu().numpy()[~wrong] >= 0).all()
    assert wrong[1, T - 1] and not wrong[0].any() and wrong[2].sum() == 1
