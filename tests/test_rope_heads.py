"""Rotary positions of few positions and many heads, where one block holds many heads of a
position: at the limits of a block's shape, with a second tile of heads and a part of one.
The tolerance is test_rope.py's."""
import pytest
import torch

import io_aware_attention_gb300 as fa

from test_rope import check, freqs_of, rand, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d, rot", [(8, 8), (16, 16), (32, 32), (40, 40), (48, 48), (64, 64), (48, 16), (16, 6)])
@pytest.mark.parametrize("H, Hk", [(56, 8), (64, 1), (64, 8), (128, 32), (300, 0)])
def test_many_heads(H, Hk, d, rot, layout):
    inv = [1000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    for B, N in ((2, 1), (1, 2), (2, 3), (1, 5)):
        pos = torch.randint(0, 5000, (B, N), generator=torch.Generator("cpu").manual_seed(H + N))
        q = rand((B, H, N, d), N)
        k = rand((B, Hk, N, d), 9) if Hk else None
        qo, ko = fa.rope(q.cuda(), None if k is None else k.cuda(), freqs_of(inv).cuda(), positions=pos.cuda(), layout=layout)
        torch.cuda.synchronize()
        for got, x in ((qo, q), (ko, k)):
            if x is not None:
                check(got, *reference(x, inv, pos, layout, 1.0), f"N{N}")
                assert torch.equal(got[..., rot:].cpu(), x[..., rot:])
