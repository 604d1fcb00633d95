"""stream= of the calls that write into given tensors: another device's stream is refused.
That device's default stream has the handle 0, which the library takes for the current device's."""
import types

import pytest
import torch

import io_aware_attention_gb300 as fa

pytestmark = pytest.mark.gpu


def test_into_calls_refuse_a_stream_of_another_device():
    here = torch.cuda.current_device()
    other = types.SimpleNamespace(device=torch.device("cuda", here + 1), cuda_stream=0)
    pool, table = fa.qcache_pool(2, 1, 64), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    lens, q = torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    freqs, _ = fa.rope_frequencies(64)
    o, lse = torch.zeros_like(q), torch.zeros((1, 1, 1), device="cuda")
    ws = torch.empty(fa.qcache_decode_workspace_bytes(1, 1, 1, 1, 64, 1), dtype=torch.uint8, device="cuda")
    pool.zero_()
    before = [t.clone() for t in (pool, o, lse)]
    for call in (lambda s: fa.rope_into(q, None, o, None, freqs, stream=s), lambda s: fa.qcache_append(q, q, pool, table, lens, stream=s),
                 lambda s: fa.qcache_decode_into(q, pool, table, lens, o, lse, ws, stream=s)):
        with pytest.raises(ValueError, match="stream is on"):
            call(other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (pool, o, lse)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    fa.qcache_append(q, q, pool, table, lens, stream=side)
    fa.qcache_decode_into(q, pool, table, lens, o, lse, ws, stream=side)
    side.synchronize()
    # One key of ones: its block's scale is the e4m3 number nearest to 1 / 6, 11 / 64, and its codes are 6.
    assert torch.equal(o, torch.full_like(o, 6 * 11 / 64)) and fa.check_device_status() == 0
