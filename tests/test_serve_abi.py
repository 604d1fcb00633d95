"""Refusals of the rotary and 4-bit cache entry points, on the CPU: bad arguments
are rejected before the GPU is touched (addresses are fakes that are never
dereferenced), and the binding refuses tensors that are not on a GPU before
the library loads."""
import ctypes
import os
import shutil

import pytest
import torch

import io_aware_attention_gb300 as fa
from io_aware_attention_gb300 import _build

needs_lib = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists(_build.LIB_PATH),
                               reason="neither nvcc nor a built library")
P = 1 << 30
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.library()


def strides(s):
    return None if s is None else (ctypes.c_int64 * 3)(*s)


def rope(lib, q=P, qs=None, k=2 * P, ks=None, qo=3 * P, qos=None, ko=4 * P, kos=None, B=1, H=2, Hk=1, N=16, d=64,
         freqs=5 * P, rot=64, inter=0, factor=1.0, inverse=0, pos=0, pos_bytes=4, pos_stride=0, lens=0):
    return lib.fa_rope(vp(q), strides(qs), vp(k), strides(ks), vp(qo), strides(qos), vp(ko), strides(kos), B, H, Hk, N,
                       d, vp(freqs), rot, inter, factor, inverse, vp(pos), pos_bytes, pos_stride, vp(lens), None)


ROW = 16 * 64  # elements of one head


@needs_lib
@pytest.mark.parametrize("kw, status", [
    (dict(q=0), 1), (dict(qo=0), 1), (dict(freqs=0), 1), (dict(k=0), 1), (dict(ko=0), 1), (dict(k=0, ko=0), 1),
    (dict(B=0), 1), (dict(H=0), 1), (dict(Hk=0), 1), (dict(N=0), 1), (dict(d=0), 1), (dict(rot=0), 1),
    (dict(rot=63), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(inter=2), 1), (dict(inverse=-1), 1),
    (dict(factor=float("nan")), 1), (dict(factor=float("inf")), 1),
    (dict(d=60, rot=60), 2), (dict(d=136), 2),
    (dict(pos=6 * P, pos_bytes=2), 1), (dict(pos=6 * P, pos_stride=-1), 1), (dict(pos=6 * P, lens=7 * P), 1),
    (dict(pos=6 * P + 2), 2), (dict(pos=6 * P + 4, pos_bytes=8), 2), (dict(lens=6 * P + 1), 2), (dict(freqs=5 * P + 4), 2),
    (dict(q=P + 1), 2), (dict(ko=4 * P + 1), 2),
    (dict(qs=(0, -64, 64)), 1), (dict(qs=(0, 1 << 60, 64)), 1),
    (dict(qos=(0, 0, 64)), 1),                 # the output's heads share places
    (dict(qos=(0, ROW - 64, 64)), 1),          # the second head begins in the first one
    (dict(qo=P + 128), 1),                     # in place, but shifted
    (dict(qo=P, qs=(0, 2 * ROW, 64)), 1),      # in place with other strides
    (dict(qo=2 * P), 1), (dict(ko=P), 1),      # onto the other tensor's input
    (dict(ko=3 * P + 64), 1),                  # outputs share places
    (dict(freqs=3 * P), 1), (dict(pos=4 * P), 1), (dict(lens=4 * P), 1),
    (dict(B=1 << 40, H=1 << 20), 1), (dict(N=1 << 58), 1),
])
def test_rope_refuses(lib, kw, status):
    assert rope(lib, **kw) == status


@needs_lib
def test_rope_accepts_views_of_one_buffer(lib):
    """Interleaved views and in-place calls pass the checks (and then meet the missing or unsuited device)."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would run on fake addresses")
    fused = dict(qs=(0, 64, 192), ks=(0, 64, 192), H=2, Hk=1, k=P + 256)
    assert rope(lib, qo=P, ko=P + 256, qos=(0, 64, 192), kos=(0, 64, 192), **fused) in (2, 3)
    assert rope(lib, **fused) in (2, 3)
    assert rope(lib, qo=P + 2, qos=(0, 64, 192), **fused) == 1
    assert rope(lib, k=0, ko=0, Hk=0) in (2, 3)
    assert rope(lib, qo=P, ko=2 * P) in (2, 3)


CACHE = dict(pool=10 * P, pages=8, table=20 * P, max_pages=4, lens=21 * P)


def append(lib, k=P, ks=None, v=2 * P, vs=None, B=2, Hkv=2, N=3, d=64, k_scale=1.0, v_scale=1.0, **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_append(vp(k), strides(ks), vp(v), strides(vs), B, Hkv, N, d, k_scale, v_scale, vp(c["pool"]),
                                c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]), None)


def read(lib, k=P, v=2 * P, B=2, Hkv=2, N=3, d=64, newest=0, k_scale=1.0, v_scale=1.0, **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_read(vp(c["pool"]), c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]), vp(k), vp(v), B, Hkv,
                              N, d, newest, k_scale, v_scale, None)


def decode(lib, q=P, o=2 * P, lse=3 * P, B=2, H=4, Hkv=2, Nq=1, d=64, causal=0, scale=0.1, k_scale=1.0, v_scale=1.0,
           ws=4 * P, ws_bytes=1 << 26, **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_decode(vp(q), vp(c["pool"]), c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]), vp(o),
                                vp(lse), B, H, Hkv, Nq, d, causal, scale, k_scale, v_scale, vp(ws), ws_bytes, None)


def weights(lib, q=P, lse=2 * P, w=3 * P, out=4 * P, W=256, B=2, H=4, Hkv=2, Nq=1, d=64, causal=0, scale=0.1, k_scale=1.0,
            **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_weights(vp(q), vp(lse), vp(c["pool"]), c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]),
                                 vp(w), vp(out), W, B, H, Hkv, Nq, d, causal, scale, k_scale, None)


def evict(lib, table_out=20 * P, max_out=4, w=3 * P, out=4 * P, W=256, kept=5 * P, lens_out=6 * P, B=2, Hkv=2, d=64,
          keep=100, sink=4, recent=16, **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_evict(vp(c["pool"]), c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]), vp(table_out), max_out,
                               vp(w), vp(out), W, vp(kept), vp(lens_out), B, Hkv, d, keep, sink, recent, None)


@needs_lib
@pytest.mark.parametrize("call", [append, read, decode, weights, evict])
@pytest.mark.parametrize("kw, status", [
    (dict(pool=0), 1), (dict(table=0), 1), (dict(lens=0), 1), (dict(pages=0), 1), (dict(max_pages=0), 1), (dict(B=0), 1),
    (dict(Hkv=0), 1), (dict(d=0), 1), (dict(d=60), 2), (dict(d=136), 2), (dict(pool=10 * P + 8), 2), (dict(table=20 * P + 2), 2),
    (dict(lens=21 * P + 1), 2), (dict(pages=1 << 31), 1), (dict(max_pages=1 << 30), 1), (dict(B=1 << 17), 1),
])
def test_cache_calls_refuse_bad_caches(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_lib
@pytest.mark.parametrize("call, kw, status", [
    (append, dict(k=0), 1), (append, dict(v=0), 1), (append, dict(N=0), 1), (append, dict(k_scale=0.0), 1),
    (append, dict(v_scale=float("inf")), 1), (append, dict(k_scale=-1.0), 1), (append, dict(v_scale=float("nan")), 1),
    (append, dict(k=P + 8), 2), (append, dict(ks=(384, 192, 60)), 2), (append, dict(ks=(384, -192, 64)), 1),
    (append, dict(k=10 * P + 64), 1), (append, dict(table=10 * P), 1), (append, dict(lens=10 * P + 4), 1),
    (read, dict(k=0), 1), (read, dict(N=0), 1), (read, dict(newest=2), 1), (read, dict(k=P + 2), 2), (read, dict(v=P + 64), 1),
    (read, dict(k=10 * P), 1), (read, dict(v=20 * P), 1), (read, dict(k_scale=0.0), 1),
    (decode, dict(q=0), 1), (decode, dict(o=0), 1), (decode, dict(lse=0), 1), (decode, dict(ws=0), 1),
    (decode, dict(H=3), 1), (decode, dict(Nq=0), 1), (decode, dict(Nq=9), 2), (decode, dict(causal=2), 1),
    (decode, dict(scale=0.0), 1), (decode, dict(scale=float("nan")), 1), (decode, dict(scale=1e38, k_scale=10.0), 1),
    (decode, dict(q=P + 4), 2), (decode, dict(o=2 * P + 8), 2), (decode, dict(lse=3 * P + 2), 2), (decode, dict(ws=4 * P + 8), 2),
    (decode, dict(o=P), 1), (decode, dict(lse=2 * P), 1), (decode, dict(o=10 * P + 4608), 1), (decode, dict(lse=20 * P), 1),
    (decode, dict(B=2049, max_pages=1), 2), (decode, dict(H=1 << 30, Hkv=1), 1),
    (weights, dict(q=0), 1), (weights, dict(lse=0), 1), (weights, dict(w=0), 1), (weights, dict(out=0), 1),
    (weights, dict(W=0), 1), (weights, dict(H=5), 1), (weights, dict(Nq=9), 2), (weights, dict(out=3 * P + 64), 1),
    (weights, dict(out=P), 1), (weights, dict(out=2 * P), 1), (weights, dict(out=10 * P), 1), (weights, dict(w=3 * P + 2), 2),
    (evict, dict(table_out=0), 1), (evict, dict(w=0), 1), (evict, dict(out=0), 1), (evict, dict(kept=0), 1),
    (evict, dict(lens_out=0), 1), (evict, dict(keep=0), 1), (evict, dict(sink=-1), 1), (evict, dict(recent=-1), 1),
    (evict, dict(sink=60, recent=60), 1), (evict, dict(keep=200, max_out=3), 1), (evict, dict(W=0), 1),
    (evict, dict(out=3 * P), 1), (evict, dict(kept=4 * P + 64), 1), (evict, dict(lens_out=21 * P), 1),
    (evict, dict(lens_out=5 * P), 1), (evict, dict(kept=10 * P), 1), (evict, dict(w=10 * P), 1), (evict, dict(kept=5 * P + 2), 2),
])
def test_cache_calls_refuse(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_lib
def test_workspace_query_refuses(lib):
    out = ctypes.c_size_t(0)
    ask = lambda *a: lib.fa_qcache_decode_workspace_bytes(*a, ctypes.byref(out))  # noqa: E731
    assert ask(1, 5, 2, 1, 64, 4) == 1 and ask(1, 4, 2, 9, 64, 4) == 2 and ask(1, 4, 2, 1, 60, 4) == 2
    assert ask(1, 4, 2, 1, 64, 0) == 1 and ask(2049, 4, 2, 1, 64, 1) == 2
    assert lib.fa_qcache_decode_workspace_bytes(1, 4, 2, 1, 64, 4, None) == 1


def test_cpu_tensors_are_refused_before_the_library_loads(monkeypatch):
    def no_library():
        raise AssertionError("the library was loaded for a call that must be refused")

    monkeypatch.setattr(fa, "library", no_library)
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    pool, table, lens = torch.zeros((2, 2, 4608), dtype=torch.uint8), torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    w = torch.zeros((1, 2, 128))
    for call in (lambda: fa.rope(q, None, torch.zeros(32, dtype=torch.int64)),
                 lambda: fa.rope_into(q, None, q, None, torch.zeros(32, dtype=torch.int64)),
                 lambda: fa.rope(q, None, torch.zeros(32, dtype=torch.int64), layout="other"),
                 lambda: fa.qcache_append(q, q, pool, table, lens),
                 lambda: fa.qcache_read(pool, table, lens, 4, 64),
                 lambda: fa.qcache_decode(q, pool, table, lens),
                 lambda: fa.qcache_weights(q, torch.zeros((1, 2, 4)), pool, table, lens, w),
                 lambda: fa.qcache_evict(pool, table, lens, w, 10),
                 lambda: fa.qcache_pool(4, 2, 60)):
        with pytest.raises(ValueError):
            call()
