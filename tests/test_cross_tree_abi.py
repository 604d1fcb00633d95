"""Refusals of cross attention, the drafted tree and its commit, on the CPU: bad
arguments are rejected before the GPU is touched (addresses are fakes that are never
dereferenced), and the binding refuses tensors that are not on a GPU before the
library loads."""
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
INVALID, UNSUPPORTED, NO_DEVICE = 1, 2, (2, 3)
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.library()


def strides(s):
    return None if s is None else (ctypes.c_int64 * 3)(*s)


SIZES = dict(B=2, H=4, Hkv=2, Nq=3, Nk=5, d=64, scale=0.1, lens=16 * P, ws=17 * P, ws_bytes=1 << 26)


def cross_fwd(lib, q=P, qs=None, k=2 * P, ks=None, v=3 * P, vs=None, o=4 * P, os=None, lse=5 * P, **kw):
    a = {**SIZES, **kw}
    return lib.fa_cross_fwd(vp(q), strides(qs), vp(k), strides(ks), vp(v), strides(vs), vp(o), strides(os), vp(lse), vp(a["lens"]),
                            a["B"], a["H"], a["Hkv"], a["Nq"], a["Nk"], a["d"], a["scale"], vp(a["ws"]), a["ws_bytes"], None)


def cross_bwd(lib, q=P, qs=None, k=2 * P, ks=None, v=3 * P, vs=None, o=4 * P, os=None, lse=5 * P, do=6 * P, dos=None, dq=7 * P,
              dqs=None, dk=8 * P, dks=None, dv=9 * P, dvs=None, **kw):
    a = {**SIZES, **kw}
    return lib.fa_cross_bwd(vp(q), strides(qs), vp(k), strides(ks), vp(v), strides(vs), vp(o), strides(os), vp(lse), vp(do),
                            strides(dos), vp(dq), strides(dqs), vp(dk), strides(dks), vp(dv), strides(dvs), vp(a["lens"]), a["B"],
                            a["H"], a["Hkv"], a["Nq"], a["Nk"], a["d"], a["scale"], vp(a["ws"]), a["ws_bytes"], None)


@needs_lib
@pytest.mark.parametrize("call", [cross_fwd, cross_bwd])
@pytest.mark.parametrize("kw, status", [
    (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(o=0), INVALID), (dict(lse=0), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(Nq=0), INVALID), (dict(Nk=0), INVALID),
    (dict(d=0), INVALID), (dict(B=-1), INVALID), (dict(H=3), INVALID), (dict(Hkv=8), INVALID),
    (dict(d=60), UNSUPPORTED), (dict(d=136), UNSUPPORTED),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=P + 8), UNSUPPORTED), (dict(k=2 * P + 2), UNSUPPORTED), (dict(v=3 * P + 4), UNSUPPORTED), (dict(o=4 * P + 8), UNSUPPORTED),
    (dict(lse=5 * P + 2), UNSUPPORTED), (dict(lens=16 * P + 2), UNSUPPORTED), (dict(ws=17 * P + 8), UNSUPPORTED),
    (dict(qs=(768, 192, 60)), UNSUPPORTED), (dict(qs=(-768, 192, 64)), INVALID), (dict(qs=(768, 192, 56)), INVALID),
    (dict(ks=(640, 324, 64)), UNSUPPORTED), (dict(ks=(640, 320, 0)), UNSUPPORTED), (dict(vs=(1 << 40, 320, 64)), UNSUPPORTED),
    (dict(B=1 << 20, H=1 << 12, Hkv=1), INVALID), (dict(Nk=(1 << 23) + 1), INVALID), (dict(Nq=1 << 40), INVALID),
    (dict(B=1 << 62, H=2, Hkv=1), INVALID), (dict(Nk=1 << 23, H=1 << 14), INVALID),
])
def test_cross_refuses(lib, call, kw, status):
    assert call(lib, **kw) == status


ROW = 3 * 64  # elements of a query head


@needs_lib
@pytest.mark.parametrize("call, kw, status", [
    (cross_fwd, dict(os=(4 * ROW, 0, 64)), INVALID),         # the result's heads share places
    (cross_fwd, dict(os=(0, ROW, 64)), INVALID),
    (cross_fwd, dict(os=(4 * ROW, ROW - 64, 64)), INVALID),  # a head begins in the one before
    (cross_fwd, dict(o=P + 128), INVALID), (cross_fwd, dict(o=2 * P), INVALID), (cross_fwd, dict(o=3 * P + 1024), INVALID),
    (cross_fwd, dict(lse=P), INVALID), (cross_fwd, dict(lse=4 * P), INVALID), (cross_fwd, dict(lse=16 * P + 4), INVALID),
    (cross_fwd, dict(o=16 * P), INVALID),
    (cross_bwd, dict(do=0), INVALID), (cross_bwd, dict(dq=0), INVALID), (cross_bwd, dict(dk=0), INVALID),
    (cross_bwd, dict(dv=0), INVALID), (cross_bwd, dict(ws=0), INVALID), (cross_bwd, dict(do=6 * P + 8), UNSUPPORTED),
    (cross_bwd, dict(dq=7 * P + 4), UNSUPPORTED), (cross_bwd, dict(dv=9 * P + 2), UNSUPPORTED),
    (cross_bwd, dict(ws_bytes=4 * 2 * 64 * 66 * 4 - 1), INVALID),
    (cross_bwd, dict(dq=P), INVALID), (cross_bwd, dict(dq=4 * P), INVALID), (cross_bwd, dict(dq=6 * P + 64), INVALID),
    (cross_bwd, dict(dk=2 * P), INVALID), (cross_bwd, dict(dv=8 * P), INVALID), (cross_bwd, dict(dv=8 * P + 128), INVALID),
    (cross_bwd, dict(dk=7 * P), INVALID), (cross_bwd, dict(dk=5 * P), INVALID), (cross_bwd, dict(dv=16 * P), INVALID),
    (cross_bwd, dict(dks=(640, 0, 64)), INVALID), (cross_bwd, dict(dvs=(0, 320, 64)), INVALID),
    (cross_bwd, dict(dqs=(4 * ROW, ROW, 0)), INVALID),
    (cross_bwd, dict(ws=P), INVALID), (cross_bwd, dict(ws=9 * P), INVALID), (cross_bwd, dict(ws=5 * P), INVALID),
    (cross_bwd, dict(ws=16 * P), INVALID),
])
def test_cross_refuses_shared_places(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_lib
def test_cross_accepts_views(lib):
    """Fused projections, expanded states and one buffer of both gradients pass the checks (and then meet the missing device)."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the call would run on fake addresses")
    for kw in (dict(), dict(lens=0), dict(qs=(3 * 256, 64, 256)), dict(ks=(0, 64, 256), vs=(0, 64, 256), v=2 * P + 256),
               dict(ks=(640, 0, 64)), dict(Nq=1, qs=(8, 0, 3), H=2, B=1)):
        assert cross_fwd(lib, **kw) in NO_DEVICE
        assert cross_bwd(lib, **kw) in NO_DEVICE
    both = (5 * 256, 64, 256)
    assert cross_bwd(lib, dks=both, dvs=both, dv=8 * P + 256) in NO_DEVICE
    assert cross_bwd(lib, ws_bytes=4 * 2 * 64 * 66 * 4) in NO_DEVICE


@needs_lib
def test_cross_workspace_queries_refuse(lib):
    out = ctypes.c_size_t(0)
    for ask in (lib.fa_cross_fwd_workspace_bytes, lib.fa_cross_bwd_workspace_bytes):
        assert ask(2, 4, 2, 3, 5, 64, None) == INVALID
        for sizes in ((0, 4, 2, 3, 5, 64), (2, 3, 2, 3, 5, 64), (2, 4, 2, 0, 5, 64), (2, 4, 2, 3, 0, 64), (2, 4, 2, 1 << 40, 5, 64)):
            assert ask(*sizes, ctypes.byref(out)) == INVALID
        assert ask(2, 4, 2, 3, 5, 60, ctypes.byref(out)) == UNSUPPORTED
    assert lib.fa_cross_bwd_workspace_bytes(2, 4, 2, 65, 5, 72, ctypes.byref(out)) == 0
    assert out.value == 2 * 4 * 128 * (128 + 2) * 4


CACHE = dict(pool=10 * P, pages=8, table=20 * P, max_pages=4, lens=21 * P)


def tree(lib, q=P, words=2 * P, o=3 * P, lse=4 * P, B=2, H=4, Hkv=2, T=3, d=64, scale=0.1, k_scale=1.0, v_scale=1.0, ws=5 * P,
         ws_bytes=1 << 28, **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_tree(vp(q), vp(words), vp(c["pool"]), c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]), vp(o),
                              vp(lse), B, H, Hkv, T, d, scale, k_scale, v_scale, vp(ws), ws_bytes, None)


def commit(lib, path=P, width=2, out=2 * P, B=2, Hkv=2, T=3, d=64, **c):
    c = {**CACHE, **c}
    return lib.fa_qcache_commit(vp(c["pool"]), c["pages"], vp(c["table"]), c["max_pages"], vp(c["lens"]), vp(path), width,
                                vp(out), B, Hkv, T, d, None)


@needs_lib
@pytest.mark.parametrize("call", [tree, commit])
@pytest.mark.parametrize("kw, status", [
    (dict(pool=0), INVALID), (dict(table=0), INVALID), (dict(lens=0), INVALID), (dict(pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(d=0), INVALID), (dict(T=0), INVALID),
    (dict(T=-1), INVALID), (dict(T=65), UNSUPPORTED), (dict(d=60), UNSUPPORTED), (dict(d=136), UNSUPPORTED),
    (dict(pool=10 * P + 8), UNSUPPORTED), (dict(table=20 * P + 2), UNSUPPORTED), (dict(lens=21 * P + 1), UNSUPPORTED),
    (dict(pages=1 << 31), INVALID), (dict(max_pages=1 << 30), INVALID), (dict(B=1 << 17), INVALID),
])
def test_tree_calls_refuse_bad_caches(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_lib
@pytest.mark.parametrize("call, kw, status", [
    (tree, dict(q=0), INVALID), (tree, dict(words=0), INVALID), (tree, dict(o=0), INVALID), (tree, dict(lse=0), INVALID),
    (tree, dict(ws=0), INVALID), (tree, dict(H=3), INVALID), (tree, dict(H=0), INVALID), (tree, dict(scale=0.0), INVALID),
    (tree, dict(scale=float("nan")), INVALID), (tree, dict(k_scale=0.0), INVALID), (tree, dict(v_scale=float("inf")), INVALID),
    (tree, dict(q=P + 8), UNSUPPORTED), (tree, dict(words=2 * P + 4), UNSUPPORTED), (tree, dict(o=3 * P + 2), UNSUPPORTED),
    (tree, dict(lse=4 * P + 2), UNSUPPORTED), (tree, dict(ws=5 * P + 8), UNSUPPORTED), (tree, dict(B=2049, max_pages=1), UNSUPPORTED),
    (tree, dict(o=P + 64), INVALID), (tree, dict(lse=P), INVALID), (tree, dict(o=2 * P), INVALID), (tree, dict(lse=3 * P), INVALID),
    (tree, dict(o=10 * P), INVALID), (tree, dict(lse=20 * P), INVALID), (tree, dict(o=21 * P), INVALID),
    (tree, dict(H=1 << 30, Hkv=1), INVALID),
    (commit, dict(path=0), INVALID), (commit, dict(out=0), INVALID), (commit, dict(width=0), INVALID), (commit, dict(width=4), INVALID),
    (commit, dict(path=P + 2), UNSUPPORTED), (commit, dict(out=2 * P + 1), UNSUPPORTED),
    (commit, dict(out=21 * P), INVALID), (commit, dict(out=21 * P + 4), INVALID), (commit, dict(out=P + 8), INVALID),
    (commit, dict(out=10 * P + 4608), INVALID), (commit, dict(out=20 * P), INVALID), (commit, dict(path=10 * P), INVALID),
    (commit, dict(table=10 * P), INVALID), (commit, dict(lens=10 * P), INVALID),
])
def test_tree_calls_refuse(lib, call, kw, status):
    assert call(lib, **kw) == status


@needs_lib
def test_tree_workspace_query_refuses(lib):
    out = ctypes.c_size_t(0)
    ask = lambda *a: lib.fa_qcache_tree_workspace_bytes(*a, ctypes.byref(out))  # noqa: E731
    assert lib.fa_qcache_tree_workspace_bytes(1, 4, 2, 3, 64, 4, None) == INVALID
    assert ask(1, 5, 2, 3, 64, 4) == INVALID and ask(1, 4, 2, 0, 64, 4) == INVALID and ask(1, 4, 2, 3, 64, 0) == INVALID
    assert ask(1, 4, 2, 65, 64, 4) == UNSUPPORTED and ask(1, 4, 2, 3, 60, 4) == UNSUPPORTED and ask(2049, 4, 2, 3, 64, 1) == UNSUPPORTED


def test_cpu_tensors_are_refused_before_the_library_loads(monkeypatch):
    def no_library():
        raise AssertionError("the library was loaded for a call that must be refused")

    monkeypatch.setattr(fa, "library", no_library)
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    lse, ws, path = torch.zeros((1, 2, 4)), torch.zeros(64, dtype=torch.uint8), torch.zeros((1, 2), dtype=torch.int32)
    pool, table, lens = torch.zeros((2, 2, 4608), dtype=torch.uint8), torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    words = torch.zeros((1, 4), dtype=torch.int64)
    for call in (lambda: fa.cross_fwd(q, q, q), lambda: fa.cross_fwd(q, q, q, lens),
                 lambda: fa.cross_fwd_into(q, q, q, q, lse),
                 lambda: fa.cross_bwd(q, q, q, q, lse, q),
                 lambda: fa.cross_bwd_into(q, q, q, q, lse, q, q, q, q, ws),
                 lambda: fa.qcache_tree(q, words, pool, table, lens),
                 lambda: fa.qcache_tree_into(q, words, pool, table, lens, q, lse, ws),
                 lambda: fa.qcache_commit(pool, table, lens, path, 4)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses():
    """Types, shapes and workspaces that do not fit are refused before a launch."""
    B, H, Hkv, Nq, Nk, d, T = 2, 4, 2, 3, 130, 64, 3
    z = lambda *s, **k: torch.zeros(s, device="cuda", **{"dtype": torch.bfloat16, **k})  # noqa: E731
    q, k, o, lse = z(B, H, Nq, d), z(B, Hkv, Nk, d), z(B, H, Nq, d), z(B, H, Nq, dtype=torch.float32)
    lens, ws = z(B, dtype=torch.int32), z(1 << 22, dtype=torch.uint8)
    for call in (lambda: fa.cross_fwd(q.half(), k, k), lambda: fa.cross_fwd(q, k.float(), k), lambda: fa.cross_fwd(q[0], k, k),
                 lambda: fa.cross_fwd(q, k[:1], k[:1]), lambda: fa.cross_fwd(q, k, k[:, :, 1:]), lambda: fa.cross_fwd(q[:, :3], k, k),
                 lambda: fa.cross_fwd(q, k[..., :56], k[..., :56]), lambda: fa.cross_fwd(q.transpose(2, 3), k, k),
                 lambda: fa.cross_fwd(q, k, k, lens.long()), lambda: fa.cross_fwd(q, k, k, lens[:1]),
                 lambda: fa.cross_fwd(q, k, k, lens.cpu()),
                 lambda: fa.cross_fwd_into(q, k, k, o[:, :2], lse), lambda: fa.cross_fwd_into(q, k, k, o, lse.bfloat16()),
                 lambda: fa.cross_fwd_into(q, k, k, o, lse[..., :2]), lambda: fa.cross_fwd_into(q, k, k, o, lse, ws.cpu()),
                 lambda: fa.cross_bwd(q, k, k, o, lse[:, :2], q), lambda: fa.cross_bwd(q, k, k, o, lse, q[:, :, :2]),
                 lambda: fa.cross_bwd(q, k, k, o, lse, q.float()),
                 lambda: fa.cross_bwd_into(q, k, k, o, lse, q, o.clone(), k.clone(), k[:, :, 1:].clone(), ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fa.FaError):
        fa.cross_bwd_into(q, k, k, o, lse, q, o.clone(), k.clone(), k.clone(), ws[:64])
    with pytest.raises(fa.FaError):
        fa.cross_fwd_into(q, k, k, q, lse, ws)
    pool, table = fa.qcache_pool(8, Hkv, d), z(B, 4, dtype=torch.int32)
    words, path = z(B, T, dtype=torch.int64), z(B, 2, dtype=torch.int32)
    for call in (lambda: fa.qcache_tree(q, words.int(), pool, table, lens), lambda: fa.qcache_tree(q, words[:, :2], pool, table, lens),
                 lambda: fa.qcache_tree(q, words.cpu(), pool, table, lens),
                 lambda: fa.qcache_tree(q, words.t().contiguous().t(), pool, table, lens),
                 lambda: fa.qcache_tree(q.half(), words, pool, table, lens), lambda: fa.qcache_tree(q, words, pool, table.long(), lens),
                 lambda: fa.qcache_tree_into(q, words, pool, table, lens, o[:, :2], lse, ws),
                 lambda: fa.qcache_tree_into(q, words, pool, table, lens, o, lse, ws[::2]),
                 lambda: fa.qcache_commit(pool, table, lens, path.long(), T), lambda: fa.qcache_commit(pool, table, lens, path[:1], T),
                 lambda: fa.qcache_commit(pool, table, lens, path[0], T), lambda: fa.qcache_commit(pool, table, lens[:1], path, T)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fa.qcache_tree_into(q, words, pool, table, lens, o, lse, ws[:64]),
                 lambda: fa.qcache_tree(q, words, pool, table, lens, scale=0.0),
                 lambda: fa.qcache_tree(q[:, :3].contiguous(), words, pool, table, lens),
                 lambda: fa.qcache_commit(pool, table, lens, path, 1), lambda: fa.qcache_commit(pool, table, lens, path, 65)):
        with pytest.raises(fa.FaError):
            call()
    torch.cuda.synchronize()
    assert fa.check_device_status() == 0
