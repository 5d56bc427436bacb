"""Host-side argument checks of the entries that move pages (no GPU: every call fails before a launch, or has
nothing to do)."""
import ctypes
import random
import timeit

import pytest

F = 1 << 34  # buffers 16 GB apart: no accidental overlap; never dereferenced


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    from gated_deltanet_linear_pre_gb300 import _native
    return _native.lib()


def remap(L, **over):
    a = dict(page=64, n_pages=100, width=8, n_old=3, table=F, ts=8, n=5, parent=2 * F, keep=3 * F, need=4 * F, out=5 * F, os=9, a=6 * F, b=7 * F,
             info=8 * F, ws=9 * F, wb=None)
    a.update(over)
    if a["wb"] is None:
        a["wb"] = L.gdn_kv_remap_workspace_bytes(a["n_pages"], a["n"], a["width"])
    return L.gdn_kv_remap(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(page=0), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(n_pages=0), 1), (dict(n_pages=(1 << 28) + 1), 2), (dict(width=-1), 1),
    (dict(width=1 << 25, ts=1 << 25, os=1 << 25), 2), (dict(n_old=-1), 1), (dict(n=-1), 1), (dict(ts=7), 1), (dict(os=7), 1),
    (dict(ts=1 << 31), 2), (dict(n=1 << 28), 2), (dict(table=None), 1), (dict(parent=None), 1), (dict(keep=None), 1), (dict(need=None), 1),
    (dict(out=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(info=None), 1), (dict(table=F + 2), 3), (dict(keep=3 * F + 1), 3),
    (dict(out=5 * F + 3), 3), (dict(info=8 * F + 2), 3), (dict(ws=None), 4), (dict(wb=1000), 4), (dict(ws=9 * F + 8), 3), (dict(out=F), 1),
    (dict(out=F + 64), 1), (dict(a=7 * F), 1), (dict(a=2 * F + 8), 1), (dict(info=9 * F + 256), 1), (dict(b=5 * F + 16), 1)])
def test_remap_refusals(L, over, status):
    assert remap(L, **over) == status
    assert L.gdn_last_error_string().decode()


def compact(L, **over):
    a = dict(n_pages=100, width=8, n=5, table=F, ts=8, out=2 * F, os=9, a=3 * F, b=4 * F, info=5 * F, ws=6 * F, wb=None)
    a.update(over)
    if a["wb"] is None:
        a["wb"] = L.gdn_kv_compact_workspace_bytes(a["n_pages"])
    return L.gdn_kv_compact(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(n_pages=0), 1), (dict(n_pages=1 << 29), 2), (dict(width=-1), 1), (dict(n=-1), 1), (dict(ts=7), 1), (dict(os=7), 1), (dict(n=1 << 28), 2),
    (dict(table=None), 1), (dict(out=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(info=None), 1), (dict(table=F + 2), 3),
    (dict(a=3 * F + 2), 3), (dict(ws=None), 4), (dict(wb=300), 4), (dict(ws=6 * F + 4), 3), (dict(out=F), 1), (dict(out=F + 4, os=8), 1),
    (dict(a=F + 8), 1), (dict(a=F, out=F, os=8), 1), (dict(b=3 * F + 196), 1), (dict(ws=2 * F), 1)])
def test_compact_refusals(L, over, status):
    assert compact(L, **over) == status
    assert L.gdn_last_error_string().decode()


def cache(i=0, **over):
    from gated_deltanet_linear_pre_gb300 import _native as N
    a = dict(heads=2, head_dim=128, page_tokens=64, n_pages=10, format=1, k=(4 * i + 1) * F, v=(4 * i + 2) * F, k_scale=(4 * i + 3) * F,
             v_scale=(4 * i + 4) * F)
    a.update(over)
    return N.gdn_kv_cache(*a.values())


def copy(L, caches, n=4, a=200 * F, b=201 * F, count=None):
    from gated_deltanet_linear_pre_gb300 import _native as N
    array = (N.gdn_kv_cache * len(caches))(*caches) if caches is not None else None
    return L.gdn_kv_copy(array, len(caches or []) if count is None else count, n, a, b, None)


def test_copy_refusals(L):
    two = [cache(0), cache(1)]
    for over, status in [(dict(n=-1), 1), (dict(count=-1), 1), (dict(count=1025), 2), (dict(a=None), 1), (dict(b=None), 1), (dict(a=200 * F + 2), 3),
                         (dict(b=F + 16), 1), (dict(a=8 * F), 1)]:
        assert copy(L, two, **over) == status, over
    assert copy(L, None, count=1) == 1
    for over, status in [(dict(heads=3), 1), (dict(head_dim=64), 1), (dict(page_tokens=32), 1), (dict(n_pages=9), 1), (dict(format=0), 1),
                         (dict(heads=0), 1), (dict(head_dim=96), 2), (dict(k=None), 1), (dict(v=6 * F + 8), 3), (dict(k=F), 1), (dict(v=5 * F), 1)]:
        assert copy(L, [cache(0), cache(1, **over)]) == status, over
    assert copy(L, []) == 0
    assert copy(L, two, n=0, a=None, b=None) == 0


def test_copy_of_many_caches(L):
    """An overlap is found wherever the two caches stand, and the search takes no time that a call would notice (a
    comparison of all pairs took 19 ms)."""
    at = random.Random(0).sample(range(1024), 1024)
    many = [cache(i) for i in at]
    lists = dict(a=5000 * F, b=5001 * F)
    assert copy(L, many, n=0, **lists) == 0
    best = min(timeit.repeat(lambda: copy(L, many, n=0, **lists), number=1, repeat=7))
    assert best < 6e-3, best
    for i, j in ((0, 1023), (1023, 0), (511, 512), (3, 700)):
        for mine, theirs in (("k", "v"), ("v", "v_scale"), ("k_scale", "k"), ("v_scale", "v_scale")):
            size, own = (163840 if name in ("k", "v") else 80 for name in (theirs, mine))
            for off, status in ((0, 1), (16, 1), (-16, 1), (size - 16, 1), (16 - own, 1), (size, 0), (-own, 0)):
                bad = list(many)
                bad[i] = cache(at[i], **{mine: getattr(many[j], theirs) + off})
                assert copy(L, bad, n=0, **lists) == status, (i, j, mine, theirs, off)
                assert status == 0 or b"overlaps" in L.gdn_last_error_string()
    assert copy(L, many, a=many[7].v + 64, b=5001 * F) == 1
    assert copy(L, many, a=5000 * F, b=many[900].k_scale) == 1


def test_lists_past_what_the_kernels_count(L):
    two = [cache(0), cache(1)]
    for n in ((1 << 30) + 1, (1 << 31) - 1024, (1 << 31) - 1):
        assert copy(L, two, n=n) == 2, n
        assert copy(L, [], n=n) == 2, n
        assert L.gdn_kv_remap_workspace_bytes(100, n, 0) == 0, n
        assert remap(L, n=n, width=0, wb=1 << 40) == 2, n


def test_workspaces(L):
    assert L.gdn_kv_remap_workspace_bytes(100, 5, 8) > 0 and L.gdn_kv_compact_workspace_bytes(100) >= 400
    for a in ((0, 5, 8), (-1, 5, 8), (100, -1, 8), (100, 5, -1), ((1 << 28) + 1, 5, 8), (100, 1 << 20, 1 << 20)):
        assert L.gdn_kv_remap_workspace_bytes(*a) == 0, a
    assert L.gdn_kv_compact_workspace_bytes(0) == L.gdn_kv_compact_workspace_bytes(-4) == L.gdn_kv_compact_workspace_bytes((1 << 28) + 1) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    from gated_deltanet_linear_pre_gb300 import _native as N
    t = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(TypeError):
        N._table(t, "page_table")
    with pytest.raises(TypeError):
        N.kv_caches([cache()])       # not from kv_cache(): nothing keeps its tensors
    with pytest.raises(TypeError):
        N.kv_caches([None])
    assert ctypes.sizeof(N.gdn_kv_cache) == 56
