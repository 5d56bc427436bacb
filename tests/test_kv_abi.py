"""Host-side argument checks of the cache, attention and draft-check entries (no GPU: every call fails
before a launch, or has nothing to do)."""
import ctypes

import pytest

F = 1 << 30  # buffers 1 GB apart: no accidental overlap; never dereferenced


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    from gated_deltanet_linear_pre_gb300 import _native
    return _native.lib()


def cache(**over):
    from gated_deltanet_linear_pre_gb300 import _native as N
    a = dict(heads=2, head_dim=128, page_tokens=64, n_pages=10, format=1, k=F, v=2 * F, k_scale=3 * F, v_scale=4 * F)
    a.update(over)
    return N.gdn_kv_cache(*a.values())


def append(L, c, **over):
    a = dict(dtype=0, n=2, T=6, cu=5 * F, past=6 * F, table=7 * F, stride=8, width=8, hq=4, q=8 * F, qs=512, k=9 * F, ks=256, v=10 * F,
             vs=256, cos=11 * F, sin=12 * F, rot=128, n_pos=100, inter=0, q_out=13 * F)
    a.update(over)
    return L.gdn_kv_append(ctypes.byref(c) if c is not None else None, *a.values(), None)


def attn(L, c, **over):
    a = dict(dtype=1, n=2, T=6, cu=5 * F, past=6 * F, table=7 * F, stride=8, width=8, hq=4, q=8 * F, qs=512, scale=0.1, y=9 * F, ws=10 * F,
             wb=None)
    a.update(over)
    if a["wb"] is None:
        a["wb"] = L.gdn_kv_attn_workspace_bytes(ctypes.byref(c), a["n"], a["T"], a["hq"], a["width"]) if c is not None else 0
    return L.gdn_kv_attn(ctypes.byref(c) if c is not None else None, *a.values(), None)


CACHE_FAULTS = [(dict(heads=0), 1), (dict(n_pages=0), 1), (dict(heads=2000), 2), (dict(head_dim=96), 2), (dict(page_tokens=48), 2),
                (dict(page_tokens=256), 2), (dict(format=2), 1), (dict(k=None), 1), (dict(v=2 * F + 8), 3), (dict(k_scale=4 * F), 1),
                (dict(v=F + 16), 1)]
BATCH_FAULTS = [(dict(n=-1), 1), (dict(T=-1), 1), (dict(n=0), 1), (dict(n=70000), 2), (dict(cu=None), 1), (dict(past=None), 1),
                (dict(past=6 * F + 2), 3), (dict(table=None), 1), (dict(stride=7), 1), (dict(width=-1), 1), (dict(dtype=2), 1),
                (dict(q=None), 1), (dict(q=8 * F + 8), 3), (dict(qs=511), 1), (dict(qs=516), 3),
                (dict(width=1 << 25, stride=1 << 25), 2)]


@pytest.mark.parametrize("call", [append, attn], ids=["append", "attn"])
def test_shared_refusals(L, call):
    assert call(L, None) == 1
    for over, status in CACHE_FAULTS:
        assert call(L, cache(**over)) == status, over
    for over, status in BATCH_FAULTS:
        assert call(L, cache(), **over) == status, over
    assert call(L, cache(), T=1 << 30) == 2
    assert call(L, cache(), n=0, T=0) == 0            # nothing to do
    assert call(L, cache(), T=0) == 0


def test_append_refusals(L):
    c = cache()
    for over, status in [(dict(hq=-1), 1), (dict(hq=70000, qs=1 << 25), 2), (dict(inter=2), 1), (dict(rot=24), 2), (dict(rot=256), 2),
                         (dict(n_pos=0), 1), (dict(ks=255), 1), (dict(vs=260), 3), (dict(cos=None), 1), (dict(sin=12 * F + 4), 3),
                         (dict(q_out=None), 1), (dict(q_out=8 * F + 1024), 1), (dict(q_out=2 * F), 1), (dict(k=F + 64), 1)]:
        assert append(L, c, **over) == status, over
    assert append(L, c, q_out=9 * F) == 1
    assert "overlaps" in L.gdn_last_error_string().decode()


def test_attention_refusals(L):
    c = cache()
    for over, status in [(dict(hq=3, qs=512), 1), (dict(hq=1), 1), (dict(hq=2 * 65, qs=1 << 15), 2), (dict(scale=float("nan")), 1),
                         (dict(scale=float("inf")), 1), (dict(y=None), 1), (dict(y=9 * F + 4), 3), (dict(y=8 * F), 1), (dict(y=F + 32), 1),
                         (dict(ws=None), 4), (dict(ws=10 * F + 8), 3), (dict(ws=9 * F), 1)]:
        assert attn(L, c, **over) == status, over
    need = L.gdn_kv_attn_workspace_bytes(ctypes.byref(c), 2, 6, 4, 8)
    assert need > 0 and need % 8 == 0
    assert attn(L, c, wb=need - 1) == 4
    assert L.gdn_kv_attn_workspace_bytes(None, 2, 6, 4, 8) == 0
    assert L.gdn_kv_attn_workspace_bytes(ctypes.byref(c), 2, 0, 4, 8) == 0
    assert L.gdn_kv_attn_check(None, None) == 1


def test_verify_refusals(L):
    def call(**over):
        a = dict(n=2, d=3, vocab=100, p=F, ps=100, q=2 * F, qs=100, draft=3 * F, n_draft=4 * F, u=5 * F, acc=6 * F, nxt=7 * F)
        a.update(over)
        return L.gdn_draft_verify(*a.values(), None)

    for over, status in [(dict(n=-1), 1), (dict(d=-1), 1), (dict(n=65536), 2), (dict(d=65536), 2), (dict(vocab=0), 1),
                         (dict(vocab=(1 << 19) + 1, ps=1 << 20, qs=1 << 20), 2), (dict(ps=99), 1), (dict(qs=99), 1), (dict(p=None), 1),
                         (dict(q=None), 1), (dict(draft=None), 1), (dict(u=None), 1), (dict(acc=None), 1), (dict(nxt=None), 1),
                         (dict(p=F + 2), 3), (dict(nxt=7 * F + 1), 3), (dict(nxt=6 * F + 4), 1), (dict(acc=F + 64), 1)]:
        assert call(**over) == status, over
    assert call(n=0) == 0


def test_binding_refuses_cpu_tensors():
    import torch
    from gated_deltanet_linear_pre_gb300 import _native as N
    k = torch.zeros((2, 1, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        N.kv_cache(k, k, torch.zeros(2, 1), torch.zeros(2, 1))
    with pytest.raises(TypeError):
        N.gdn_draft_verify(torch.zeros(1, 2, 4), torch.zeros(1, 1, 4), None, None, None, None, None)


def test_workspace_of_refused_shapes_is_nothing(L):
    def need(hq=4, width=8, n=2, T=300, **over):
        return L.gdn_kv_attn_workspace_bytes(ctypes.byref(cache(**over)), n, T, hq, width)

    assert need() > 0
    assert need(hq=2 * 64) > 0
    for dim in (0, 1, 96, 256, -128):
        assert need(head_dim=dim) == 0, dim
    for page in (0, 8, 48, 256, -16):
        assert need(page_tokens=page) == 0, page
    for hq in (-4, 0, 1, 3, 2 * 65, 2 * 129, 2 * 4000):
        assert need(hq=hq) == 0, hq
    assert need(heads=0) == need(heads=-2) == need(width=-1) == need(n=-1) == need(T=-1) == 0
