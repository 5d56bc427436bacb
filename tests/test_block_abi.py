"""Host-side argument checks of the entries around the layers (no GPU: every call fails before a launch, or
has nothing to do)."""
import pytest

F = 1 << 34  # buffers 16 GB apart: no accidental overlap; never dereferenced


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    from gated_deltanet_linear_pre_gb300 import _native
    return _native.lib()


def norm(L, **over):
    a = dict(x_dtype=1, dtype=1, T=6, width=256, x=F, xs=256, y=2 * F, ys=512, gate=3 * F, gs=0, kind=2, scale=1.0, post=4 * F, pre=5 * F,
             eps=1e-6, x_out=6 * F, h=7 * F)
    a.update(over)
    return L.gdn_block_norm(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2, x_dtype=2), 1), (dict(dtype=3), 1), (dict(x_dtype=0), 1), (dict(x_dtype=3), 1), (dict(T=-1), 1), (dict(width=0), 1),
    (dict(width=-8), 1), (dict(width=252, xs=256, ys=256), 2), (dict(width=16392, xs=1 << 15, ys=1 << 15), 2), (dict(kind=-1), 1),
    (dict(kind=4), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(x_out=None, h=None, pre=None), 1), (dict(h=None), 1), (dict(pre=None), 1),
    (dict(kind=0), 1), (dict(gate=None), 1), (dict(y=None), 1), (dict(y=None, gate=None, kind=0, post=None), 1),
    (dict(y=None, gate=None, kind=0, x_out=None), 1), (dict(xs=248), 1), (dict(xs=260), 3), (dict(ys=255), 1), (dict(gs=8), 1), (dict(gs=260), 3),
    (dict(xs=1 << 31), 2), (dict(ys=(1 << 30) + 8), 2), (dict(x=None), 1), (dict(x=F + 8), 3), (dict(y=2 * F + 2), 3), (dict(post=4 * F + 4), 3),
    (dict(h=7 * F + 8), 3), (dict(x_out=F, xs=512), 1), (dict(x_out=F + 16), 1), (dict(x_out=2 * F), 1), (dict(h=F), 1), (dict(h=6 * F), 1),
    (dict(h=F, x_out=F), 1), (dict(h=3 * F), 1), (dict(x_out=5 * F), 1), (dict(x_dtype=2, x_out=7 * F - 16), 1)])
def test_norm_refusals(L, over, status):
    assert norm(L, **over) == status
    assert L.gdn_last_error_string().decode()


def test_norm_without_tokens(L):
    assert norm(L, T=0) == 0
    assert norm(L, T=0, x=None, y=None, gate=None, kind=0, post=None, x_out=None) == 0


def test_binding_refusals():
    import torch
    from gated_deltanet_linear_pre_gb300 import _native as N
    x = torch.zeros((2, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        N.gdn_block_norm(x.int(), x, None, "none", 1.0, None, None, 1e-6, x, None)
    with pytest.raises(TypeError):
        N.gdn_block_norm(x, x.float(), None, "none", 1.0, None, None, 1e-6, x, None)
    with pytest.raises(ValueError):
        N.gdn_block_norm(x, x, None, "tanh", 1.0, None, None, 1e-6, x, None)


def adapter(L, **over):
    a = dict(dtype=1, n=3, T=100, cu=F, ids=2 * F, n_adapters=4, rank=16, ranks=3 * F, down=4 * F, up=5 * F, scales=6 * F, d_in=256, x=7 * F, xs=256,
             d_out=512, y=8 * F, ys=1024, out=9 * F, os=512, ws=10 * F, wb=None)
    a.update(over)
    if a["wb"] is None:
        a["wb"] = L.gdn_adapter_workspace_bytes(a["n"], a["T"], a["rank"], a["d_in"])
    return L.gdn_adapter_add(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(n=-1), 1), (dict(T=-1), 1), (dict(n=0), 1), (dict(n=65536), 2), (dict(cu=None), 1),
    (dict(cu=F + 2), 3), (dict(n_adapters=-1), 1), (dict(rank=0), 2), (dict(rank=12), 2), (dict(rank=136), 2), (dict(d_in=0, xs=256), 2),
    (dict(d_in=252, xs=256), 2), (dict(d_in=65544, xs=1 << 17), 2), (dict(d_out=508), 2), (dict(xs=248), 1), (dict(xs=260), 3), (dict(ys=511), 1),
    (dict(ys=1 << 31), 2), (dict(os=504), 1), (dict(os=516), 3), (dict(ids=None), 1), (dict(ids=2 * F + 1), 3), (dict(ranks=3 * F + 2), 3),
    (dict(down=None), 1), (dict(down=4 * F + 8), 3), (dict(up=None), 1), (dict(scales=None), 1), (dict(x=None), 1), (dict(x=7 * F + 8), 3),
    (dict(y=None), 1), (dict(out=None), 1), (dict(ws=None), 4), (dict(wb=100), 4), (dict(ws=10 * F + 8), 3), (dict(out=8 * F), 1),
    (dict(out=8 * F + 16, os=1024), 1), (dict(out=7 * F), 1), (dict(out=5 * F, os=512), 1), (dict(ws=7 * F), 1), (dict(ws=9 * F + 256), 1),
    (dict(out=8 * F, os=1024, ws=8 * F + 4096), 1), (dict(out=6 * F), 1)])
def test_adapter_refusals(L, over, status):
    assert adapter(L, **over) == status
    assert L.gdn_last_error_string().decode()


def test_adapter_without_tokens(L):
    assert adapter(L, T=0) == 0
    assert adapter(L, T=0, n=0, x=None, y=None, out=None, ids=None, ws=None, wb=0) == 0


def test_adapter_workspace(L):
    assert L.gdn_adapter_workspace_bytes(3, 100, 16, 256) >= 100 * 16 * 4
    for a in ((3, 0, 16, 256), (-1, 100, 16, 256), (0, 100, 16, 256), (65536, 100, 16, 256), (3, -1, 16, 256), (3, 100, 0, 256), (3, 100, 20, 256),
              (3, 100, 136, 256), (3, 100, 16, 0), (3, 100, 16, 260), (3, 100, 16, 70000)):
        assert L.gdn_adapter_workspace_bytes(*a) == 0, a
