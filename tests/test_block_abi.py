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
