"""The paged 8-bit cache and its attention where values are not finite or differ in size by many powers of
two: what a row does not see does not reach it, and what a call does not store leaves no mark."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()


def batch(*args, **kw):
    from test_gpu_kv_attention import Batch
    return Batch(*args, **kw)


def same_cache(a, b):
    for x, y in ((a.k, b.k), (a.v, b.v), (a.ks, b.ks), (a.vs, b.vs)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ---- the append -------------------------------------------------------------------------------------

@pytest.mark.parametrize("new,past,page", [([1], [3], 64), ([1, 1, 1], [3, 3, 70], 16), ([5], [3], 64), ([9, 2], [70, 71], 32),
                                           ([40] * 40, [5] * 40, 16), ([300], [17], 128), ([130, 129], [17, 17], 32)])
@pytest.mark.parametrize("dim,rot,interleaved", [(128, None, False), (128, 64, True), (64, 32, False)])
def test_append_reads_the_rotation_of_its_own_positions(new, past, page, dim, rot, interleaved):
    """Rows of the rotation table that belong to no token of the call may hold anything."""
    a, b = (batch(new, past, 4, 2, dim, page, "int8", "bf16", seed=3, rot=rot, interleaved=interleaved) for _ in range(2))
    used = sorted({p + i for n, p in zip(new, past) for i in range(n)})
    for x in (a, b):
        x.fill_past()
    for t in (b.cos, b.sin):
        kept = t[used].clone()
        t.fill_(float("nan"))
        t[used] = kept
    assert torch.equal(a.append(), b.append())
    same_cache(a, b)
