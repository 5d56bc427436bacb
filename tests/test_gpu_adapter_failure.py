"""Failure detection of the adapters' tensor-core kernels without a fault: their waits are bounded, and one that
expires is reported to the host.

A library of its own is built here in which every CTA of those kernels leaves out its first copy.  The product warp's
wait for it runs out (seconds), and with it the waits of the CTA's other warps; the CTA begins nothing more, waits for
what it has under way, frees its tensor memory and ends.  gdn_adapter_check then reports GDN_ERR_TIMEOUT, and the same
context, workspace and buffers go on to compute right results."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def withholding(tmp_path_factory):
    """Path of the library without those kernels' first copies."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from selftest_lib import adapter_library
    return adapter_library(str(tmp_path_factory.mktemp("withholding")), "GDN_ADAPTER_SELFTEST_WITHHOLD_COPY")


@pytest.mark.parametrize("lengths,rank", [([3000, 5, 700, 1], 64), ([40, 900], 128)])
def test_expired_wait_is_reported_and_the_next_call_is_right(withholding, monkeypatch, lengths, rank):
    import gated_deltanet_linear_pre_gb300 as gdn
    from gated_deltanet_linear_pre_gb300 import _native
    from test_gpu_adapter import Case
    n = len(lengths)
    c = Case(lengths, [i % 2 for i in range(n)], 2, rank, 1000, 2120, "bf16", seed=4)
    ws = torch.full((gdn.gdn_adapter_workspace_bytes(n, c.T, rank, 1000),), 0xA5, dtype=torch.uint8, device="cuda")
    good = c.run(gdn, workspace=ws).clone()
    gdn.gdn_adapter_check(ws)
    with monkeypatch.context() as m:
        m.setattr(_native, "_lib", None)
        m.setattr(_native._build, "LIB", withholding)
        c.run(gdn, workspace=ws)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_adapter_check(ws)
        assert e.value.status == 6 and "expired" in str(e.value)
    gdn.gdn_last_async_error()                        # no fault was seen: the context is intact
    assert torch.equal(c.run(gdn, workspace=ws), good)
    gdn.gdn_adapter_check(ws)


def test_check_of_few_tokens_is_clean():
    """A batch that never waits leaves a clean record, whatever the workspace held."""
    import gated_deltanet_linear_pre_gb300 as gdn
    from test_gpu_adapter import Case
    c = Case([1, 2, 1], [0, 1, -1], 2, 16, 256, 512, "fp16")
    ws = torch.full((gdn.gdn_adapter_workspace_bytes(3, 4, 16, 256),), 0xA5, dtype=torch.uint8, device="cuda")
    c.check(c.run(gdn, workspace=ws))
    gdn.gdn_adapter_check(ws)
