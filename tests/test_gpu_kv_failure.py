"""Failure detection of the attention's prompt kernel without a fault: its waits are bounded, and one that
expires is reported to the host.

A library of its own is built here in which every CTA of that kernel leaves out its first copy.  The products'
wait for it runs out (about two seconds), and with it, as they give up once one has, the waits of the CTA's
other warps; the kernel waits for what it has under way, frees its tensor memory and ends.
gdn_kv_attn_check then reports GDN_ERR_TIMEOUT, and the same context, workspace and buffers go on to compute
a correct attention."""
import glob
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def withholding(tmp_path_factory):
    """Path of the library without the prompt kernel's first copies."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    out = tmp_path_factory.mktemp("withholding")
    obj, lib = str(out / "prompt.o"), str(out / "libgdn_withholding.so")
    nvcc = build._nvcc()
    src = os.path.join(build.CSRC, "gdn_kv_prompt.cu")
    subprocess.run([nvcc, *build.ARCH, *build.NVCC_FLAGS, "-DGDN_KV_SELFTEST_WITHHOLD_COPY", "-c", src, "-o", obj], check=True)
    others = [o for o in glob.glob(os.path.join(build.BUILD, "*.o")) if not o.endswith("gdn_kv_prompt.o")]
    libs = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    subprocess.run([nvcc, *build.ARCH, "-shared", "-cudart", "shared", "-o", lib, obj, *others, "-Xlinker", f"-rpath,{libs}"], check=True)
    return lib


@pytest.mark.parametrize("new,past,hq,heads,dim", [
    ([150, 1, 90], [700, 300, 10], 8, 2, 128),        # cut units
    ([333, 40, 1, 300], [30, 0, 500, 100], 128, 32, 64),  # more units than CTAs: handed out
])
def test_expired_wait_is_reported_and_the_next_call_is_right(withholding, monkeypatch, new, past, hq, heads, dim):
    import gated_deltanet_linear_pre_gb300 as gdn
    from gated_deltanet_linear_pre_gb300 import _native
    from test_gpu_kv_attention import Batch
    b = Batch(new, past, hq, heads, dim, 64, "int8", "bf16", seed=7)
    b.fill_past()
    b.append()
    good = b.attend().clone()
    size = gdn.gdn_kv_attn_workspace_bytes(b.cache, len(new), b.T, hq, b.table.shape[1])
    ws = torch.full((size,), 0xA5, dtype=torch.uint8, device="cuda")
    with monkeypatch.context() as m:
        m.setattr(_native, "_lib", None)
        m.setattr(_native._build, "LIB", withholding)
        with pytest.raises(gdn.GdnError) as e:
            b.attend(workspace=ws)
        assert e.value.status == 6 and "expired" in str(e.value)
    gdn.gdn_last_async_error()                        # no fault was seen: the context is intact
    assert torch.equal(b.attend(workspace=ws), good)
