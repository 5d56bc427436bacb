"""The library with gdn_adapter.cu compiled another way, for tests of what its rules or its luck would not show."""
import glob
import os
import subprocess


def adapter_library(out, macro):
    """Path of the library, below the folder `out`, with `macro` defined for the adapters' kernels."""
    from gated_deltanet_linear_pre_gb300 import build
    build.build()
    obj, lib = os.path.join(out, "adapter.o"), os.path.join(out, "libgdn_selftest.so")
    nvcc = build._nvcc()
    src = os.path.join(build.CSRC, "gdn_adapter.cu")
    subprocess.run([nvcc, *build.ARCH, *build.NVCC_FLAGS, "-D" + macro, "-c", src, "-o", obj], check=True)
    others = [o for o in glob.glob(os.path.join(build.BUILD, "*.o")) if not o.endswith("gdn_adapter.o")]
    libs = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    subprocess.run([nvcc, *build.ARCH, "-shared", "-cudart", "shared", "-o", lib, obj, *others, "-Xlinker", f"-rpath,{libs}"], check=True)
    return lib
