"""Which of the adapters' workspace adapter_up reads, by the kernel's own index functions compiled for the host.

A form that once shipped read all 8 rows of a block of columns, whatever the adapter's rank, up to 28 KB behind the
workspace, and dropped what it read: no output shows that, so the indexes are counted here."""
import ctypes
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    lib = os.path.join(str(tmp_path_factory.mktemp("index")), "index.so")
    csrc = os.path.join(os.path.dirname(HERE), "gated_deltanet_linear_pre_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-x", "c++", "-I", csrc,
                    os.path.join(HERE, "host_adapter_index.cpp"), "-o", lib], check=True)
    L = ctypes.CDLL(lib)
    L.first_mistake.restype = ctypes.c_char_p
    L.mistakes.restype = ctypes.c_long
    return L


def test_every_read_of_h_was_written_for_its_tile(host):
    assert host.mistakes(0) == 0, host.first_mistake().decode()


def test_reads_that_the_rank_does_not_guard_are_found(host):
    assert host.mistakes(1) > 0
    assert "behind the workspace" in host.first_mistake().decode() or "not written" in host.first_mistake().decode()


def test_the_kernel_reads_through_these(host):
    """The kernel's only loads of h for its operand go through the functions that are counted here."""
    with open(os.path.join(os.path.dirname(HERE), "gated_deltanet_linear_pre_gb300", "csrc", "gdn_adapter.cu")) as f:
        text = f.read()
    body = text[text.index("void operand("):text.index("float inv = 1.0f, factor")]
    assert body.count("p.h") == 1 and "h_place(p.T, p.rank, r + i, t.start, r + i == b.x) + row" in body
    assert body.count("load_now(") == 1 and "load_now(src + (rows.at + e) * t.n, e < left)" in body
    assert "const OperandRows rows(steps, t.rank, col + j);" in body and "row < t.n && r + i <= b.y ? rows.left : 0" in body
