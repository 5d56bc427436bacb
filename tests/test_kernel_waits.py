"""Kernels that may start while the one in front of them still runs: each waits for it before it reads any global memory.

Only the grid that waits is promised to see what was written before, so the wait belongs to every block of every kernel,
whoever wrote its inputs.  This reads the sources: a kernel's first statements, up to a wait that no condition guards."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_pre_gb300", "csrc")
# the chunk recurrence takes each chunk when the flag of its preparation is set, and waits at its end
BY_FLAGS = {"scan_chain_kernel"}
READS = re.compile(r"__ld|ld\.global|\bp\.\w+\s*\[|\bp\.\w+\s*\+|cu_at|few_tile|find_starts|\.next\(|_g2s|atomic|cp\.async\.(cg|ca|bulk)")


def kernels(text):
    """(name, body) of each kernel's definition."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__[^{;]*?(\w+_kernel)\((?:[^()]|\([^()]*\))*\)\s*\{", text):
        depth, end = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        yield m.group(1), text[m.end():end - 1]


def before_wait(body):
    """The statements in front of the first wait that every block comes to, or None."""
    depth, seen = 0, []
    for line in body.split("\n"):
        if depth == 0 and re.match(r"\s*pdl_wait\(\);", line):
            return "\n".join(seen)
        depth += line.count("{") - line.count("}")
        seen.append(line)
    return None


def all_kernels():
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            found += [(os.path.basename(path), *k) for k in kernels(f.read())]
    return found


@pytest.mark.parametrize("file,name,body", all_kernels(), ids=lambda v: v if isinstance(v, str) and len(v) < 40 else "")
def test_waits_before_it_reads(file, name, body):
    if name in BY_FLAGS:
        assert "flag_wait" in body and "pdl_wait();" in body
        return
    head = before_wait(body)
    assert head is not None, "no wait that every block comes to"
    assert not READS.search(head), READS.search(head).group(0)


def test_this_finds_the_kernels_and_their_mistakes():
    names = [k[1] for k in all_kernels()]
    assert len(names) >= 20 and {"few_down_kernel", "few_up_kernel", "adapter_up_kernel", "scan_chain_kernel", "block_norm_kernel"} <= set(names)
    ok = "__global__ void __launch_bounds__(32) a_kernel(const P p)\n{\n    int i = 0;\n    pdl_wait();\n    f(p.x[0]);\n}\n"
    (name, body), = kernels(ok)
    assert name == "a_kernel" and before_wait(body) is not None and not READS.search(before_wait(body))
    assert before_wait(next(kernels(ok.replace("    pdl_wait();", "    if (i) pdl_wait();")))[1]) is None
    assert before_wait(next(kernels(ok.replace("    pdl_wait();", "    if (i) {\n    pdl_wait();\n    }")))[1]) is None
    assert READS.search(before_wait(next(kernels(ok.replace("int i = 0;", "int i = __ldg(p.x);")))[1]))
