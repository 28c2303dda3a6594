"""A block of a tensor-core kernel leaves at its start as a whole or not at all.

The status word may change while the threads of one block read it (another
block records an expired wait), so a kernel whose warps share barriers, a wait
bound and tensor memory must not let threads return on their own reading of
it.  Read from the sources: no GPU takes part.
"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "variable_length_sequence_gb300", "csrc")


def kernels(text):
    """(name, body) of every __global__ function of a source."""
    for m in re.finditer(r"__global__", text):
        # the body is the first brace outside parentheses
        start = depth = 0
        for i in range(m.end(), len(text)):
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            if text[i] == "{" and depth == 0:
                start = i
                break
        level, end = 0, start
        for end in range(start, len(text)):
            level += {"{": 1, "}": -1}.get(text[end], 0)
            if level == 0:
                break
        names = re.findall(r"(\w+)\s*\(", text[m.end():start])
        yield next(n for n in names if not n.startswith("__")), text[start:end + 1]


def test_tensor_core_kernels_leave_as_a_block():
    seen = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for name, body in kernels(text):
            if "tmem_alloc(" not in body:
                continue
            seen.append(name)
            at = body.index("tmem_alloc(")
            reads = [m.start() for m in re.finditer(r"status_bad\(", body)]
            assert reads and reads[-1] < at, name
            for r in reads:
                assert re.search(r"block_leaves\(\s*$", body[:r]), name
    assert len(seen) == 7, seen
