"""The rule of kernels that are set up while the kernel before them ends, read
from their sources: a kernel launched by launch_dependent waits for the stream,
and takes no tensor memory before it does (a kernel before it that lets its
dependents start early and wants tensor memory itself would wait for this one,
which waits for that one's end).  Needs no GPU: the case that would hang is not
run anywhere."""

import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_vector_15_b200", "csrc")


def kernels():
    """(file, name, body) of every kernel in a file that launches by launch_dependent."""
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        if "launch_dependent(" not in text:
            continue
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(k_\w+)\s*\(", text):
            at, depth = text.index("{", m.end()), 0
            for end in range(at, len(text)):
                depth += (text[end] == "{") - (text[end] == "}")
                if depth == 0:
                    break
            found.append((os.path.basename(path), m.group(1), text[at:end]))
    return found


def test_every_kernel_is_found():
    names = {n for _, n, _ in kernels()}
    launched = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        for call in re.findall(r"launch_dependent\(([^;]*);", re.sub(r"//[^\n]*", "", open(path).read())):
            launched |= set(re.findall(r"\bk_\w+", call))
    assert launched and launched <= names, launched - names


def test_kernels_wait_before_they_take_tensor_memory_or_touch_global_memory():
    for path, name, body in kernels():
        wait = body.find("wait_for_stream()")
        assert wait >= 0, (path, name)
        before = body[:wait]
        for taken in ("tmem_alloc(", "tcgen05.alloc", "P.desc", "seq_of(", "part_of<", "atomicOr(", "return;"):
            assert taken not in before, (path, name, taken)
