"""What a kernel that is launched while the kernel before it still runs may not do, read
off the sources (no device needed)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "attention_decode_megakernel_b200", "csrc")


def _code(path):
    text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _with_headers(path, seen):
    if path not in seen:
        seen.add(path)
        for name in re.findall(r'#include "(mk_\w+\.cuh)"', open(path).read()):
            _with_headers(os.path.join(CSRC, name), seen)
    return seen


def test_no_loads_that_need_constant_memory():
    """Non-coherent loads are for memory that nothing writes while the kernel lives. The
    operators' kernels live while the kernel in front, a cache write say, still writes."""
    files = set()
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        if re.search(r"\blaunch\(", _code(path)) and "mk_ops.cuh" in open(path).read():
            _with_headers(path, files)
    assert {"mk_flash.cuh", "mk_paged.cuh", "mk_kvcache.cuh"} <= {os.path.basename(f) for f in files}
    for path in sorted(files):
        for what in (r"__ldg\b", r"ld\.global\.nc", r"\b__restrict__\b"):
            assert not re.search(what, _code(path)), (os.path.basename(path), what)
