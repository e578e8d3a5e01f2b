"""Which buffers the operators' kernels read through the non-coherent path.

Each is a programmatic dependent launch: it may be resident while the kernel before it still writes what
it is going to read.  The non-coherent load (__ldg, ld.global.nc, and what the compiler makes of a
const __restrict__ pointer) asks for memory that nobody writes while the kernel lives, and the dependency
wait does not order it; it is for a handle's packed weights only.
"""
import os
import re

from gemv_projection_layers_gb300 import build as libbuild

FILES = ["moe.cu", "norm.cu", "vec.cuh", "w4.cu", "w4_num.cuh", "w4_tc.cu"]
WEIGHTS = {"codes", "scales", "zeros"}


def source(name):
    text = open(os.path.join(libbuild.CSRC, name)).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_non_coherent_loads_are_of_packed_weights():
    found = []
    for name in FILES:
        text = source(name)
        assert ".nc." not in text, name
        found += [(name, *m) for m in re.findall(r"\b(__ldg|ld_stream_v4)\(\s*(?:p\.)?(\w+)", text)]
    assert found, "the weights at least are read so"
    assert not [f for f in found if f[2] not in WEIGHTS], found


def test_restrict_is_for_the_packing_kernels():
    """They run when a handle is made, as ordinary launches."""
    for name in FILES:
        for part in re.split(r"(?=__global__|__device__)", source(name)):
            head = part.split("{")[0]
            if "__restrict__" in head:
                assert re.search(r"\bpack_\w+_kernel\(", head), (name, head)
