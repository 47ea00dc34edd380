"""Arrays of the kernels that are read or written as 16-byte vectors say so in their declaration: an array of 4-byte
elements is only sure of 4 bytes, and where it lands otherwise is the compiler's choice."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CAST = re.compile(r"reinterpret_cast<(?:const )?(?:float4|uint4|int4|double2)\*>\(&?(\w+)\[")


def declarations(src, name):
    """Statements that declare an array `name` of scalars."""
    return re.findall(rf"^[^\n;/]*\b(?:float|uint32_t|int32_t|uint8_t|double)\s+(?:\w+\[[^;]*\],\s*)*{name}\[[^\n;]*;", src, re.M)


def test_arrays_accessed_as_vectors_are_aligned():
    seen = 0
    for path in glob.glob(os.path.join(ROOT, "long_context_sparse_11_b200", "csrc", "*.cuh")):
        src = open(path).read()
        for name in set(CAST.findall(src)):
            for line in declarations(src, name):
                seen += 1
                assert "__align__(16)" in line, (os.path.basename(path), line)
    assert seen
