"""Shared arrays that are read or written 16 bytes at a time say so in their declaration: where the compiler places an
array of smaller elements is otherwise up to its neighbours."""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "rollout_x128_act_gb300", "csrc", "*.cu*")))
WIDE = r"(?:u?int4|float4|u?longlong2|double2)"


def unaligned(source):
    """(line, name) of the shared arrays that are cast to a 16-byte vector without being declared aligned to one."""
    found = []
    for m in re.finditer(r"^[ \t]*__shared__ ([^;]*);", source, re.M):
        decl = m.group(1)
        if "__align__(" in decl or "alignas(" in decl or re.match(WIDE + r"\b", decl):
            continue
        body = source[m.end():source.find("\n}\n", m.end())]  # the kernel's
        for name in re.findall(r"(\w+)(?:\[[^\]]*\])+", decl):
            if re.search(r"reinterpret_cast<(?:const )?(?:volatile )?" + WIDE + r" \*>\(&?" + name + r"\b", body):
                found.append((source[:m.start()].count("\n") + 1, name))
    return found


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_arrays_read_as_vectors_are_aligned(path):
    with open(path) as f:
        assert unaligned(f.read()) == []


def test_the_search_finds_them():
    kernel = "void k()\n{\n    __shared__ %s;\n    use(reinterpret_cast<const uint4 *>(marks)[0]);\n}\n"
    assert unaligned(kernel % "uint32_t marks[4]") == [(3, "marks")]
    assert unaligned(kernel % "alignas(16) uint32_t marks[4]") == []
    assert unaligned(kernel % "__align__(16) uint32_t marks[4]") == []
    assert unaligned(kernel % "uint4 marks[4]") == []
    assert unaligned(kernel % "uint32_t others[4]") == []
