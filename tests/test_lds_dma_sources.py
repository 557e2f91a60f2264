"""lds_dma writes M0 behind the compiler's back, and the builtin transfers into LDS keep their target in M0
across instructions: no source file, with the headers it includes, may use both."""
import os
import re

from sparse_rank_adapter_amd import build

ASM = re.compile(r"\blds_dma\s*\(")
BUILTIN = re.compile(r"__builtin_amdgcn_\w*load\w*lds|__builtin_amdgcn_(?:ds_gws|s_sendmsg|interp)\w*")


def text(path, seen):
    """The file's code and that of the project headers it includes, without comments."""
    if path in seen or not os.path.exists(path):
        return ""
    seen.add(path)
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
    return code + "".join(text(os.path.join(os.path.dirname(path), h), seen) for h in re.findall(r'#include "([^"]+)"', code))


def calls(src):
    """(calls of lds_dma outside its definition, builtin transfers)"""
    t = text(os.path.join(build.CSRC, src), set())
    return len(ASM.findall(t)) - len(re.findall(r"void lds_dma\s*\(", t)), len(BUILTIN.findall(t))


def test_one_kind_of_transfer_per_file():
    found = {s: calls(s) for s in build.SOURCES if os.path.exists(os.path.join(build.CSRC, s))}
    assert any(a for a, _ in found.values()) and any(b for _, b in found.values())  # the search finds both kinds
    assert [s for s, (a, b) in found.items() if a and b] == []
