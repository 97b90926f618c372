"""Inline assembly of the kernels names every register that it writes beside its outputs (CPU
only, on the source): the compiler may hold an m0, vcc or scc of its own across the statement."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "place_batchnorm_activation_amd", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".hpp")))


def statements(text):
    """(assembly, clobbers) of every asm statement."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        body = text[m.end():at - 1]
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body.split(":")[0]))
        parts = re.split(r":", re.sub(r'"(?:[^"\\]|\\.)*"', lambda s: s.group().replace(":", ";"),
                                      body))
        yield code, set(re.findall(r'"([^"]*)"', parts[3])) if len(parts) > 3 else set()


def written(code):
    """Fixed registers that instructions of the statement write (their first operand)."""
    out = set()
    for line in re.split(r"\\n|;", code):
        words = line.replace("\\t", " ").split()
        if len(words) > 1 and not words[0].startswith(("s_waitcnt", "s_nop", "s_barrier")):
            dst = words[1].rstrip(",")
            if dst in ("m0", "vcc", "exec", "scc") or re.fullmatch(r"[vas]\d+|[vas]\[\d+:\d+\]", dst):
                out.add(dst)
    return out


@pytest.mark.parametrize("name", FILES)
def test_written_registers_are_clobbered(name):
    with open(os.path.join(CSRC, name)) as fh:
        for code, clobbers in statements(fh.read()):
            assert written(code) <= clobbers, code


def test_the_check_sees_a_write():
    text = r'asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tds_read_b32 v7, %1" :: "s"(a), "v"(b) : "memory");'
    (code, clobbers), = statements(text)
    assert written(code) == {"m0", "v7"} and clobbers == {"memory"}
