"""A CUDA source of the library compiled for the host (host_cuda.h).

``translate`` takes the text of a .cu file and turns what a host compiler does
not know into what host_cuda.h has: includes go, dynamic shared memory becomes
a pointer that is never followed (every access to it is inline PTX), and each
inline PTX statement becomes a call of the function of its name, outputs
first:

    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    ptx::ld_shared_u32(v, a);
"""
from __future__ import annotations

import os
import re
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "linear_attention_recurrence_step_gb300", "csrc")


def _sections(text, start):
    """The parts of an asm(...) whose '(' is at `start`, split at its colons, and
    the index after its ')'."""
    parts, depth, i, begin, quoted = [], 0, start, start + 1, False
    while True:
        c = text[i]
        if quoted:
            if c == "\\":
                i += 1
            elif c == '"':
                quoted = False
        elif c == '"':
            quoted = True
        elif c == "(":
            depth += 1
        elif c == ")":
            depth -= 1
            if depth == 0:
                return parts + [text[begin:i]], i + 1
        elif c == ":" and depth == 1:
            parts.append(text[begin:i])
            begin = i + 1
        i += 1


def _operands(section):
    """The expressions of a section: "=r"(x), "r"(y + 1) -> ["x", "y + 1"]."""
    found, i = [], 0
    while True:
        i = section.find("(", i)
        if i < 0:
            return found
        depth, j = 1, i + 1
        while depth:
            depth += {"(": 1, ")": -1}.get(section[j], 0)
            j += 1
        found.append(section[i + 1:j - 1])
        i = j


def translate(text: str) -> str:
    text = re.sub(r"^#\s*(include|pragma once).*$", "", text, flags=re.M)
    text = re.sub(r"extern __shared__[^;]*?(\w+)\[\];", r"unsigned char *const \1 = nullptr;", text)
    out, i = [], 0
    for hit in re.finditer(r"\basm(?: volatile)?(?=\()", text):
        parts, end = _sections(text, hit.end())
        name = re.match(r'\s*"\s*([\w.:]+)', parts[0]).group(1)
        args = [e for s in parts[1:3] for e in _operands(s)]
        out += [text[i:hit.start()], "ptx::", re.sub(r"\W+", "_", name), "(", ", ".join(args), ")"]
        i = end
    return "".join(out + [text[i:]])


def compile_unit(sources, entry: str, out_dir: str, name: str) -> str:
    """A shared library of the csrc files named, one after another, and the C
    entry given."""
    unit = ['#include "host_cuda.h"\nuint3 threadIdx, blockIdx;\ndim3 blockDim, gridDim;\n',
            "namespace gdn { enum class DType : int { F32 = 0, BF16 = 1, F16 = 2 }; }\n"]
    for s in sources:
        with open(os.path.join(CSRC, s)) as f:
            unit.append(translate(f.read()))
    unit.append(entry)
    src, lib = os.path.join(out_dir, name + ".cpp"), os.path.join(out_dir, name + ".so")
    with open(src, "w") as f:
        f.write("\n".join(unit))
    subprocess.run(["g++", "-std=c++17", "-O2", "-fno-strict-aliasing", "-ffp-contract=off", "-fPIC", "-shared", "-w",
                    "-I", HERE, src, "-o", lib], check=True)
    return lib
