"""Reads the order of kernels launched with programmatic serialization out of the
CUDA sources, without a GPU.

Such a kernel may start before its predecessor on the stream has finished, and a
successor's wait covers this kernel alone.  So a grid has to wait
(``griddepcontrol.wait``, ``pdl_wait()``) before it may end, or what follows it loses
its order behind what came before it.  ``unwaited_exits`` lists the ways out of a
kernel on which that is not certain.
"""
from __future__ import annotations

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "head_latent_attention_absorbed_gb300", "csrc")


def source() -> str:
    """Every source file, without comments and preprocessor lines."""
    text = "\n".join(open(f).read() for f in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))))
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return re.sub(r"^\s*#[^\n]*(\\\n[^\n]*)*", " ", text, flags=re.M)


def closing(text: str, at: int) -> int:
    """Index behind the bracket that closes the one at ``at``."""
    pairs = {"(": ")", "{": "}", "[": "]"}
    depth, i = 0, at
    while True:
        if text[i] == '"':
            i = text.index('"', i + 1)
        elif text[i] in pairs:
            depth += 1
        elif text[i] in pairs.values():
            depth -= 1
            if depth == 0:
                return i + 1
        i += 1


def body_of(kernel: str, text: str) -> str:
    """The statements of a __global__ function."""
    for m in re.finditer(r"__global__\b", text):
        at = m.end()
        head = text.index("{", at)
        if re.search(rf"\b{kernel}\s*\(", text[at:head]):
            return text[head:closing(text, head)]
    raise KeyError(kernel)


def overlapped_kernels(text: str):
    """Names of the kernels that are launched with programmatic serialization."""
    names = set()
    for m in re.finditer(r"\blaunch_pdl\s*\(", text):
        call = text[m.end() - 1:closing(text, m.end() - 1)]
        names.update(re.findall(r"\b(\w+_kernel)\b", call))
    # launched with an attribute list of their own
    for m in re.finditer(r"ProgrammaticStreamSerialization;", text):
        call = re.search(r"cudaLaunchKernelEx\(&cfg,\s*(\w+)", text[m.end():])
        if call.group(1) != "kernel":           # launch_pdl itself
            names.add(call.group(1))
    return sorted(names)


# Conditions that only tell the threads of a CTA, or the instances of a template, apart:
# some thread of every CTA takes the branch.
ROLE = re.compile(r"^[\s!&|()=<>\d+]*((warp|tid|lane|kSoftWarps|k[A-Z]\w*|L::k\w+)[\s!&|()=<>\d+]*)+$")
# A condition that some CTA of every grid meets: it is the first along an axis.
FIRST = re.compile(r"\b(r0|j0|blockIdx\.[xyz])\s*==\s*0\b(?!\s*&&)")


def statement(text: str, i: int):
    """(kind, parts, end) of the statement at ``i``."""
    while text[i].isspace():
        i += 1
    if text[i] == "{":
        end = closing(text, i)
        return "block", text[i + 1:end - 1], end
    m = re.match(r"(if\s+constexpr|if|for|while)\s*\(", text[i:])
    if m:
        c0 = i + m.end() - 1
        c1 = closing(text, c0)
        end = statement(text, c1)[2]
        parts = [text[c0 + 1:c1 - 1], text[c1:end], None]
        kind = "if" if m.group(1).startswith("if") else "loop"
        if kind == "if":
            e = re.match(r"\s*else\b", text[end:])
            if e:
                e0 = end + e.end()
                end = statement(text, e0)[2]
                parts[2] = text[e0:end]
        return kind, parts, end
    if re.match(r"do\b", text[i:]):
        e0 = statement(text, i + 2)[2]
        return "block", text[i + 2:e0], text.index(";", e0) + 1
    j = i
    while text[j] != ";":
        j = closing(text, j) if text[j] in "({[" else j + 1
    return "plain", text[i:j], j + 1


def walk(text: str, waited: bool, exits: list):
    """Whether the CTA has waited where ``text`` falls through (None: it never does)."""
    i = 0
    while text[i:].strip():
        kind, part, i = statement(text, i)
        if kind == "plain":
            s = part.strip()
            if re.match(r"return\b", s):
                if not waited:
                    exits.append(s)
                return None
            if s == "pdl_wait()":
                waited = True
        elif kind == "block":
            w = walk(part, waited, exits)
            if w is None:
                return None
            waited = w
        elif kind == "loop":
            walk(part[1], waited, exits)    # may run no time
        else:
            cond, then, other = part
            a = walk(then, waited, exits)
            b = walk(other, waited, exits) if other is not None else waited
            if a is None and b is None:
                return None
            if ROLE.match(cond):            # some threads go one way, others the other
                waited = bool(a) or bool(b)
            elif a is None or b is None:
                waited = b if a is None else a
            else:
                waited = (a and b) or (a and bool(FIRST.search(cond)))
    return waited


def unwaited_exits(kernel: str, text: str):
    exits: list = []
    if walk(body_of(kernel, text)[1:-1], False, exits) is False:
        exits.append("end")
    return exits
