"""Looks an assembly listing over for matrix instructions that the compiler does
not know as such (they come from inline assembly): the wait states that it
would put around its own have to be there all the same.

* A result may be read or overwritten 12 wait states after its instruction was
  issued: v_mfma_scale_f32_16x16x128_f8f6f4 takes 4 passes with FP4 operands and
  8 in its longest form, and a result is out 4 wait states after the last pass.
* A register that a vector instruction has written may be read 2 wait states
  later.
Every instruction is one wait state, ``s_nop N`` is N + 1.
"""
from __future__ import annotations

import re

RESULT_WAIT = 12
SOURCE_WAIT = 2

_REG = re.compile(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def _regs(text: str) -> set[str]:
    out = set()
    for kind, lo, hi, one in _REG.findall(text):
        out.update("%s%d" % (kind, i) for i in (range(int(lo), int(hi) + 1) if lo else (int(one),)))
    return out


def _functions(text: str) -> dict[str, list[tuple[str, str, bool]]]:
    """Name -> lines of code: ("label", name, False), or (mnemonic, operands,
    whether the line comes from inline assembly)."""
    funcs, lines, inline = {}, None, False
    for raw in text.splitlines():
        if "ASMSTART" in raw or "ASMEND" in raw:
            inline = "ASMSTART" in raw
        line = raw.split(";")[0].split("//")[0].strip()
        m = re.match(r"^([\w.$]+):$", line)
        if m and m.group(1).startswith("_Z"):
            lines = funcs.setdefault(m.group(1), [])
        elif m and lines is not None:
            if m.group(1).startswith(".Lfunc_end"):
                lines = None
            else:
                lines.append(("label", m.group(1), False))
        elif line and lines is not None and not line.startswith("."):
            op, _, rest = line.partition(" ") if " " in line else line.partition("\t")
            lines.append((op.strip(), rest.strip(), inline))
    return funcs


def _blocks(lines):
    """Basic blocks: lists of instructions, and each one's successors."""
    blocks, labels, cur = [[]], {}, 0
    for op, rest, inline in lines:
        if op == "label":
            if blocks[cur]:
                blocks.append([])
                cur += 1
            labels[rest] = cur
            continue
        blocks[cur].append((op, rest, inline))
        if op.startswith(("s_cbranch", "s_branch", "s_endpgm")):
            blocks.append([])
            cur += 1
    succ = []
    for i, b in enumerate(blocks):
        last = b[-1] if b else ("", "", False)
        to = [labels[last[1]]] if last[0].startswith(("s_cbranch", "s_branch")) else []
        if not last[0].startswith(("s_branch", "s_endpgm")) and i + 1 < len(blocks):
            to.append(i + 1)
        succ.append(to)
    return blocks, succ


def _walk(block, results, written, found=None):
    """Ages of the registers that matter, in wait states, through a block."""
    results, written = dict(results), dict(written)
    for op, rest, inline in block:
        mfma = inline and op.startswith("v_mfma")
        used = _regs(rest)
        if found is not None:
            if mfma:
                first = _regs(rest.split(",")[0])
                late = [r for r in used if written.get(r, SOURCE_WAIT) < SOURCE_WAIT]
                # (a result that the same kind of instruction adds to is the hardware's own affair)
                late += [r for r in used - first if results.get(r, RESULT_WAIT) < RESULT_WAIT]
            else:
                late = [r for r in used if results.get(r, RESULT_WAIT) < RESULT_WAIT]
            if late:
                found.append("%s %s: %s" % (op, rest, " ".join(sorted(late))))
        step = int(rest, 0) + 1 if op == "s_nop" else 1
        results = {r: a + step for r, a in results.items() if a + step < RESULT_WAIT}
        written = {r: a + step for r, a in written.items() if a + step < SOURCE_WAIT}
        if op.startswith("v_") and rest:
            first = _regs(rest.split(",")[0])
            (results if mfma else written).update(dict.fromkeys(first, 0))
    return results, written


def _merge(a, b):
    out = dict(a)
    for r, v in b.items():
        out[r] = min(v, out.get(r, v))
    return out


def check(text: str) -> dict[str, tuple[int, list[str]]]:
    """Function -> its inline matrix instructions, and what comes too early, for
    every function of the listing that has any."""
    report = {}
    for name, lines in _functions(text).items():
        count = sum(inline and op.startswith("v_mfma") for op, _, inline in lines)
        if not count:
            continue
        blocks, succ = _blocks(lines)
        entry = [({}, {}) for _ in blocks]
        todo = list(range(len(blocks)))
        while todo:
            i = todo.pop()
            out = _walk(blocks[i], *entry[i])
            for j in succ[i]:
                new = (_merge(entry[j][0], out[0]), _merge(entry[j][1], out[1]))
                if new != entry[j]:
                    entry[j] = new
                    todo.append(j)
        found = []
        for b, e in zip(blocks, entry):
            _walk(b, *e, found)
        report[name] = (count, found)
    return report
