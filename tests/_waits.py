"""Reads the gfx950 instructions of this library's own kernels for one thing: that a barrier behind which waves read LDS
that others had loaded straight into (buffer_load ... lds) is met only when those loads have arrived.

Vector memory operations of a wave end in order and s_waitcnt vmcnt(n) waits until n are under way, so a wait that is
right in the source is wrong in the binary if the compiler dropped one of the loads that it counts.  `outstanding`
follows every path back from a barrier."""
import glob
import os
import re
import shutil
import subprocess

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MEMORY = re.compile(r"(buffer|global|flat|scratch)_(load|store|atomic)")
MOST = 64  # operations under way that vmcnt can count


def disassemble(lib, folder):
    """{kernel: lines} of the library's gfx950 code."""
    so = os.path.join(folder, "lib.so")
    shutil.copy(lib, so)
    subprocess.run([OBJDUMP, "--offloading", so], check=True, capture_output=True)
    kernels = {}
    for obj in sorted(glob.glob(so + ".*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", obj], check=True, capture_output=True,
                              text=True).stdout
        lines = None
        for line in text.splitlines():
            m = re.match(r"[0-9a-f]+ <(.+)>:$", line)
            if m and not re.match(r"L\d+$", m.group(1)):
                lines = kernels.setdefault(m.group(1), [])
            elif lines is not None:
                lines.append(line)
    return kernels


def parse(lines):
    """(instructions, the places from which each is reached)."""
    ins, labels = [], {}
    for line in lines:
        m = re.match(r"(?:[0-9a-f]+ )?<(L\d+)>:", line)
        line = line.split("//")[0].strip()
        if m:
            labels[m.group(1)] = len(ins)
        elif line:
            ins.append(line)
    before = [[] for _ in ins]
    for k, t in enumerate(ins):
        op = t.split()[0]
        if op.startswith(("s_branch", "s_cbranch")):
            before[labels[t.split()[1]]].append(k)
        if op not in ("s_branch", "s_endpgm") and k + 1 < len(ins):
            before[k + 1].append(k)
    return ins, before


def into_lds(t):
    return t.startswith("buffer_load") and t.endswith(" lds")


def stage_behind(ins, b):
    """Loads into LDS that are issued behind barrier b, before the next barrier or branch."""
    n = 0
    for t in ins[b + 1:]:
        if t.startswith(("s_barrier", "s_branch", "s_cbranch", "s_endpgm")):
            break
        n += into_lds(t)
    return n


def outstanding(ins, before, b, newest):
    """How many operations may be under way at barrier b since a load into LDS older than the `newest` last ones, that
    one with them: 0 if all such loads have arrived, on every path."""
    worst, seen, todo = 0, set(), [(k, 0, MOST) for k in before[b]]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        k, passed, left = at  # of what was issued up to here, the last `left` operations may be under way
        t = ins[k]
        if t.startswith("s_waitcnt"):
            m = re.search(r"vmcnt\((\d+)\)", t)
            left = min(left, int(m.group(1))) if m else left
        elif MEMORY.match(t) and left:
            if into_lds(t) and passed == newest:
                worst = max(worst, left)
                continue
            passed += into_lds(t)
            left -= 1
        if left:
            todo += [(p, passed, left) for p in before[k]]
    return worst
