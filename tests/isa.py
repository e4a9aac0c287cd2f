"""Disassembly of the built library's gfx950 code and the checks of it that
tests/test_isa_cpu.py makes: what the hardware wants between two instructions
where one of them stands in inline assembly, into which the compiler's hazard
recogniser does not look.

A listing is a list of kernels (name, [(address, mnemonic, operands)]).
"""
import os
import re
import subprocess

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def disassemble(lib, workdir):
    """The listings of a library's device code objects."""
    copy = os.path.join(workdir, os.path.basename(lib))
    os.symlink(lib, copy)
    subprocess.run([OBJDUMP, "--offloading", copy], check=True, capture_output=True, cwd=workdir)
    text = ""
    for name in sorted(os.listdir(workdir)):
        if name.endswith("gfx950"):
            text += subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", os.path.join(workdir, name)], check=True,
                                   capture_output=True, text=True).stdout
    return parse(text)


def parse(text):
    kernels = []
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(.*)>:$", line)
        if head:
            kernels.append((head.group(1), []))
            continue
        m = re.match(r"\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):", line)
        if m and kernels:
            kernels[-1][1].append((int(m.group(3), 16), m.group(1), m.group(2)))
    return kernels


def _scalars(text):
    """Scalar registers that an operand text names."""
    out = set()
    for m in re.finditer(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b", text):
        out |= {int(m.group(3))} if m.group(3) else set(range(int(m.group(1)), int(m.group(2)) + 1))
    return out | {r for r in ("m0", "vcc") if re.search(rf"\b{r}\b", text)}


def _vector_scalar_results(ins):
    """Scalar registers that a vector instruction writes."""
    _, name, text = ins
    ops = text.split(",")
    if re.match(r"v_(readfirstlane|readlane|cmp)", name):
        return _scalars(ops[0])
    if re.match(r"v_(add|sub|subrev|addc|subb|subbrev)_co_|v_div_scale|v_mad_[ui]64", name) and len(ops) > 1:
        return _scalars(ops[1])
    return set()


def _predecessors(code):
    at = {a: k for k, (a, _, _) in enumerate(code)}
    pred = [[] for _ in code]
    for k, (a, name, text) in enumerate(code):
        if k + 1 < len(code) and name not in ("s_branch", "s_endpgm"):
            pred[k + 1].append(k)
        if name == "s_branch" or name.startswith("s_cbranch"):
            offset = int(text.split()[0])
            target = a + 4 + 4 * (offset - 65536 if offset >= 32768 else offset)
            if target in at:
                pred[at[target]].append(k)
    return pred


def hazards(code):
    """(kind, producer, consumer) of a vector-memory instruction that follows a write of a scalar
    register it reads too closely, over every path: a scalar write of M0 before a copy to LDS wants one
    wait state between them, a vector instruction's write of a scalar register before any access that
    reads it five.  An instruction is one wait state, s_nop n is n + 1."""
    pred, found = _predecessors(code), []
    for k, ins in enumerate(code):
        if not re.match(r"(global|buffer|flat|scratch)_", ins[1]):
            continue
        to_lds, reads = "lds" in ins[1] or "lds" in ins[2], _scalars(ins[2])
        todo, seen = [(p, 0) for p in pred[k]], set()
        while todo:
            p, waited = todo.pop()
            if (p, waited) in seen:
                continue
            seen.add((p, waited))
            other = code[p]
            if to_lds and waited < 1 and other[1].startswith("s_") and re.match(r"m0\b", other[2]):
                found.append(("M0", other, ins))
            if _vector_scalar_results(other) & reads:
                found.append(("vector write", other, ins))
            waited += int(other[2], 0) + 1 if other[1] == "s_nop" else 1
            if waited < 5:
                todo += [(q, waited) for q in pred[p]]
    return found


def lds_outstanding_at_barriers(code):
    """Barriers (addresses) in front of which, on some path, an LDS operation of the wave may still be
    outstanding: behind the barrier another wave may overwrite what it reads."""
    pred = _predecessors(code)
    follow = [[] for _ in code]
    for k, ps in enumerate(pred):
        for p in ps:
            follow[p].append(k)
    most, todo = [0] * len(code), list(range(len(code)))
    while todo:
        k = todo.pop()
        n = max((most[p] for p in pred[k]), default=0)
        if code[k][1].startswith("ds_"):
            n = min(n + 1, 16)   # the counter has four bits
        wait = re.search(r"lgkmcnt\((\d+)\)", code[k][2]) if code[k][1] == "s_waitcnt" else None
        if wait:
            n = min(n, int(wait.group(1)))
        if n != most[k]:
            most[k] = n
            todo += follow[k]
    return [i[0] for i, n in zip(code, most) if i[1] == "s_barrier" and n]
