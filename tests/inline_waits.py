"""Checks of the waits that instructions written inline need and that no compiler
inserts for them, over a disassembly of the built library (gfx950).

Each instruction is one wait state, s_nop N is N + 1.  The paths to an instruction
are followed backwards over branches, as far as the wait states reach:

  * a matrix instruction reads no register that a vector instruction other than one
    of its kind wrote less than 2 wait states before;
  * the registers of its result are touched by nothing else, other than matrix
    instructions that add to all of them, for 18 wait states;
  * a load into LDS takes its base from scalar registers that no vector instruction
    wrote less than 5 wait states before;
  * M0 is written for such a load alone, one wait state or more before it, and
    nothing between writes it again or reads it.
"""
import os
import re
import struct
import subprocess

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
READ_WAIT = 2
RESULT_WAIT = 18
BASE_WAIT = 5

_MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(path, wanted, directory):
    """The gfx950 code objects in the library at `path` that hold the bytes
    `wanted`, written to files below `directory`."""
    with open(path, "rb") as f:
        data = f.read()
    out = []
    at = data.find(_MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", data, at + len(_MAGIC))
        entry = at + len(_MAGIC) + 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, entry)
            target = data[entry + 24: entry + 24 + length].decode()
            entry += 24 + length
            code = data[at + offset: at + offset + size]
            if target.endswith("gfx950") and wanted in code:
                name = os.path.join(directory, "code%d.co" % len(out))
                with open(name, "wb") as f:
                    f.write(code)
                out.append(name)
        at = data.find(_MAGIC, at + 1)
    return out


def disassemble(code_object):
    return subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", code_object], check=True,
                          capture_output=True, text=True).stdout


def _registers(operand):
    """The registers that an operand names: a set of (file, number)."""
    found = set()
    for file, first, last in re.findall(r"\b([vas])\[(\d+):(\d+)\]", operand):
        found |= {(file, i) for i in range(int(first), int(last) + 1)}
    for file, one in re.findall(r"\b([vas])(\d+)\b", operand):
        found.add((file, int(one)))
    return found


class Instruction:
    def __init__(self, text, address):
        parts = text.split(None, 1)
        self.text = text
        self.address = address
        self.name = parts[0]
        self.operands = [o.strip() for o in re.split(r",(?![^\[]*\])", parts[1])] \
            if len(parts) > 1 else []
        self.target = None

    @property
    def states(self):
        return int(self.operands[0], 0) + 1 if self.name == "s_nop" else 1

    @property
    def matrix(self):
        return self.name.startswith("v_mfma")

    @property
    def vector(self):
        return self.name.startswith("v_") and not self.matrix

    def named(self):
        return set().union(*(_registers(o) for o in self.operands)) if self.operands else set()

    def written(self):
        """What a vector instruction writes: its first operand, and VCC, which is not
        among the registers looked for."""
        return _registers(self.operands[0]) if self.operands else set()


def functions(listing):
    """{name: its instructions} of a disassembly."""
    out, code = {}, None
    for line in listing.splitlines():
        head = re.match(r"[0-9a-f]+ <(.*)>:$", line)
        if head:
            code = out.setdefault(head.group(1), [])
            base, name = int(line.split()[0], 16), head.group(1)
            continue
        m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if code is None or m is None:
            continue
        i = Instruction(m.group(1), int(m.group(2), 16))
        t = re.search(r"<%s(?:\+0x([0-9a-f]+))?>\s*$" % re.escape(name), m.group(3))
        if t and ("branch" in i.name):
            i.target = base + int(t.group(1) or "0", 16)
        code.append(i)
    return out


def _before(code):
    """The instructions that may run right before each one."""
    at = {i.address: k for k, i in enumerate(code)}
    before = [[] for _ in code]
    for k, i in enumerate(code):
        if k + 1 < len(code) and i.name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
            before[k + 1].append(k)
        if i.target is not None:
            before[at[i.target]].append(k)
    return before


def _within(code, before, k, states):
    """The instructions with fewer than `states` wait states between them and k."""
    seen, work, out = {}, [(k, 0)], []
    while work:
        j, passed = work.pop()
        for b in before[j]:
            if passed < states and seen.get(b, states) > passed:
                if b not in seen:
                    out.append(b)
                seen[b] = passed
                work.append((b, passed + code[b].states))
    return out


def faults(code):
    """What the instructions of a function do too early, as texts."""
    before = _before(code)
    out = []

    def say(k, b, what):
        out.append("%x %s: %s (%x %s)" % (code[k].address, code[k].text, what, code[b].address,
                                          code[b].text))

    for k, i in enumerate(code):
        if i.matrix:
            reads = set().union(*(_registers(o) for o in i.operands[1:4]))
            for b in _within(code, before, k, READ_WAIT):
                if code[b].vector and code[b].written() & reads:
                    say(k, b, "an operand was just written")
        named = i.named()
        if named:
            for b in _within(code, before, k, RESULT_WAIT):
                if code[b].matrix and _registers(code[b].operands[0]) & named:
                    result = _registers(code[b].operands[0])
                    adds = i.matrix and _registers(i.operands[0]) == result and \
                        _registers(i.operands[3]) == result and \
                        not result & (_registers(i.operands[1]) | _registers(i.operands[2]))
                    if not adds:
                        say(k, b, "a matrix result is touched")
        if "_load_lds_" in i.name:
            base = _registers(i.operands[1])
            for b in _within(code, before, k, BASE_WAIT):
                if code[b].name.startswith("v_") and code[b].written() & base:
                    say(k, b, "the base was just written")
            if not (k >= 2 and before[k] == [k - 1] and before[k - 1] == [k - 2] and
                    code[k - 1].name == "s_nop" and code[k - 2].name == "s_mov_b32" and
                    code[k - 2].operands[0] == "m0"):
                say(k, max(k - 1, 0), "M0 is not set right before")
        if "m0" in i.text and not (i.name == "s_mov_b32" and i.operands[0] == "m0" and
                                   k + 2 < len(code) and "_load_lds_" in code[k + 2].name):
            say(k, k, "M0 for something else")
    return out
