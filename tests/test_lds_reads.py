"""No instruction of the built kernels touches a register that an LDS read in flight will still write.

The grouped GEMMs read their fragments by inline assembly and wait for them by hand, a few fragments later.
The compiler takes such a register as written at once: a spill, copy or reuse that it placed before the wait
would use a stale value, or lose the read's, and no numerical test has to show it.  So the machine code that was built is
checked: LDS operations return in order, so `s_waitcnt lgkmcnt(N)` leaves at most the last N in flight, and until
a wait has covered a read nothing may name its destination.
"""

import os
import re
import shutil
import subprocess

import pytest

from expert_ffn_layer_top_amd import build

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
LINE = re.compile(r"^\s+([a-z]\w+)(.*?)\s*// ([0-9A-F]+): ")
REG = re.compile(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])")
TARGET = re.compile(r"<(.+?)(?:\+0x([0-9a-f]+))?>\s*$")


def regs(text):
    out = set()
    for kind, one, lo, hi in REG.findall(text):
        out.update((kind, i) for i in (range(int(lo), int(hi) + 1) if lo else [int(one)]))
    return out


def functions(listing):
    """{name: [(address, mnemonic, operands, branch target or None)]} of a disassembly."""
    out, name, start = {}, None, {}
    for line in listing.splitlines():
        head = re.match(r"^([0-9a-f]{8,}) <(.+)>:$", line)
        if head:
            name = head.group(2)
            start[name] = int(head.group(1), 16)
            out[name] = []
            continue
        m = LINE.match(line)
        if m and name:
            target = None
            if "branch" in m.group(1):
                t = TARGET.search(line)
                target = start[t.group(1)] + int(t.group(2) or "0", 16)
            out[name].append((int(m.group(3), 16), m.group(1), m.group(2), target))
    return out


def merge(a, b):
    """Both paths' reads in flight, aligned at the newest."""
    if a is None or a == b:
        return b
    n = max(len(a), len(b))
    pad = lambda s: ((frozenset(),) * (n - len(s))) + s   # noqa: E731
    return tuple(x | y for x, y in zip(pad(a), pad(b)))


def step(state, op, args):
    """(registers in flight that the instruction names, the reads in flight after it)."""
    named = regs(args)
    bad = named & frozenset().union(*state) if state else frozenset()
    if op == "s_waitcnt":
        n = re.search(r"lgkmcnt\((\d+)\)", args)
        if n:
            state = state[len(state) - int(n.group(1)):] if int(n.group(1)) < len(state) else state
            state = () if n.group(1) == "0" else state
    elif op.startswith("ds_"):
        returns = not op.startswith("ds_write") and ("read" in op or "permute" in op or "swizzle" in op or "_rtn" in op)
        dest = regs(args.split(",")[0]) if returns else ()
        state = (*state, frozenset(dest))[-64:]
    return bad, state


def hazards(code):
    """[(address, instruction)] of one function's instructions that name a register in flight."""
    at = {a: i for i, (a, _, _, _) in enumerate(code)}
    entry = {0: ()}
    work, found = [0], {}
    while work:
        i = work.pop()
        state = entry[i]
        while True:
            a, op, args, target = code[i]
            bad, state = step(state, op, args)
            if bad:
                found[a] = f"{op}{args}"
            nexts = [] if op in ("s_branch", "s_endpgm") or op.startswith("s_setpc") else [i + 1]
            if target is not None:
                nexts.append(at[target])
            follow = None
            for j in nexts:
                if j >= len(code):
                    continue
                if j == i + 1 and target is None and j not in entry:
                    entry[j] = state
                    follow = j
                else:
                    new = merge(entry.get(j), state)
                    if j not in entry or new != entry[j]:
                        entry[j] = new
                        work.append(j)
            if follow is None:
                break
            i = follow
    return sorted(found.items())


def listing(*lines):
    body = "\n".join(f"\t{l}  // {8 * i:012X}: 00000000{' <f+0x0>' if 'cbranch' in l else ''}" for i, l in enumerate(lines))
    return functions(f"0000000000000000 <f>:\n{body}\n")["f"]


def test_the_check_itself():
    read, use = "ds_read_b128 v[0:3], v9 offset:16", "v_mov_b32_e32 v8, v2"
    assert hazards(listing(read, use, "s_endpgm"))
    assert not hazards(listing(read, "s_waitcnt lgkmcnt(0)", use, "s_endpgm"))
    assert not hazards(listing(read, "ds_read_b32 v4, v9", "s_waitcnt lgkmcnt(1)", use, "s_endpgm"))
    assert hazards(listing(read, "ds_read_b32 v4, v9", "s_waitcnt lgkmcnt(1)", "v_mov_b32_e32 v4, 0", "s_endpgm"))
    assert hazards(listing(read, "s_waitcnt vmcnt(0)", "scratch_store_dword off, v3, off offset:4", "s_endpgm"))
    # a read before a branch is in flight at its target, also backwards
    assert hazards(listing(use, read, "s_cbranch_scc1 65533", "s_endpgm"))
    assert not hazards(listing(use, read, "s_waitcnt lgkmcnt(0)", "s_cbranch_scc1 65533", "s_endpgm"))


def test_no_instruction_touches_a_read_in_flight(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no llvm-objdump")
    assert os.path.exists(build.LIB), "the library is not built"
    shutil.copy(build.LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    objects = [p for p in tmp_path.iterdir() if p.name.endswith(build.ARCH)]
    checked, found = 0, []
    for p in objects:
        text = subprocess.run([OBJDUMP, "-d", p], check=True, capture_output=True, text=True).stdout
        for name, code in functions(text).items():
            if code:
                checked += 1
                found += [(name, hex(a), i) for a, i in hazards(code)]
    assert checked > 60 and not found, found[:10]
