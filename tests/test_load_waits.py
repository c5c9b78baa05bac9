"""Wait states in front of the direct global-to-LDS loads, read from the
gfx950 code of the built library (no GPU). The kernels issue these loads as
inline assembly, where the compiler sees no load and adds no wait states, so
what the instruction set asks for has to be in the code itself:

  * a scalar write of M0 (the LDS address) and the load: 1 wait state;
  * a vector instruction that writes a scalar register of the base address
    (v_readlane, v_readfirstlane, v_cmp, carries) and the load: 5.

Every instruction between counts as one wait state, s_nop N as N + 1.
"""
import os
import re
import shutil
import subprocess

import pytest

import hashed_head_gram_amd as pg

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
M0_STATES, VALU_STATES = 1, 5


def scalars(op):
    """Scalar registers an operand names, as one set of names."""
    op = op.strip().split(" ")[0]
    if op == "vcc":
        return {"vcc_lo", "vcc_hi"}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", op)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {op} if re.fullmatch(r"s\d+|m0|vcc_lo|vcc_hi", op) else set()


def parse(text):
    """Functions of a disassembly, each a list of (op, operands, address, branch target)."""
    funcs, code, start = [], None, 0
    for line in text.splitlines():
        m = re.match(r"([0-9a-f]+) <(.+)>:", line)
        if m:
            start, code = int(m[1], 16), []
            funcs.append((m[2], code))
            continue
        m = re.match(r"\s+(\S+)\s*(.*?)\s*//\s*([0-9A-Fa-f]+):(.*)$", line)
        if m and code is not None:
            t = re.search(r"<[^>+]+(?:\+0x([0-9a-f]+))?>", m[4])
            ops = [x.strip() for x in m[2].split(",")]
            branch = "branch" in m[1] and t
            code.append((m[1], ops, int(m[3], 16),
                         start + int(t[1] or "0", 16) if branch else None))
    return funcs


def written(op, ops):
    """(scalar registers written, by a vector instruction?)"""
    if op.startswith("v_"):
        n = 2 if re.search(r"_co_|div_scale|mad_[ui]64", op) else 1    # a carry or flag too
        return set().union(*(scalars(x) for x in ops[:n])), True
    if op.startswith("s_") and not re.match(r"s_(cmp|bitcmp|waitcnt|nop|c?branch|barrier)", op):
        return scalars(ops[0]), False
    return set(), False


def missing(code):
    """Loads of one function that come too early, as (address, reason), and
    the number of its loads."""
    at = {c[2]: i for i, c in enumerate(code)}
    preds = [[] for _ in code]
    for i, (op, _, _, target) in enumerate(code):
        if i + 1 < len(code) and op not in ("s_branch", "s_endpgm"):
            preds[i + 1].append(i)
        if target is not None:
            preds[at[target]].append(i)
    bad, loads = [], 0
    for i, (op, ops, addr, _) in enumerate(code):
        if not op.startswith("global_load_lds"):
            continue
        loads += 1
        base = scalars(ops[1])
        assert base, (op, ops)
        todo, seen = [(p, 0) for p in preds[i]], {}
        while todo:
            j, states = todo.pop()
            if states >= VALU_STATES or seen.get(j, VALU_STATES) <= states:
                continue
            seen[j] = states
            out, vector = written(*code[j][:2])
            if not vector and "m0" in out and states < M0_STATES:
                bad.append((hex(addr), f"{code[j][0]} m0, {states} wait states"))
            if vector and out & (base | {"m0"}):
                bad.append((hex(addr), f"{code[j][0]} {code[j][1]}, {states} wait states"))
            states += int(code[j][1][0], 0) + 1 if code[j][0] == "s_nop" else 1
            todo += [(p, states) for p in preds[j]]
    return bad, loads


LISTING = """
0000000000001000 <k>:
\ts_mov_b32 m0, s4                                 // 000000001000: 00
{nop}\tglobal_load_lds_dwordx4 v1, s[2:3]           // 000000001008: 00
\tv_readlane_b32 s7, v2, 1                         // 000000001010: 00
\ts_cbranch_scc1 65533                             // 000000001018: 00 <k+0x20>
\ts_add_i32 m0, s4, s5                             // 00000000101C: 00
\ts_nop {n}                                        // 000000001020: 00
\tglobal_load_lds_dword v1, s[6:7]                 // 000000001024: 00
\ts_endpgm                                         // 000000001028: 00
"""


def test_checker():
    nop = "\ts_nop 0                                    // 000000001004: 00\n"
    (_, code), = parse(LISTING.format(nop=nop, n=3))
    assert missing(code) == ([], 2)
    (_, code), = parse(LISTING.format(nop="", n=3))
    assert [b[0] for b in missing(code)[0]] == ["0x1008"]
    (_, code), = parse(LISTING.format(nop=nop, n=2))     # 1 + 3 states by way of the branch
    assert [b[0] for b in missing(code)[0]] == ["0x1024"]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_every_load_waits(tmp_path):
    lib = shutil.copy(pg.LIB_PATH, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True,
                   cwd=tmp_path)
    loads, bad = 0, []
    for f in sorted(tmp_path.glob("lib.so.*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", str(f)], check=True, capture_output=True,
                              text=True).stdout
        for name, code in parse(text):
            b, n = missing(code)
            loads += n
            bad += [(name, *x) for x in b]
    assert loads > 100
    assert not bad, f"{len(bad)} of {loads} loads: {bad[:4]}"
