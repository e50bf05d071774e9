"""CPU check of the built kernels' LDS ordering.  A raw s_barrier does not wait
for the LDS writes of the waves that reach it: what a wave writes for others
to read has to be waited for (s_waitcnt lgkmcnt(0)) before the barrier.  The
compiler does so for __syncthreads(), not for a barrier of the kernel's own.
Every path through every kernel is followed in the assembly of the library
built here."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "sparse_linear_layers_absmean_amd", "libsbl.so")
OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")) if p and os.path.exists(p)),
               None)

WRITES = ("ds_write", "ds_add", "ds_sub", "ds_inc", "ds_dec", "ds_min", "ds_max", "ds_and", "ds_or", "ds_xor", "ds_cmpst",
          "ds_wrxchg")
CLEAN, DIRTY = 1, 2


def functions(text):
    """(name, [(address, instruction, the rest of its line)]) of a disassembly."""
    name, body = None, []
    for line in text.splitlines():
        head = re.match(r"([0-9a-f]+) <(\S+)>:", line)
        if head:
            if name:
                yield name, body
            name, body = head.group(2), []
            continue
        m = re.match(r"\s+(\S.*?)\s*// ([0-9A-F]+):(.*)", line)
        if m and name:
            body.append((int(m.group(2), 16), m.group(1), m.group(3)))
    if name:
        yield name, body


def open_barriers(body):
    """Addresses of the barriers that some path reaches with an LDS write not waited for."""
    at = {a: i for i, (a, _, _) in enumerate(body)}
    seen, bad, todo = [0] * len(body), set(), [(0, CLEAN)]
    while todo:
        i, state = todo.pop()
        if i >= len(body) or seen[i] & state:
            continue
        seen[i] |= state
        address, text, rest = body[i]
        op = text.split()[0]
        if op.startswith(WRITES):
            state = DIRTY
        elif op == "s_waitcnt" and ("lgkmcnt(0)" in text or text.split()[1:] == ["0"]):
            state = CLEAN
        elif op == "s_barrier" and state == DIRTY:
            bad.add(address)
        if op == "s_endpgm":
            continue
        if op == "s_branch" or op.startswith("s_cbranch"):
            to = re.search(r"<[^>+]+(?:\+0x([0-9a-f]+))?>", rest)
            todo.append((at[body[0][0] + int(to.group(1) or "0", 16)], state))
            if op == "s_branch":
                continue
        todo.append((i + 1, state))
    return bad


def _listing(*code):
    lines = ["0000000000001000 <k>:"]
    for n, c in enumerate(code):
        lines.append(f"\t{c.split('@')[0]:40s}// {0x1000 + 4 * n:012X}: 00000000" + (f" <k+0x{4 * int(c.split('@')[1]):x}>"
                                                                             if "@" in c else ""))
    (_, body), = functions("\n".join(lines))
    return body


@pytest.mark.parametrize("code,bad", [
    (("ds_write_b32 v0, v1", "s_waitcnt lgkmcnt(0)", "s_barrier", "s_endpgm"), []),
    (("ds_write_b32 v0, v1", "s_waitcnt vmcnt(0)", "s_barrier", "s_endpgm"), [0x1008]),
    # around the wait on one path
    (("ds_write_b32 v0, v1", "s_cbranch_vccz 3 @3", "s_waitcnt vmcnt(0) lgkmcnt(0)", "s_barrier", "s_endpgm"), [0x100c]),
    # the second turn of a loop
    (("s_barrier", "ds_add_u32 v0, v1", "s_cbranch_scc1 0 @0", "s_endpgm"), [0x1000]),
    (("ds_read_b32 v0, v1", "s_barrier", "s_endpgm"), []),
])
def test_the_check_itself(code, bad):
    assert sorted(open_barriers(_listing(*code))) == bad


@pytest.mark.skipif(OBJDUMP is None, reason="llvm-objdump (part of ROCm) is not here")
def test_lds_writes_are_done_before_every_barrier(tmp_path):
    if not os.path.exists(LIB):
        pytest.fail("libsbl.so is not built (run __graft_entry__.build())")
    shutil.copy(LIB, tmp_path / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", "lib.so"], cwd=tmp_path, check=True, capture_output=True)
    kernels, barriers, bad = 0, 0, {}
    for obj in sorted(tmp_path.glob("lib.so.*gfx950*")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(obj)], check=True, capture_output=True,
                              text=True).stdout
        for name, body in functions(text):
            kernels += 1
            barriers += sum(op.startswith("s_barrier") for _, op, _ in body)
            found = open_barriers(body)
            if found:
                bad[name] = [hex(a) for a in sorted(found)]
    assert kernels > 50 and barriers > 100         # the library was read
    assert not bad, bad
