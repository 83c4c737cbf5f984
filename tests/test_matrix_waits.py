"""Waits between matrix instructions and the readers of their results, in the assembly of the built kernels.

The hardware does not hold back a vector instruction that reads a matrix instruction's result: the compiler
has to leave 8 issue slots between (for 16 x 16 x 32 in bf16; more in fp32).  Where a branch target lies between
the two, this compiler has left them out, and the first value read was wrong.  The kernels avoid that with
positions that advance without branches and with an explicit wait; this test follows every path from every
matrix instruction through the assembly."""
import os
import re
import subprocess

import pytest

from chunked_gated_delta_amd import build

SLOTS = 8
SOURCES = [s for s in build.sources() if s.endswith(".hip") and os.path.basename(s).startswith("gdr_")]


def registers(text):
    found = {int(n) for n in re.findall(r"(?<![\w\[])v(\d+)\b", text)}
    for lo, hi in re.findall(r"\bv\[(\d+):(\d+)\]", text):
        found |= set(range(int(lo), int(hi) + 1))
    return found


def split_dst(args):
    dst = re.match(r"\s*([^,]+),", args)
    return registers(dst[1]), args[dst.end():]


def functions(path):
    """(name, [(instruction, operands, line)], {label: index}) of every function in an assembly file."""
    name, code, labels = None, [], {}
    with open(path) as f:
        for n, line in enumerate(f, 1):
            line = line.split(";")[0].rstrip()
            label = re.match(r"^(\S+):", line)
            if label and label[1].startswith("_Z"):
                if name:
                    yield name, code, labels
                name, code, labels = label[1], [], {}
            elif label:
                labels[label[1]] = len(code)
            elif line.startswith("\t") and not line.startswith("\t."):
                op, _, args = line.strip().partition(" ")
                op, _, more = op.partition("\t")
                code.append((op, more + args, n))
    if name:
        yield name, code, labels


def early_reads(code, labels):
    """Readers of a matrix result fewer than SLOTS issue slots behind it, on any path."""
    for i, (op, args, line) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        todo, seen = [(i + 1, 0, split_dst(args)[0])], set()
        while todo:
            j, slots, live = todo.pop()
            while j < len(code) and slots < SLOTS and live and (j, slots) not in seen:
                seen.add((j, slots))
                o, a, at = code[j]
                j += 1
                if o == "s_endpgm":
                    break
                if o == "s_nop":
                    slots += int(a) + 1
                    continue
                if o.startswith(("s_branch", "s_cbranch")):
                    if a.strip() in labels:
                        todo.append((labels[a.strip()], slots + 1, live))
                    if o == "s_branch":
                        break
                elif o.startswith("v_mfma"):
                    dst, rest = split_dst(a)
                    if registers(",".join(rest.split(",")[:2])) & live:   # the addend may follow at once
                        yield line, at, slots, o
                        break
                    live = live - dst
                elif o.startswith(("v_", "ds_", "global_", "flat_", "scratch_", "buffer_")) and registers(a) & live:
                    yield line, at, slots, o
                    break
                slots += 1


def test_the_check_itself(tmp_path):
    """A read behind a branch target is found, one behind the wait is not."""
    text = "_Zk:\n\tv_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0\n\ts_cbranch_scc0 .L1\n\ts_nop 3\n.L1:\n\tv_add_f32_e32 v5, v0, v6\n\ts_endpgm\n"
    for wait, found in (("3", [1, 4 + 1]), ("11", [1])):
        f = tmp_path / "k.s"
        f.write_text(text.replace("s_nop 3", "s_nop " + wait))
        (name, code, labels), = functions(f)
        assert name == "_Zk" and sorted(s for _, _, s, _ in early_reads(code, labels)) == found


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("src", SOURCES, ids=os.path.basename)
def test_matrix_results_are_waited_for(src, tmp_path):
    out = str(tmp_path / "k.s")
    cmd = [build.HIPCC, *build.FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-S", "--offload-device-only", "-o", out, src]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels, matrix = 0, 0
    for name, code, labels in functions(out):
        kernels += 1
        matrix += sum(op.startswith("v_mfma") for op, _, _ in code)
        bad = list(early_reads(code, labels))
        assert not bad, f"{name}: (matrix instruction's line, reader's line, slots between, reader) {bad[:5]}"
    print(f"   {os.path.basename(src)}: {kernels} kernels, {matrix} matrix instructions", flush=True)
    assert kernels > 0
