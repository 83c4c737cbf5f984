"""The wait behind each kind of matrix instruction, in the assembly of the built kernels: a 16 x 16 x 32 product
in bf16 needs 8 issue slots before a reader of its result, a 16 x 16 x 4 one in fp32 needs 10.  Instructions of
another kind are not known to this test and fail it, so that their wait is looked up when they come in."""
import os
import subprocess

import pytest

import test_matrix_waits as waits
from chunked_gated_delta_amd import build

SLOTS = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}


def kind(op):
    """The instruction without its encoding's suffix."""
    for end in ("_e64", "_vop3p"):
        op = op.removesuffix(end)
    return op


def early_reads(code, labels, monkeypatch):
    """(instruction's line, reader's line, slots, reader) of every reader too early for the instruction it reads."""
    at = {line: kind(op) for op, _, line in code if op.startswith(("v_mfma", "v_smfma"))}
    unknown = set(at.values()) - set(SLOTS)
    assert not unknown, f"no wait is known for {unknown}"
    found = []
    for op, slots in SLOTS.items():
        monkeypatch.setattr(waits, "SLOTS", slots)
        found += [r for r in waits.early_reads(code, labels) if at[r[0]] == op]
    return found


def listing(tmp_path, op, nops):
    f = tmp_path / "k.s"
    f.write_text(f"_Zk:\n\t{op} v[0:3], v[8:11], v[12:15], 0\n\ts_nop {nops - 1}\n\tv_add_f32_e32 v5, v0, v6\n\ts_endpgm\n")
    (_, code, labels), = waits.functions(f)
    return code, labels


@pytest.mark.parametrize("op,slots,early", [("v_mfma_f32_16x16x32_bf16", 7, True), ("v_mfma_f32_16x16x32_bf16", 8, False), ("v_mfma_f32_16x16x4_f32", 7, True),
                                            ("v_mfma_f32_16x16x4_f32", 8, True), ("v_mfma_f32_16x16x4_f32", 9, True), ("v_mfma_f32_16x16x4_f32", 10, False)])
def test_the_check_itself(tmp_path, monkeypatch, op, slots, early):
    assert [r[2] for r in early_reads(*listing(tmp_path, op, slots), monkeypatch)] == ([slots] if early else [])


def test_unknown_instructions_are_named(tmp_path, monkeypatch):
    with pytest.raises(AssertionError, match="v_mfma_f32_32x32x2_f32"):
        early_reads(*listing(tmp_path, "v_mfma_f32_32x32x2_f32", 16), monkeypatch)


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("src", waits.SOURCES, ids=os.path.basename)
def test_each_matrix_result_is_waited_for(src, tmp_path, monkeypatch):
    out = str(tmp_path / "k.s")
    cmd = [build.HIPCC, *build.FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-S", "--offload-device-only", "-o", out, src]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    count = dict.fromkeys(SLOTS, 0)
    for name, code, labels in waits.functions(out):
        bad = early_reads(code, labels, monkeypatch)
        assert not bad, f"{name}: (matrix instruction's line, reader's line, slots between, reader) {bad[:5]}"
        for op, _, _ in code:
            if kind(op) in count:
                count[kind(op)] += 1
    print(f"   {os.path.basename(src)}: {count}", flush=True)
