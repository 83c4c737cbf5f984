"""The waits between matrix instructions and the readers of their results, in the assembly of the built kernels of linear
attention with a decay for each head: 8 issue slots behind a 16 x 16 x 32 product in bf16, 10 behind a 16 x 16 x 4
one in fp32, on every path."""
import os
import subprocess

import pytest

import test_matrix_waits as waits
import test_matrix_waits_each as each
from chunked_gated_delta_amd import build

SOURCES = [s for s in build.sources() if s.endswith(".hip") and os.path.basename(s).startswith("lad_")]


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("src", SOURCES, ids=os.path.basename)
def test_matrix_results_are_waited_for(src, tmp_path, monkeypatch):
    out = str(tmp_path / "k.s")
    cmd = [build.HIPCC, *build.FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-S", "--offload-device-only", "-o", out, src]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    kernels = 0
    for name, code, labels in waits.functions(out):
        kernels += 1
        bad = each.early_reads(code, labels, monkeypatch)
        assert not bad, f"{name}: (matrix instruction's line, reader's line, slots between, reader) {bad[:5]}"
    assert kernels > 0
