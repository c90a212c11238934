"""The int8 kernels' roundings do not hang on the compiler's choice of what to fuse (no GPU): their
gfx950 assembly is the same whether it may contract products into sums or not, since every fused
operation of theirs is written as one.  Routes give the same bits only so."""
import os
import subprocess

import pytest

from test_wait_counts_cpu import CSRC, ROOT, _hipcc


@pytest.mark.parametrize("src", ["few_i8.hip", "gemm_i8.hip", "quant_i8.hip"])
def test_contraction_changes_nothing(src, tmp_path):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    runs = []
    for mode in ("fast-honor-pragmas", "off"):
        out = tmp_path / (mode + ".s")
        runs.append((out, subprocess.Popen(
            [hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-ffp-contract=" + mode, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "--cuda-device-only", "-S",
             "-o", str(out), os.path.join(CSRC, src)], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL)))
    text = []
    for out, p in runs:
        assert p.wait(timeout=600) == 0
        text.append([ln for ln in out.read_text().splitlines() if "__hip_cuid_" not in ln])   # differs per compilation
    assert any("v_fma" in ln for ln in text[0])
    differing = sum(a != b for a, b in zip(*text)) + abs(len(text[0]) - len(text[1]))
    assert differing == 0, f"{src}: {differing} lines depend on contraction"
