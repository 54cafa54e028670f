"""Loads in flight when a kernel of the window and cache attention ends: the
drain of its ring on the CPU (tests/host/ring_drain_check.cu), and that every
loading kernel drains whatever became of its waits."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_long_sequence_attn_b200", "csrc")
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


@pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not available")
def test_drain_ring():
    out_dir = os.path.join(ROOT, "_build")
    os.makedirs(out_dir, exist_ok=True)
    exe = os.path.join(out_dir, "ring_drain_check")
    subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-I", os.path.join(ROOT, "include"),
                    "-I", CSRC, "--expt-relaxed-constexpr", "-o", exe,
                    os.path.join(ROOT, "tests", "host", "ring_drain_check.cu")], check=True, capture_output=True, timeout=600)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0 and "fails=0" in res.stdout, res.stdout[-2000:]


@pytest.mark.parametrize("name,others", [("decode.cu", []), ("window_tc.cu", ["bar_q", "bar_tail"]), ("weights_tc.cu", ["bar_k"]),
                                         ("window_bwd_tc.cu", ["bar_tile"])])
def test_every_loader_drains(name, others):
    text = open(os.path.join(CSRC, name)).read()
    at = text.index("// drain: every issued load has landed before the CTA may exit")
    drain = text[at:text.index("drain_loads(", at) + 80].split("drain_loads(")
    assert len(drain) == 2 and not re.search(r"\bok\b", drain[0]), "the drain depends on the waits before it"
    for bar in others:  # loads on barriers of their own
        assert f"mbar_wait({bar}, 0" in drain[0], bar
