"""What the paged indexer leaves when a wait gives up, on the host: a program compiled from the kernel's
own header (no GPU is used: no wait is made to give up on one)."""

import os
import subprocess

from deepseek_sparse_attention_ragged_gb300 import _build as build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_key_is_scored_or_minus_infinity(tmp_path):
    exe = tmp_path / "unscored"
    subprocess.run([build.nvcc(), "-std=c++17", "-O2", "-I", build.CSRC, os.path.join(ROOT, "tests", "c", "unscored.cu"),
                    "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "every key once" in r.stdout, r.stdout + r.stderr


def test_the_epilogue_leaves_no_key_unwritten():
    """The kernel's only way out of its scoring loop before the last tile goes through that function."""
    text = open(os.path.join(build.CSRC, "paged_indexer.cu")).read()
    loop = text[text.index("// ---- epilogue"):text.index("// ---- widening")]
    assert loop.count("break;") == 1 and "return" not in loop and "continue" not in loop
    before = loop[:loop.index("break;")].rstrip().splitlines()[-1]
    assert before.strip().startswith("unscored(out, it, mine, kEpiSets, j, kEpiSets * step * kTileKeys, kv_len);")
