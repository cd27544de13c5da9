"""The CTA size of dt_kv_append for every head count, compiled for the host with checked arithmetic (no GPU needed)."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_tree_top_gb300", "csrc")
CODE = """
#include "append_shape.cuh"
#include <cstdio>
#include <initializer_list>
int main() {
  for (int items : {4, 8})
    for (int heads = 2; heads <= 768; ++heads) {
      const int threads = dt::append_threads(heads, items);
      std::printf("%d %d %d\\n", items, heads, threads);
    }
}
"""


def test_append_cta_sizes(tmp_path):
    src, exe = tmp_path / "shape.cpp", tmp_path / "shape"
    src.write_text(CODE)
    r = subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", f"-I{CSRC}", str(src),
                        "-o", str(exe)], capture_output=True, text=True)
    if "cannot find" in r.stderr and "ubsan" in r.stderr:
        pytest.skip("no undefined-behaviour runtime here")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    for line in r.stdout.splitlines():
        items, heads, threads = map(int, line.split())
        idle = {n: -(-heads // (n // items)) * (n // items) - heads for n in range(64, 257, 32)}
        least = min(idle[n] / n for n in idle)
        assert threads in idle and idle[threads] / threads == least, (items, heads, threads)
        assert all(idle[n] / n > least for n in idle if n > threads)  # the largest of the best
