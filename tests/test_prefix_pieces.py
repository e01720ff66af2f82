"""How a unit of the prefix pass is cut, compiled by itself for the host."""
import os
import shutil
import subprocess

import pytest

from test_attention_source import CSRC, body

STANDS = """
#include <cstdint>
#include <cstdio>
struct Walk {
  struct { int count; } en;
  int x = 0, tile, n, at;
  int& piece() { return at; }
  void take_piece(int each) {%s}
};
int main() {
  for (int count : {1, 2, 7, 235, 1 << 20, (1 << 24) - 1, 1 << 24})
    for (int each : {1, 2, 3, 32, 159, 160}) {
      if (each > count) continue;
      Walk w;
      w.en.count = count;
      int64_t next = 0, least = count, most = 0;
      bool good = true;
      for (w.at = 0; w.at < each; ++w.at) {
        w.take_piece(each);
        good &= w.tile == next && w.n > 0;
        next += w.n;
        least = w.n < least ? w.n : least;
        most = w.n > most ? w.n : most;
      }
      std::printf("%%d %%d %%d\\n", count, each, good && next == count && most - least <= 1);
    }
}
"""


def test_pieces_cover_a_unit_evenly(tmp_path):
    """Up to 160 pieces of 2^24 key tiles, which are 2^31 tokens."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    with open(os.path.join(CSRC, "prefill_attention.cu")) as f:
        src = body(f.read(), "void take_piece(int each)")
    (tmp_path / "pieces.cpp").write_text("#include <initializer_list>\n" + STANDS % src)
    exe = tmp_path / "pieces"
    subprocess.run([cxx, "-std=c++17", "-fwrapv", str(tmp_path / "pieces.cpp"), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    assert len(lines) == 30 and all(line.endswith(" 1") for line in lines), [line for line in lines if not line.endswith(" 1")]
