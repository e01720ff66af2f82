"""The count of a device's SMs, compiled by itself against a stand-in for the runtime."""
import os
import shutil
import subprocess

import pytest

from test_attention_source import CSRC, body

STANDS = """
#include <atomic>
#include <cstdio>
#include <initializer_list>
enum { cudaSuccess = 0, cudaDevAttrMultiProcessorCount = 16 };
static int device = 0, asked = 0, broken = 0;
int cudaGetDevice(int* d) { *d = device; return broken; }
int cudaDeviceGetAttribute(int* n, int, int d) { ++asked; *n = 100 + d; return broken; }
int sm_count() {%s}
int main() {
  for (int d : {0, 1, 63, 64, 200}) {
    device = d;
    const int first = sm_count(), before = asked, again = sm_count();
    std::printf("%%d %%d %%d\\n", first, again, asked - before);
  }
  broken = 1;
  std::printf("%%d\\n", sm_count());
}
"""


def test_any_device_has_its_count(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    with open(os.path.join(CSRC, "decode_attention.cu")) as f:
        src = body(f.read(), "int sm_count()")
    (tmp_path / "count.cpp").write_text(STANDS % src)
    exe = tmp_path / "count"
    subprocess.run([cxx, "-std=c++17", str(tmp_path / "count.cpp"), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert lines[:5] == ["100 100 0", "101 101 0", "163 163 0", "164 164 1", "300 300 1"]     # asked once for the devices that are kept
    assert lines[5] == "0"
