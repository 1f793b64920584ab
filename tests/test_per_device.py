"""Setup that is made once for each device (csrc/per_device.h), with devices and a failing setup played by the host."""
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

PROGRAM = r"""
#include "per_device.h"
#include <cstdio>
int main() {
  std::atomic<uint64_t> done{0};
  int made[100] = {0};
  auto on = [&](int device, int result) {
    return mlora::once_per_device<int>(done, device, [&] { ++made[device]; return result; });
  };
  // a first failure is returned, tried again, and does not touch the other devices
  if (on(0, 2) != 2 || on(0, 0) != 0 || on(0, 5) != 0 || made[0] != 2) return 1;
  // a second device is set up too, and a change back sets up nothing again
  if (on(1, 0) != 0 || on(0, 7) != 0 || on(1, 7) != 0 || made[0] != 2 || made[1] != 1) return 2;
  if (on(63, 0) != 0 || on(63, 7) != 0 || made[63] != 1) return 3;
  // beyond the 64 that are kept: every time
  if (on(64, 0) != 0 || on(64, 3) != 3 || made[64] != 2) return 4;
  std::puts("ok");
  return 0;
}
"""


def test_once_for_each_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("g++ missing")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.check_call([cxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "rank_adapter_gemm_token_gb300", "csrc"),
                           str(src), "-o", str(exe)])
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == "ok\n"


def test_attention_launchers_keep_no_setup_of_one_device():
    """Their kernels want more than 48 KB of shared memory, which each device has to be asked for."""
    for name in ("attention_rows.cu", "attention_tiles.cu"):
        text = open(os.path.join(ROOT, "rank_adapter_gemm_token_gb300", "csrc", name)).read()
        assert "allow_shared_memory<" in text and "cudaFuncSetAttribute" not in text
