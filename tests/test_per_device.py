"""State kept for each device (csrc/per_device.h), in a small host program: the
machine these tests run on has one GPU or none."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_mla_decode_08_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "per_device.h"

int main() {
  mla::OncePerDevice once;
  int runs[mla::kMaxDevices] = {};
  // every device has its own turn, whichever comes first
  for (int d : {0, 1, 0, 63, 1, 63}) {
    if (once.run(d, [&] { ++runs[d]; return 0; }) != 0) return 1;
  }
  if (runs[0] != 1 || runs[1] != 1 || runs[63] != 1 || runs[2] != 0) return 2;
  // a failure is reported and tried again, on its device alone
  int tries = 0;
  auto flaky = [&] { return ++tries < 3 ? 7 : 0; };
  if (once.run(5, flaky) != 7 || once.run(5, flaky) != 7 || once.run(5, flaky) != 0 || once.run(5, flaky) != 0) return 3;
  if (tries != 3) return 4;
  // threads that come at once wait for the one setup and see what it wrote
  mla::OncePerDevice shared;
  int value = 0, bad = 0;
  std::vector<std::thread> threads;
  for (int i = 0; i < 16; ++i)
    threads.emplace_back([&] {
      shared.run(3, [&] { std::this_thread::yield(); value += 41; return 0; });
      if (value != 41) bad = 1;
    });
  for (auto& t : threads) t.join();
  if (bad || value != 41) return 5;
  std::puts("ok");
  return 0;
}
"""


def test_setup_runs_once_on_every_device(tmp_path):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    done = subprocess.run([str(exe)], stdout=subprocess.PIPE, text=True, timeout=60)
    assert done.returncode == 0 and done.stdout.strip() == "ok"


def test_no_kernel_is_set_up_once_per_process():
    """cudaFuncSetAttribute acts on the current device: every use of it stands
    inside a setup that runs on each."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as fh:
            text = fh.read()
        at = text.find("cudaFuncSetAttribute(")
        while at >= 0:
            before = text[max(0, at - 400):at]
            assert before.rfind("once.run(") > before.rfind("call_once("), (name, at)
            at = text.find("cudaFuncSetAttribute(", at + 1)
