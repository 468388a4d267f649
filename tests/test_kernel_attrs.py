"""The shared memory limits kept per kernel and device (csrc/kernel_attrs.h), compiled for
the host with a stand-in for the call that sets them."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "kernel_attrs.h"

#include <cstdio>
#include <map>
#include <utility>

// A launch on a device fits if the limit set there last is at least its size.
static std::map<std::pair<const void*, int>, int> limit;
static int sets = 0;
static attn::SharedMemoryLimits limits;

static bool launch(const void* kernel, int dev, int bytes, int fail = 0) {
  const int err = limits.allow(kernel, dev, bytes, [&](const void* k, int n) {
    ++sets;
    if (!fail) limit[{k, dev}] = n;
    return fail;
  });
  return err == 0 && limit[{kernel, dev}] >= bytes;
}

#define CHECK(x)                                   \
  if (!(x)) {                                      \
    std::printf("line %d: %s\n", __LINE__, #x);    \
    return 1;                                      \
  }

int main() {
  static char kernels[80];
  // A larger call on another device says nothing about this one ...
  CHECK(launch(kernels, 0, 55));
  CHECK(launch(kernels, 1, 75));
  CHECK(launch(kernels, 0, 73));
  // ... and a smaller one there lowers nothing here.
  CHECK(launch(kernels + 1, 0, 90));
  CHECK(launch(kernels + 1, 1, 50));
  CHECK(launch(kernels + 1, 0, 60));
  CHECK((limit[{kernels + 1, 0}] == 90));
  // Set once a size and device.
  const int before = sets;
  CHECK(launch(kernels, 0, 73) && launch(kernels, 0, 20) && launch(kernels, 1, 75));
  CHECK(sets == before);
  // A failed call is reported and not remembered.
  CHECK(!launch(kernels + 2, 63, 10, 7));
  CHECK(launch(kernels + 2, 63, 10));
  // More kernels than places: each call sets its own.
  for (int round = 0; round < 2; ++round)
    for (int i = 0; i < 80; ++i) CHECK(launch(kernels + i, 2, 100 + 10 * round));
  return 0;
}
"""


def test_limits_are_kept_per_kernel_and_device(tmp_path):
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "tensor_attn_fwd_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
