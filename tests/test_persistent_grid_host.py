"""The launch of a persistent kernel on several devices of one process, with a
stand-in for the CUDA runtime (CPU): what a device has been told or asked does
not count for another one."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "state_space_model_analytic_gb300", "csrc")

RUNTIME = r"""
#pragma once
#include <stddef.h>
enum cudaError_t { cudaSuccess = 0, cudaErrorInvalidDevice = 1 };
enum cudaDeviceAttr { cudaDevAttrMultiProcessorCount };
enum cudaFuncAttribute { cudaFuncAttributeMaxDynamicSharedMemorySize };
extern int device, limit[3], asked[3];  // current device; a kernel's limit and questions per device
inline cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
inline cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int d) {
  const int sms[3] = {152, 20, 152};
  if (d < 0 || d > 2) return cudaErrorInvalidDevice;
  *v = sms[d];
  return cudaSuccess;
}
template <typename K>
cudaError_t cudaFuncSetAttribute(K, cudaFuncAttribute, int bytes) {
  if (device == 2) return cudaErrorInvalidDevice;
  limit[device] = bytes;
  return cudaSuccess;
}
template <typename K>
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int* n, K, int, size_t) {
  ++asked[device];
  *n = device == 0 ? 3 : 2;
  return cudaSuccess;
}
"""

MAIN = r"""
#include "persistent_grid.h"
#include <stdio.h>
int device, limit[3], asked[3];
static void kernel() {}
int main() {
  static ssd::FitOf fit;
  const int devices[] = {0, 1, 0, 1, 2, 1};
  for (int d : devices) {
    device = d;
    int grid = -1;
    const cudaError_t e = ssd::persistent_grid(kernel, 256, 70000, 1000, 608, &fit, &grid);
    printf("%d %d %d %d\n", d, (int)e, grid, limit[d]);
  }
  int few = -1, cap = -1;
  device = 0;
  ssd::persistent_grid(kernel, 256, 70000, 7, 608, &fit, &few);
  ssd::persistent_grid(kernel, 256, 70000, 1000, 100, &fit, &cap);
  printf("%d %d %d %d\n", few, cap, asked[0], asked[1]);
}
"""


def test_every_device_is_asked_and_told(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no g++")
    (tmp_path / "cuda_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cc").write_text(MAIN)
    exe = str(tmp_path / "main")
    subprocess.run([cxx, "-std=c++17", "-I", str(tmp_path), "-I", CSRC, str(tmp_path / "main.cc"),
                    "-o", exe], check=True)
    rows = [tuple(map(int, r.split())) for r in
            subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()]
    # device, error, CTAs, the kernel's shared-memory limit there
    assert rows[:4] == [(0, 0, 456, 70000), (1, 0, 40, 70000), (0, 0, 456, 70000), (1, 0, 40, 70000)]
    assert rows[4][1] != 0 and rows[5] == (1, 0, 40, 70000)
    assert rows[6] == (7, 100, 1, 1)  # few steps, the cap; occupancy is asked for once a device
