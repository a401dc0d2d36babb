"""Host-side arithmetic of the operators' kernels, compiled with the host compiler and
run on the CPU."""
import ctypes
import importlib.util
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_layer_stable_gb300", "csrc")


def compiled(tmp_path, source, *flags):
    """The shared library of a C++ source that may include the kernels' host headers."""
    src, so = tmp_path / "t.cpp", tmp_path / "t.so"
    src.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                    str(so), *flags], check=True)
    return ctypes.CDLL(str(so))


TILES = """
#include "row_tiles.h"
extern "C" int max_tok() { return moe::kMaxTok; }
extern "C" int tiles(int c) { return moe::tok_tiles(c); }
extern "C" int most(int c) { return moe::tok_most(c); }
extern "C" void starts(int c, int* out) {
  const int n = moe::tok_tiles(c);
  for (int t = 0; t < n; ++t) out[t] = moe::tok_start(c, n, t);
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("tiles"), TILES)


@pytest.mark.parametrize("counts", [range(0, 1300), [5136960, 5136961, 6000000, (1 << 24) + 1, 100000007],
                                    [(1 << 28) - 191, (1 << 28) - 1, 1 << 28]])
def test_tiles_cover_an_expert_s_rows(tiles, counts):
    """Tiles begin at 0, on multiples of 64, and none is empty or longer than the largest."""
    for c in counts:
        n, most = tiles.tiles(c), tiles.most(c)
        assert n == -(-c // tiles.max_tok()) and most <= tiles.max_tok()
        if n == 0:
            assert most == 0
            continue
        s = np.zeros(n, dtype=np.int32)
        tiles.starts(c, s.ctypes.data_as(ctypes.c_void_p))
        rows = np.diff(np.append(s.astype(np.int64), c))
        assert s[0] == 0 and not (s % 64).any() and rows.min() >= 1, c
        assert rows.max() == most if n <= 4 else rows.max() <= most, c
        # 128-row scale tiles that a tile touches: one where the largest tile has up to 128 rows, else two
        assert (s % 128 + rows).max() <= (128 if most <= 128 else 256), c


# The CUDA runtime's calls as fakes.  Two threads ask for 60 and 120 KB and both come to the call that
# sets the limit; the larger one's takes effect first and returns last (all waits end after half a second).
LIMIT = """
#include <chrono>
#include <condition_variable>
#include <initializer_list>
#include <mutex>
#include <stdio.h>
#include <thread>
#include "smem_limit.h"
static std::mutex m;
static std::condition_variable cv;
static int device = 0, limit = 0, sets = 0, in_set = 0;
static bool large_set = false, small_done = false;
static thread_local int who = 0;  // 1: the smaller, 2: the larger
template <typename P> static void until(std::unique_lock<std::mutex>& l, P p) {
  cv.wait_for(l, std::chrono::milliseconds(500), p);
}
extern "C" cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  if (a != cudaDevAttrMaxSharedMemoryPerBlockOptin) return cudaErrorInvalidValue;
  *v = 232448;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  *a = cudaFuncAttributes();
  a->sharedSizeBytes = 1000;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int v) {
  std::unique_lock<std::mutex> l(m);
  if (v > 232448 - 1000) return cudaErrorInvalidValue;
  ++sets;
  if (who != 0) {
    ++in_set;
    cv.notify_all();
    until(l, [] { return in_set == 2; });
    if (who == 1) until(l, [] { return large_set; });
  }
  limit = v;
  if (who == 2) {
    large_set = true;
    cv.notify_all();
    until(l, [] { return small_done; });
  }
  return cudaSuccess;
}
static int fail(const char* what) { return printf("%s, limit %d\\n", what, limit), 1; }
static void kernel(int) {}
static moe::SmemAllowed allowed, other;
int main() {
  const size_t small = 60000, large = 120000;
  cudaError_t es = cudaSuccess, el = cudaSuccess;
  std::thread a([&] {
    who = 1;
    es = moe::allow_smem(kernel, small, allowed);
    std::lock_guard<std::mutex> l(m);
    small_done = true;
    cv.notify_all();
  });
  std::thread b([&] { who = 2; el = moe::allow_smem(kernel, large, allowed); });
  a.join();
  b.join();
  if (es != cudaSuccess || el != cudaSuccess) return fail("refused");
  if (moe::allow_smem(kernel, large, allowed) != cudaSuccess || limit < (int)large)
    return fail("lowered");
  // once set, no more calls; sizes that need no limit make none
  const int n = sets;
  for (size_t bytes : {small, large, (size_t)200000})
    if (moe::allow_smem(kernel, bytes, allowed) != cudaSuccess || limit < (int)bytes) return fail("later call");
  if (sets != n) return fail("set again");
  if (moe::allow_smem(kernel, 1000, other) != cudaSuccess || sets != n) return fail("small size");
  // another device has a limit of its own; one past the table works too
  for (int d : {1, 64}) {
    device = d;
    limit = 0;
    if (moe::allow_smem(kernel, large, allowed) != cudaSuccess || limit < (int)large) return fail("other device");
  }
  return 0;
}
"""


def test_two_threads_cannot_lower_a_kernel_s_shared_memory(tmp_path):
    from mixture_experts_layer_stable_gb300 import build
    nvcc = shutil.which(build._nvcc()) or build._nvcc()
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(LIMIT)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC, "-isystem", include, str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("prenorm_block", os.path.join(ROOT, "examples", "prenorm_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("capacity", [0, 1, 2, 100])
def test_example_caps_ids_that_have_no_expert(example, capacity):
    """Rows that are dropped already (any id outside the experts) stay as they are and take no place."""
    E, ids = 4, [2, -1, 2, 0, 7, 2, 3, -1, 0, 2, -2 ** 31]
    seen, want = [0] * E, []
    for i in ids:
        if 0 <= i < E:
            seen[i] += 1
            want.append(i if seen[i] <= capacity else -1)
        else:
            want.append(i)
    got = example.cap_ids(torch.tensor(ids, dtype=torch.int32), E, capacity)
    assert got.dtype == torch.int32 and got.tolist() == want
