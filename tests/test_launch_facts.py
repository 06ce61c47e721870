"""What the launchers look up about a kernel is asked of CUDA once, however many kernels and
sizes a process runs: csrc/occupancy.cu compiled against a runtime that counts (no GPU)."""
import ctypes
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A runtime of one device whose answers are made of the question, and the library's error hook.
FAKE = r"""
#include <cuda_runtime_api.h>
namespace nvfp4 {
int resident_blocks_fn(const void *fn, int threads, size_t smem);
int resident_clusters_fn(const void *fn, int threads, size_t smem, int size);
void set_last_cuda_error(cudaError_t) {}
}
static int g_blocks, g_clusters, g_attrs, g_fail;
extern "C" {
cudaError_t cudaGetDevice(int *d) { *d = 0; return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { *v = 148; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) {
  ++g_attrs;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int t, size_t s) {
  ++g_blocks;
  *n = t + (int)s;
  return g_fail ? cudaErrorInvalidValue : cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *c) {
  ++g_clusters;
  *n = (int)c->attrs[0].val.clusterDim.x;
  return cudaSuccess;
}
int ask_blocks(long fn, int threads, long smem) {
  return nvfp4::resident_blocks_fn((const void *)fn, threads, (size_t)smem);
}
int ask_clusters(long fn, int threads, long smem, int size) {
  return nvfp4::resident_clusters_fn((const void *)fn, threads, (size_t)smem, size);
}
void fail(int on) { g_fail = on; }
int asked(int what) { return what == 0 ? g_blocks : what == 1 ? g_clusters : g_attrs; }
}
"""


def test_each_question_is_asked_once(tmp_path):
    from bit_quantized_moe_nvfp4_b200 import build
    src, fake, facts, so = (str(tmp_path / n) for n in ("fake.cpp", "fake.o", "facts.o", "l.so"))
    with open(src, "w") as f:
        f.write(FAKE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.NVCC)), "include")
    subprocess.run(["g++", "-std=c++17", "-fPIC", "-I", cuda, "-c", src, "-o", fake], check=True)
    subprocess.run([build.NVCC, *build.FLAGS, "-c", os.path.join(build.CSRC, "occupancy.cu"),
                    "-o", facts], check=True)
    # linked without a CUDA runtime: the calls go to the stand-ins above
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", fake, facts, "-o", so], check=True)
    L = ctypes.CDLL(str(so), mode=os.RTLD_LAZY)
    L.ask_blocks.argtypes = [ctypes.c_long, ctypes.c_int, ctypes.c_long]
    L.ask_clusters.argtypes = [ctypes.c_long, ctypes.c_int, ctypes.c_long, ctypes.c_int]
    keys = [(fn, 32 * t, 1024 * m) for fn in range(1, 41) for t in range(1, 33) for m in (1, 2)]
    for _ in range(2):
        for fn, t, m in keys:
            assert L.ask_blocks(fn, t, m) == t + m
            assert L.ask_clusters(fn, t, m, 4) == 4
    assert L.asked(0) == len(keys) and L.asked(1) == len(keys)
    assert L.asked(2) == 40 * 2      # a kernel's limit is raised as its memory grows, never again
    # a failed query is not an answer
    L.fail(1)
    assert L.ask_blocks(99, 32, 0) == -1
    L.fail(0)
    assert L.ask_blocks(99, 32, 0) == 32
