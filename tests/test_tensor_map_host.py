"""The tensor-map encoder's lookup against a stand-in for the driver: CPU only."""
import ctypes
import os
import subprocess

from early_exit_decoding_layer_gb300 import build

SOURCE = """
#include <cuda.h>
#include <cuda_runtime.h>

// the driver: not there for the first `missing` lookups, then an encoder that says what it got
static int missing = 0, lookups = 0, last_rank = 0, last_type = 0;
static CUresult encode(CUtensorMap*, CUtensorMapDataType type, cuuint32_t rank, void*, const cuuint64_t*, const cuuint64_t*,
                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
  last_rank = (int)rank;
  last_type = (int)type;
  return CUDA_SUCCESS;
}
static cudaError_t stand_in(const char*, void** f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult* q) {
  *f = nullptr;
  *q = cudaDriverEntryPointSymbolNotFound;
  if (++lookups <= missing) return cudaErrorInitializationError;
  *f = (void*)encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
#define cudaGetDriverEntryPointByVersion stand_in
#include "ee_tensor_map.cu"

extern "C" void set_missing(int n) { missing = n; }
extern "C" int lookup_count() { return lookups; }
extern "C" int rank_seen() { return last_rank; }
extern "C" int try_encode(int rank) {
  CUtensorMap m;
  const uint64_t dims[5] = {64, 8, 8, 8, 8}, strides[4] = {128, 1024, 8192, 65536};
  const uint32_t box[5] = {64, 1, 1, 1, 1};
  return ee::encode_tensor_map(&m, false, rank, nullptr, dims, strides, box);
}
"""


def test_a_failed_lookup_is_tried_again(tmp_path):
    src, out = tmp_path / "t.cu", tmp_path / "t.so"
    src.write_text(SOURCE)
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-I" + build.CSRC, "-I" + os.path.join(build.CSRC, "..", "include"),
                        "-shared", str(src), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(out))
    lib.set_missing(2)
    assert [lib.try_encode(2) for _ in range(4)] == [0, 0, 1, 1]
    assert lib.lookup_count() == 3 and lib.rank_seen() == 2   # found once, kept
    assert [lib.try_encode(n) for n in (0, 1, 3, 4, 5, 6)] == [0, 1, 1, 1, 1, 0]
