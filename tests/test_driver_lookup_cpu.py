"""The tensor-map encoder is looked up in the driver once it is there: a lookup that fails
is not kept.  The built objects are linked against a stand-in for the CUDA runtime whose
lookup fails at first; nothing is launched and no GPU is needed."""
import os
import subprocess

import pytest

import speculative_decoding_draft_02_gb300 as dsp  # noqa: F401
from speculative_decoding_draft_02_gb300 import build as dsp_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <cstdio>
#include <cstdlib>
#include "dspark.h"
#include <cuda.h>
#include <cuda_runtime_api.h>

static int lookups = 0, fail = 2, encoded = 0, launches = 0;

extern "C" {
static CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                       const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
  ++encoded;
  return CUDA_SUCCESS;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult *q) {
  ++lookups;
  if (fail-- > 0) {
    *fn = nullptr;
    *q = cudaDriverEntryPointSymbolNotFound;
    return fail % 2 ? cudaErrorInsufficientDriver : cudaSuccess;
  }
  *fn = (void *)encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
// what else the objects name
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *, const void *, void **) {
  ++launches;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int *d) { return *d = 0, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaMemcpyFromSymbol(void *, const void *, size_t, size_t, cudaMemcpyKind) {
  return cudaSuccess;
}
cudaError_t cudaMemcpyToSymbol(const void *, const void *, size_t, size_t, cudaMemcpyKind) {
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int *n, const void *, const cudaLaunchConfig_t *) {
  return *n = 76, cudaSuccess;
}
void **__cudaRegisterFatBinary(void *) { static void *h; return &h; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, void *, void *, void *,
                            void *, int *) {}
void __cudaRegisterVar(void **, char *, char *, const char *, int, size_t, int, int) {}
unsigned __cudaPushCallConfiguration(dim3, dim3, size_t, void *) { return 0; }
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaSuccess; }
cudaError_t __cudaGetKernel(cudaKernel_t *k, const void *f) { return *k = (cudaKernel_t)f, cudaSuccess; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) {
  ++launches;
  return cudaSuccess;
}
}
void dspark_count_launches(unsigned long) {}

int dspark_make_tmap_bf16(CUtensorMap *, const void *, uint64_t, uint64_t, uint32_t);

int main(int argc, char **argv) {
  const bool head = argv[1][0] == 'h';
  int rc[4];
  for (int &r : rc) {
    if (head) {
      alignas(64) CUtensorMap m;
      r = dspark_make_tmap_bf16(&m, (void *)4096, 128, 64, 128);
    } else {
      void *p = (void *)4096;
      dspark_kv_cache c = {p, p, nullptr, nullptr, 2048, 128, 64, 4, 16, 2, 64, DSPARK_KV_BF16};
      r = dspark_tree_attention(&c, 1, 8, 1, 1, 1, p, 512, 64, (int *)p, (int *)p, nullptr, (int *)p,
                                0.1f, p, 512, 64, nullptr, p, (size_t)1 << 40, nullptr);
    }
  }
  std::printf("%d %d %d %d lookups %d encoded %d launches %d\n", rc[0], rc[1], rc[2], rc[3], lookups,
              encoded, launches);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    dsp_build.build(force=not os.path.exists(os.path.join(dsp_build.BUILD, "lm_head.o")))
    d = tmp_path_factory.mktemp("lookup")
    src, exe = d / "fake.cpp", d / "fake"
    src.write_text(FAKE)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(dsp_build.nvcc())))
    objs = [os.path.join(dsp_build.BUILD, f) for f in ("lm_head.o", "tree_attention.o")]
    p = subprocess.run(["g++", "-std=c++17", "-w", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.join(cuda, "include"), str(src), *objs,
                        "-Wl,--unresolved-symbols=ignore-all", "-o", str(exe)],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr[-4000:]
    return str(exe)


def out_of(program, which):
    p = subprocess.run([program, which], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0, p
    return p.stdout.split()


def test_the_lm_heads_lookup_is_tried_again(program):
    got = out_of(program, "head")
    assert got[:4] == ["-1", "-1", "0", "0"] and got[5] == "3" and got[7] == "2"


def test_the_attentions_lookup_is_tried_again(program):
    got = out_of(program, "attention")
    assert got[:4] == ["3", "3", "0", "0"]        # DSPARK_ERR_CUDA while there is no encoder
    assert got[5] == "3" and got[7] == "6" and got[9] == "4"
