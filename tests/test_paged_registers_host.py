"""The many-row attention kernels share out the registers that their blocks are launched
with.  Where the compiler gives another count than they are written for they must not
run; every other call has to.  On the host: the kernel's own file with the count stood
in for, and the API's own check of a batch."""
import os
import subprocess

import pytest

import decode_qwen2_block_gb300 as blk
from decode_qwen2_block_gb300 import build as gpu_build

MANY = r"""
#include <cuda_runtime.h>
int test_regs = 168;
template <typename K> cudaError_t attributes(cudaFuncAttributes* a, K) {
  a->numRegs = test_regs;
  return cudaSuccess;
}
template <typename K> cudaError_t set_attribute(K, cudaFuncAttribute, int) { return cudaSuccess; }
#define cudaFuncGetAttributes attributes
#define cudaFuncSetAttribute set_attribute
#include "paged_many.cu"
"""
MAIN = r"""
#include <stdio.h>
#include "blk_api.cu"
extern int test_regs;
int main() {
  static int64_t ints[4];
  static int32_t table[4];
  blk_handle_s h = {};
  h.cfg.n_heads = 12; h.cfg.n_kv_heads = 2; h.cfg.head_dim = 128;
  h.num_sms = 152;
  for (int regs : {168, 160}) {
    test_regs = regs;
    printf("%d", (int)blk::configure_paged_many(&h.paged_many));
    for (int64_t most : {1, 5, 6, 700}) {
      blk_paged_batch b = {};
      b.n_seqs = 1; b.n_rows = 1000; b.max_new = most; b.max_len = 4096;
      b.row_start = ints; b.cache_lens = ints; b.block_table = table;
      b.max_blocks = 64; b.n_pages = 64; b.page_size = 64;
      printf(" %d", check_paged(&h, &b));
    }
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def output(tmp_path_factory):
    gpu_build.build()
    d = tmp_path_factory.mktemp("registers")
    (d / "t_many.cu").write_text(MANY)
    (d / "t_main.cu").write_text(MAIN)
    names = [os.path.basename(f)[:-3] for f in gpu_build.sources()]
    objs = [os.path.join(gpu_build.BUILD, f"{n}.o") for n in names
            if n not in ("blk_api", "paged_many")]
    if not all(os.path.exists(o) for o in objs):
        gpu_build.build(force=True)
    for f in ("t_many", "t_main"):
        subprocess.run([gpu_build.NVCC, *gpu_build.ARCH, *gpu_build.FLAGS, "-I", gpu_build.CSRC, "-c",
                        str(d / f"{f}.cu"), "-o", str(d / f"{f}.o")], check=True)
    subprocess.run([gpu_build.NVCC, *gpu_build.ARCH, "-o", str(d / "t"), str(d / "t_many.o"),
                    str(d / "t_main.o"), *objs], check=True)
    return subprocess.run([str(d / "t")], capture_output=True, text=True,
                          check=True).stdout.splitlines()


def test_the_count_that_the_kernels_are_written_for_serves_every_batch(output):
    assert output[0].split() == ["0", "0", "0", "0", "0"]


def test_another_count_refuses_many_rows_alone(output):
    """6 heads per kv head: up to five tokens are few rows."""
    refused = str(blk.BLK_ERR_CUDA)
    assert output[1].split() == ["0", "0", "0", refused, refused]
