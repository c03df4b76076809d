"""The 8-bit caches' attention kernels for many rows, and for more than 16 of the few, share
out the registers that their blocks are launched with.  Where the compiler gives another
count than they are written for they must not run; every other call has to.  On the host: the
kernels' own files with the count stood in for, and the API's own check of a batch."""
import os
import subprocess

import pytest

import decode_qwen2_block_gb300 as blk
from decode_qwen2_block_gb300 import build as gpu_build

KERNELS = r"""
#include <cuda_runtime.h>
int %(regs)s;
template <typename K> cudaError_t attributes(cudaFuncAttributes* a, K) {
  a->numRegs = %(regs)s;
  return cudaSuccess;
}
template <typename K> cudaError_t set_attribute(K, cudaFuncAttribute, int) { return cudaSuccess; }
#define cudaFuncGetAttributes attributes
#define cudaFuncSetAttribute set_attribute
#include "%(file)s"
"""
MAIN = r"""
#include <stdio.h>
#include "blk_api.cu"
extern int many_regs, few_regs;
int main() {
  static int64_t ints[4];
  static int32_t table[4];
  blk_handle_s h = {};
  h.cfg.n_heads = 12; h.cfg.n_kv_heads = 2; h.cfg.head_dim = 128;
  h.num_sms = 152;
  h.paged_many = true;
  const int counts[3][2] = {{128, 168}, {120, 168}, {128, 160}};
  for (auto& c : counts) {
    many_regs = c[0];
    few_regs = c[1];
    printf("%d %d", (int)blk::configure_paged_many_kv8(&h.paged_many8),
           (int)blk::configure_paged_few_kv8(&h.paged_wide8));
    for (bool kv8 : {true, false})
      for (int64_t most : {1, 2, 3, 5, 6, 700}) {
        blk_paged_batch b = {};
        b.n_seqs = 1; b.n_rows = 1000; b.max_new = most; b.max_len = 4096;
        b.row_start = ints; b.cache_lens = ints; b.block_table = table;
        b.max_blocks = 64; b.n_pages = 64; b.page_size = 64;
        printf(" %d", check_paged(&h, &b, kv8));
      }
    printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def output(tmp_path_factory):
    gpu_build.build()
    d = tmp_path_factory.mktemp("registers8")
    (d / "t_many.cu").write_text(KERNELS % dict(regs="many_regs", file="paged_many_kv8.cu"))
    (d / "t_few.cu").write_text(KERNELS % dict(regs="few_regs", file="paged_few_kv8.cu"))
    (d / "t_main.cu").write_text(MAIN)
    names = [os.path.basename(f)[:-3] for f in gpu_build.sources()]
    objs = [os.path.join(gpu_build.BUILD, f"{n}.o") for n in names
            if n not in ("blk_api", "paged_many_kv8", "paged_few_kv8")]
    if not all(os.path.exists(o) for o in objs):
        gpu_build.build(force=True)
    jobs = [subprocess.Popen([gpu_build.NVCC, *gpu_build.ARCH, *gpu_build.FLAGS, "-I", gpu_build.CSRC,
                              "-c", str(d / f"{f}.cu"), "-o", str(d / f"{f}.o")])
            for f in ("t_many", "t_few", "t_main")]
    assert [j.wait() for j in jobs] == [0, 0, 0]
    subprocess.run([gpu_build.NVCC, *gpu_build.ARCH, "-o", str(d / "t"),
                    *(str(d / f"{f}.o") for f in ("t_many", "t_few", "t_main")), *objs], check=True)
    return [line.split() for line in subprocess.run([str(d / "t")], capture_output=True, text=True,
                                                    check=True).stdout.splitlines()]


def test_the_counts_that_the_kernels_are_written_for_serve_every_batch(output):
    assert output[0] == ["0"] * 14


def test_another_count_refuses_its_own_kernels_rows_alone(output):
    """6 heads per kv head: up to two tokens are 16 rows, up to five few; fp16 pools always."""
    no = str(blk.BLK_ERR_CUDA)
    assert output[1] == ["0", "0", "0", "0", "0", "0", no, no] + ["0"] * 6
    assert output[2] == ["0", "0", "0", "0", no, no, "0", "0"] + ["0"] * 6
