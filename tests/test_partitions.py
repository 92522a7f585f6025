"""Partition sizes far above every context ("do not split") up to the largest
int32 multiple: the sizes the library reports, and the kernels' 32-bit
arithmetic on them, which is the same inline code on the host."""

import os
import subprocess

import pytest

from paged_kv_cache_247_gb300 import build as _build

LARGEST = 2**31 - 128          # a multiple of 128, the tensor-core kernel's quantum

CHECK = r"""
#include <stdio.h>
#include "kernels.h"
int main() {
  const int sizes[] = {32, 128, 2048, 1 << 30, 0x7fffff80 - 128, 0x7fffff80};
  const int lens[] = {0, 1, 127, 128, 129, 8192, 1 << 30, 0x7fffff00, 0x7fffffff};
  int bad = 0;
  for (int part : sizes)
    for (int ctx : lens) {
      const long long parts = ((long long)ctx + part - 1) / part;
      if (pkv::context_partitions(ctx, part) != parts) ++bad;
      for (long long i = 0; i < parts; i += parts > 64 ? parts / 64 : 1) {
        const long long end = (i + 1) * part < ctx ? (i + 1) * part : ctx;
        if (pkv::partition_end(ctx, (int)(i * part), part) != end) ++bad;
      }
      // a partition of a longer context of the batch: nothing of this one is in it
      if (parts * part < 0x7fffffff && pkv::partition_end(ctx, (int)(parts * part), part) != ctx) ++bad;
    }
  printf("%d bad\n", bad);
  return bad != 0;
}
"""


def test_kernel_arithmetic(tmp_path):
    src, exe = tmp_path / "check.cpp", str(tmp_path / "check")
    src.write_text(CHECK)
    r = subprocess.run([_build._nvcc(), "-std=c++17", "-I", _build.CSRC, "-I", _build.INCLUDE,
                        str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("max_ctx", [0, 1, 129, 8192])
def test_reported_sizes(lib, max_ctx):
    whole = max(128, -(-max_ctx // 128) * 128)
    for size in (lib.pkv_decode_workspace_size, lib.pkv_decode_weights_workspace_size,
                 lib.pkv_contiguous_workspace_size):
        assert size(4, 8, 2, 64, max_ctx, LARGEST) == size(4, 8, 2, 64, max_ctx, whole)
