"""The norms' sums over a block, alone, at every number of warps.

A compiler has read the warps' parts of two sums at a wrong stride where one call
stood ahead of a loop with another (the norms' own tests saw it in the first row
of a block); the probe has that form.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    import fp4_quant_gb300.build as B
    B.build()  # the generated tables
    out = str(tmp_path_factory.mktemp("probe") / "libblocksum.so")
    subprocess.run([B._nvcc(), *B.ARCH, *B.NVCC_FLAGS, "-I", os.path.join(ROOT, "fp4_quant_gb300", "csrc"), "-I", B.INCLUDE, "-shared",
                    os.path.join(ROOT, "tests", "block_sum_probe.cu"), "-o", out], check=True)
    return ctypes.CDLL(out).gq_probe_block_sum


@pytest.mark.parametrize("n,warps", [(1, w) for w in range(1, 33)] + [(n, w) for n in (2, 3) for w in range(1, 17)])
def test_every_thread_has_the_sum(probe, n, warps):
    threads = 32 * warps
    got = np.full((4, n, threads), np.nan, np.float32)
    assert probe(n, warps, got.ctypes.data_as(ctypes.c_void_p)) == 0
    t = np.arange(threads)
    for c in range(4):
        for j in range(n):
            want = np.float32(((t * (2 * j + 1) + 7 * c + 3 * j) % 61).sum())
            assert (got[c, j] == want).all(), (c, j, want, got[c, j])
