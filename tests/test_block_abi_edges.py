"""Calls at the edges of what the entry points between a block's linear layers
accept, on the CPU: what is refused before anything touches the GPU, and sizes
that the host works out."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIP_INCLUDE = "/opt/rocm/include"
P, Q = ctypes.c_void_p(4096), ctypes.c_void_p(8192)  # never dereferenced
REACHED = fp8q.ERR_DEVICE  # accepted, without a GPU


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fp8q.LIB_PATH):
        pytest.skip("libfp8q.so is not built")
    return fp8q.load_library()


def test_dx_over_dresidual_at_another_stride_is_refused(lib):
    """A workgroup's rows of dx would land on rows of dresidual that another has yet to read."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would run")
    # 0 dy, dtype, rows, N, ld, 5 h, dtype, ld, 8 rstd, weight, dtype, 11 dres, ld, 13 dx, dtype, ld, 16 mode, codes, ld, scales, 20 dweight, workspace, bytes, stream
    for rows, dres, ldr, dx, ldx, status in ((4, P, 16, P, 8, fp8q.ERR_SHAPE), (4, P, 8, P, 16, fp8q.ERR_SHAPE), (2, P, 9, P, 8, fp8q.ERR_SHAPE), (4, P, 16, P, 16, REACHED),
                                             (4, P, 16, Q, 8, REACHED), (1, P, 16, P, 8, REACHED), (4, P, 16, None, 8, REACHED)):
        codes = None if dx else Q
        args = [Q, 1, rows, 8, 8, Q, 1, 8, Q, Q, 1, dres, ldr, dx, 1, ldx, 0, codes, 8, codes, None, None, 0, None]
        assert lib.fp8q_rmsnorm_backward(*args) == status, (rows, ldr, ldx)


def test_gradients_workspace_holds_the_shares_that_are_written(lib):
    """A share a workgroup, or of rows beyond a workgroup's registers one of every 32 rows: not one of every row."""
    need = lib.fp8q_rmsnorm_backward_workspace
    for rows, n, shares in ((8192, 7168, 256), (512, 20000, 16), (64, 1 << 29, 2), (1, 16385, 1), (33, 40000, 2), (1 << 20, 40000, 512), (100000, 512, 512), (5, 512, 5), (8192, 7169, 512)):
        assert need(rows, n) == shares * ((n + 7) // 8 * 8) * 4, (rows, n)


def test_host_sizes_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("g++ or the HIP headers are not available")
    exe = str(tmp_path / "host_block_sizes_check")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-Wall", "-Werror",
           "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "fine_grained_fp8_fp8q_amd", "csrc"),
           os.path.join(ROOT, "tests", "host_block_sizes_check.cpp"), "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "host block size checks passed" in run.stdout
