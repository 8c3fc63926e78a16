"""The entry points between a block's linear layers on the CPU: refusals come
before anything touches the GPU (through the built library), the same host code
under AddressSanitizer and UndefinedBehaviorSanitizer, and the binding's own
checks."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import fine_grained_fp8_fp8q_amd as fp8q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fine_grained_fp8_fp8q_amd", "csrc")
HIP_INCLUDE = "/opt/rocm/include"
P, P8, Q = ctypes.c_void_p(4096), ctypes.c_void_p(4104), ctypes.c_void_p(8192)  # never dereferenced
OK, ARG, SHAPE, ALIGN = fp8q.OK, fp8q.ERR_INVALID_ARG, fp8q.ERR_SHAPE, fp8q.ERR_ALIGN
BIG = 1 << 31


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fp8q.LIB_PATH):
        pytest.skip("libfp8q.so is not built")
    return fp8q.load_library()


def refused(fn, good, changes):
    """Each change of one argument of a call that would be accepted gives its status."""
    for at, value, status in changes:
        args = list(good)
        args[at] = value
        assert fn(*args) == status, (at, value, status)


def test_rmsnorm_refusals(lib):
    # 0 x, x_dtype, rows, N, ld_x, 5 residual, dtype, ld, 8 h, ld_h, 10 weight, dtype, eps, 13 y, ld_y, mode, 16 codes, ld, scales, rstd, stream
    good = [P, 1, 4, 8, 8, P, 1, 8, Q, 8, P, 1, 1e-6, P, 8, 0, P, 8, P, P, None]
    nan = float("nan")
    refused(lib.fp8q_rmsnorm_quantize, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (2, BIG, ARG), (3, -1, ARG), (4, 7, SHAPE), (4, BIG, ARG), (5, None, ARG), (6, 2, ARG), (7, 7, SHAPE), (9, 7, SHAPE),
        (10, None, ARG), (11, -1, ARG), (12, 0.0, ARG), (12, -1.0, ARG), (12, nan, ARG), (12, float("inf"), ARG), (14, 7, SHAPE), (15, 2, ARG), (17, 7, SHAPE),
        (18, None, ARG), (0, P8, ALIGN), (5, P8, ALIGN), (8, P8, ALIGN), (10, P8, ALIGN), (13, P8, ALIGN), (16, P8, ALIGN), (18, P8, ALIGN), (19, P8, ALIGN), (2, 0, OK)])
    none = list(good)
    for at in (8, 13, 16, 19):
        none[at] = None
    assert lib.fp8q_rmsnorm_quantize(*none) == ARG  # nothing to write
    over = list(good)
    over[8], over[9] = P, 16  # the stream over its own input, at another stride
    assert lib.fp8q_rmsnorm_quantize(*over) == SHAPE
    wide = list(good)
    wide[3] = wide[4] = wide[7] = wide[9] = wide[14] = wide[17] = 1 << 30
    assert lib.fp8q_rmsnorm_quantize(*wide) == SHAPE
    empty = list(good)
    empty[3], empty[19] = 0, None
    assert lib.fp8q_rmsnorm_quantize(*empty) == OK


def test_rmsnorm_backward_refusals(lib):
    # 0 dy, dtype, rows, N, ld, 5 h, dtype, ld, 8 rstd, 9 weight, dtype, 11 dres, ld, 13 dx, dtype, ld, 16 mode, codes, ld, scales, 20 dweight, workspace, bytes, stream
    need = lib.fp8q_rmsnorm_backward_workspace(4, 8)
    good = [P, 1, 4, 8, 8, P, 1, 8, P, P, 1, P, 8, P, 1, 8, 0, P, 8, P, P, P, need, None]
    refused(lib.fp8q_rmsnorm_backward, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (3, -1, ARG), (4, 7, SHAPE), (5, None, ARG), (6, 2, ARG), (7, 7, SHAPE), (8, None, ARG), (9, None, ARG), (10, 5, ARG),
        (12, 7, SHAPE), (14, 2, ARG), (15, 7, SHAPE), (16, 2, ARG), (18, 7, SHAPE), (19, None, ARG), (22, -1, ARG), (0, P8, ALIGN), (5, P8, ALIGN), (8, P8, ALIGN),
        (9, P8, ALIGN), (11, P8, ALIGN), (13, P8, ALIGN), (17, P8, ALIGN), (19, P8, ALIGN), (20, P8, ALIGN), (3, 0, OK)])
    if need:
        refused(lib.fp8q_rmsnorm_backward, good, [(21, None, ARG), (22, need - 1, ARG), (21, P8, ALIGN)])
    none = list(good)
    for at in (13, 17, 20):
        none[at] = None
    assert lib.fp8q_rmsnorm_backward(*none) == ARG
    nothing = list(good)
    nothing[2], nothing[20] = 0, None
    assert lib.fp8q_rmsnorm_backward(*nothing) == OK  # no rows and no dweight


def test_rmsnorm_quantize_t_refusals(lib):
    # h, dtype, h_rows, N, ld_h, 5 rstd, weight, dtype, 8 index, rows, mode, 11 codes, ld, scales, stream
    good = [P, 1, 4, 8, 8, P, P, 1, P, 6, 0, P, 6, P, None]
    refused(lib.fp8q_rmsnorm_quantize_t, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (3, -1, ARG), (4, 7, SHAPE), (5, None, ARG), (6, None, ARG), (7, 2, ARG), (8, None, SHAPE), (9, -1, ARG), (10, 2, ARG),
        (11, None, ARG), (12, 5, SHAPE), (13, None, ARG), (0, P8, ALIGN), (5, P8, ALIGN), (6, P8, ALIGN), (8, P8, ALIGN), (11, P8, ALIGN), (13, P8, ALIGN), (9, 0, OK), (3, 0, OK)])
    many = list(good)
    many[9] = many[12] = BIG - 1
    many[3] = many[4] = 64
    assert lib.fp8q_rmsnorm_quantize_t(*many) == SHAPE


def test_route_refusals(lib):
    # 0 logits, dtype, tokens, E, ld, 5 bias, score, groups, top_groups, group_score, 10 topk, renormalize, scale, index_dtype, 14 experts, weights, scores, load, stream
    good = [P, 0, 4, 16, 16, P, 1, 4, 2, 1, 8, 1, 1.0, 0, P, P, P, P, None]
    refused(lib.fp8q_moe_route, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (3, -1, ARG), (4, 15, SHAPE), (6, 2, ARG), (6, -1, ARG), (7, 0, ARG), (7, 3, SHAPE), (7, 65, SHAPE), (8, 0, ARG), (8, 5, SHAPE),
        (9, 2, ARG), (10, -1, ARG), (10, 9, SHAPE), (10, 65, SHAPE), (12, float("nan"), ARG), (12, float("inf"), ARG), (13, 2, ARG), (14, None, ARG), (15, None, ARG),
        (0, P8, ALIGN), (5, P8, ALIGN), (14, P8, ALIGN), (15, P8, ALIGN), (16, P8, ALIGN), (17, P8, ALIGN), (2, 0, OK)])
    big = list(good)
    big[3] = big[4] = 516
    assert lib.fp8q_moe_route(*big) == SHAPE
    assert lib.fp8q_moe_route(P, 0, 4, 0, 0, None, 0, 1, 1, 0, 0, 0, 1.0, 0, None, None, None, None, None) == OK


def test_route_backward_refusals(lib):
    # 0 dweights, experts, index_dtype, tokens, topk, 5 logits, dtype, E, ld, 9 score, renormalize, scale, dscores, 13 dlogits, dtype, ld, stream
    good = [P, P, 0, 4, 8, P, 0, 16, 16, 1, 1, 1.0, P, P, 0, 16, None]
    refused(lib.fp8q_moe_route_backward, good, [
        (0, None, ARG), (1, None, ARG), (2, 2, ARG), (3, -1, ARG), (4, -1, ARG), (4, 17, SHAPE), (5, None, ARG), (6, 2, ARG), (7, -1, ARG), (7, 513, SHAPE), (8, 15, SHAPE),
        (9, 2, ARG), (11, float("nan"), ARG), (13, None, ARG), (14, 2, ARG), (15, 15, SHAPE), (15, -1, ARG), (0, P8, ALIGN), (1, P8, ALIGN), (5, P8, ALIGN), (12, P8, ALIGN),
        (13, P8, ALIGN), (3, 0, OK)])


def test_good_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    dev, need = fp8q.ERR_DEVICE, lib.fp8q_rmsnorm_backward_workspace(4, 7)
    assert lib.fp8q_rmsnorm_quantize(P, 0, 4, 7, 9, None, 1, 0, None, 0, P, 0, 1e-6, None, 0, 1, P, 7, P, None, None) == dev
    assert lib.fp8q_rmsnorm_quantize(None, 0, 4, 0, 0, None, 1, 0, None, 0, None, 0, 1e-6, None, 0, 1, None, 0, None, P, None) == dev  # rstd of empty rows
    assert lib.fp8q_rmsnorm_backward(P, 0, 4, 7, 7, P, 1, 7, P, P, 0, None, 0, P, 0, 7, 0, None, 0, None, P, P, need, None) == dev
    assert lib.fp8q_rmsnorm_backward(None, 0, 0, 7, 7, None, 1, 7, None, None, 0, None, 0, None, 0, 7, 0, None, 0, None, P, None, 0, None) == dev  # zeros
    assert lib.fp8q_rmsnorm_quantize_t(P, 0, 4, 7, 7, P, P, 0, None, 4, 0, P, 4, P, None) == dev
    assert lib.fp8q_rmsnorm_quantize_t(None, 0, 0, 7, 7, None, P, 0, P, 4, 0, P, 4, P, None) == dev  # an index outside: zeros
    assert lib.fp8q_moe_route(P, 0, 1, 7, 0, None, 0, 1, 1, 0, 2, 0, 1.0, 1, P, P, None, None, None) == dev
    assert lib.fp8q_moe_route_backward(P, P, 1, 4, 2, P, 0, 7, 7, 0, 0, 1.0, None, P, 1, 7, None) == dev


def test_binding_refuses_host_tensors_and_what_is_no_tensor(monkeypatch):
    x, w, r = torch.zeros((4, 8)), torch.zeros(8), torch.zeros(4)
    e = torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: fp8q.rmsnorm_quantize(x, w), lambda: fp8q.rmsnorm_backward(x, x, r, w), lambda: fp8q.rmsnorm_quantize_t(x, r, w),
                 lambda: fp8q.moe_route(x, 2), lambda: fp8q.moe_route_backward(x[:, :2].contiguous(), e, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()

    def rows_of(t, name, dtypes, checked=fp8q._rows_of):
        return (*t.shape, t.shape[1], 4096) if isinstance(t, torch.Tensor) else checked(t, name, dtypes)

    def vector(t, n, dtypes, name, checked=fp8q._vector):
        return 4096 if isinstance(t, torch.Tensor) else checked(t, n, dtypes, name)

    monkeypatch.setattr(fp8q, "_rows_of", rows_of)
    monkeypatch.setattr(fp8q, "_vector", vector)
    monkeypatch.setattr(fp8q, "_contig_f32", lambda t, name: fp8q._need(t, torch.int64, name) if not isinstance(t, torch.Tensor) else None)
    for name, call in (("x", lambda: fp8q.rmsnorm_quantize(x.tolist(), w)), ("weight", lambda: fp8q.rmsnorm_quantize(x, w.tolist())),
                       ("residual", lambda: fp8q.rmsnorm_quantize(x, w, residual=x.tolist())), ("h_out", lambda: fp8q.rmsnorm_quantize(x, w, residual=x, h_out=x.tolist())),
                       ("dy", lambda: fp8q.rmsnorm_backward(x.tolist(), x, r, w)), ("h", lambda: fp8q.rmsnorm_backward(x, x.tolist(), r, w)),
                       ("rstd", lambda: fp8q.rmsnorm_backward(x, x, r.tolist(), w)), ("dres", lambda: fp8q.rmsnorm_backward(x, x, r, w, dres=x.tolist())),
                       ("index", lambda: fp8q.rmsnorm_quantize_t(x, r, w, index=[0])), ("bias", lambda: fp8q.moe_route(x, 2, bias=[0.0] * 8)),
                       ("load", lambda: fp8q.moe_route(x, 2, load=[0] * 8)), ("dweights", lambda: fp8q.moe_route_backward(r.tolist(), e, x)),
                       ("experts", lambda: fp8q.moe_route_backward(x[:, :2], e.tolist(), x)), ("dscores", lambda: fp8q.moe_route_backward(x[:, :2], e, x, dscores=x.tolist()))):
        with pytest.raises(TypeError, match=name):
            call()


def test_numbers_that_do_not_fit_are_refused_before_the_call(monkeypatch):
    """ctypes keeps the low bits of a number that does not fit: none gets that far."""
    class Lib:
        @staticmethod
        def fp8q_moe_route(*_):
            raise AssertionError("called")

    monkeypatch.setattr(fp8q, "_lib", Lib)
    monkeypatch.setattr(fp8q, "_rows_of", lambda t, name, dtypes: (2, 8, 8, 4096))
    x = torch.zeros((2, 8))
    for bad in (dict(topk=1 << 64), dict(topk=(1 << 64) + 2), dict(topk=9), dict(topk=-1), dict(topk=2, groups=1 << 32), dict(topk=2, groups=(1 << 32) + 2, top_groups=1),
                dict(topk=2, top_groups=0), dict(topk=2, groups=2, top_groups=(1 << 32) + 1)):
        with pytest.raises(ValueError):
            fp8q.moe_route(x, **bad)


def test_host_code_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("g++ or the HIP headers are not available")
    exe = str(tmp_path / "host_block_abi_check")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE,
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "fp8q_block_api.cpp"), os.path.join(ROOT, "tests", "host_block_abi_check.cpp"), "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "host block ABI checks passed" in run.stdout
