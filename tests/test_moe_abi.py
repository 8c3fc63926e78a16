"""The expert-layer entry points on the CPU: refusals come before anything
touches the GPU (through the built library), the same host code under
AddressSanitizer and UndefinedBehaviorSanitizer, and the binding's own checks."""

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
P, P8 = ctypes.c_void_p(4096), ctypes.c_void_p(4104)  # never dereferenced
ARG, SHAPE, ALIGN = fp8q.ERR_INVALID_ARG, fp8q.ERR_SHAPE, fp8q.ERR_ALIGN


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


def test_sort_refusals(lib):
    # experts, index, tokens, topk, ld, first, G, align, cap, offsets, token, row_of, workspace, bytes, stream
    good = [P, 0, 4, 2, 2, 0, 3, 4, 16, P, P, P, None, 0, None]
    refused(lib.fp8q_moe_sort, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (3, -1, ARG), (4, 1, SHAPE), (5, -1, ARG), (6, -1, ARG), (6, 513, SHAPE),
        (7, 0, ARG), (7, 3, SHAPE), (8, 18, SHAPE), (8, 1 << 31, ARG), (9, None, ARG), (10, None, ARG), (11, None, ARG),
        (13, -1, ARG), (0, P8, ALIGN), (9, P8, ALIGN), (10, P8, ALIGN), (11, P8, ALIGN)])
    good[6] = 0
    assert lib.fp8q_moe_sort(*good) == fp8q.OK  # no experts: nothing is written


def test_combine_refusals(lib):
    # y, y_dtype, cap, N, ld_y, row_of, weights, tokens, topk, out_dtype, out, ld_out, stream
    good = [P, 1, 16, 8, 8, P, P, 4, 2, 1, P, 8, None]
    refused(lib.fp8q_moe_combine, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (3, -1, ARG), (4, 7, SHAPE), (5, None, ARG), (8, -1, ARG), (9, 7, ARG),
        (10, None, ARG), (11, 7, SHAPE), (0, P8, ALIGN), (5, P8, ALIGN), (6, P8, ALIGN), (10, P8, ALIGN),
        (7, 0, fp8q.OK), (3, 0, fp8q.OK)])


def test_combine_backward_refusals(lib):
    # dout, dtype, tokens, N, ld, y, dtype, cap, ld_y, row_of, weights, topk, token, dy, ld_dy, mode, codes, ld, scales, dweights, stream
    good = [P, 1, 4, 8, 8, P, 1, 16, 8, P, P, 2, P, P, 8, 0, P, 8, P, P, None]
    refused(lib.fp8q_moe_combine_backward, good, [
        (0, None, ARG), (1, 2, ARG), (2, -1, ARG), (3, -1, ARG), (4, 7, SHAPE), (5, None, ARG), (6, 2, ARG), (7, -1, ARG),
        (8, 7, SHAPE), (9, None, ARG), (11, -1, ARG), (14, 7, SHAPE), (15, 2, ARG), (17, 7, SHAPE), (18, None, ARG),
        (0, P8, ALIGN), (5, P8, ALIGN), (9, P8, ALIGN), (10, P8, ALIGN), (12, P8, ALIGN), (13, P8, ALIGN), (16, P8, ALIGN),
        (18, P8, ALIGN), (19, P8, ALIGN)])


def test_swiglu_backward_refusals(lib):
    # x, x_scales, rows, inter, ld_x, dy, ld_dy, dx, ld_dx, mode, codes, ld_codes, scales, y, ld_y, stream
    good = [P, P, 4, 128, 256, P, 128, P, 256, 0, P, 256, P, P, 128, None]
    refused(lib.fp8q_swiglu_backward, good, [
        (0, None, ARG), (2, -1, ARG), (3, -1, ARG), (3, 100, SHAPE), (4, 255, SHAPE), (5, None, ARG), (6, 127, SHAPE),
        (8, 255, SHAPE), (9, 2, ARG), (11, 255, SHAPE), (12, None, ARG), (14, 127, SHAPE), (0, P8, ALIGN), (1, P8, ALIGN),
        (5, P8, ALIGN), (7, P8, ALIGN), (10, P8, ALIGN), (12, P8, ALIGN), (13, P8, ALIGN), (2, 0, fp8q.OK), (3, 0, fp8q.OK)])
    none = [P, None, 4, 100, 200, P, 100, None, 0, 0, None, 0, None, None, 0, None]
    assert lib.fp8q_swiglu_backward(*none) == ARG  # nothing to write


def test_grouped_wgrad_refusals(lib):
    # dy_t, dy_scales, x_t, x_scales, offsets, G, cap, Nout, Kin, dw, ld_dw, stream
    good = [P, P, P, P, P, 2, 256, 4, 8, P, 8, None]
    refused(lib.fp8q_grouped_wgrad, good, [
        (0, None, ARG), (1, None, ARG), (2, None, ARG), (3, None, ARG), (4, None, ARG), (5, -1, ARG), (6, 200, SHAPE),
        (6, -128, ARG), (9, None, ARG), (10, 7, SHAPE), (7, 1 << 24, SHAPE), (0, P8, ALIGN), (1, P8, ALIGN), (2, P8, ALIGN),
        (3, P8, ALIGN), (4, P8, ALIGN), (9, P8, ALIGN), (5, 0, fp8q.OK), (7, 0, fp8q.OK), (8, 0, fp8q.OK)])
    ex = good[:9] + [4] + good[9:]
    assert lib.fp8q_grouped_wgrad_ex(*ex) == ARG  # accumulation form


def test_good_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    dev = fp8q.ERR_DEVICE
    assert lib.fp8q_moe_sort(P, 0, 4, 2, 2, 0, 3, 4, 16, P, P, P, None, 0, None) == dev
    assert lib.fp8q_moe_combine(P, 1, 16, 7, 9, P, None, 4, 2, 0, P, 7, None) == dev
    assert lib.fp8q_moe_combine_backward(P, 0, 4, 7, 7, None, 0, 16, 0, P, None, 2, None, P, 7, 0, None, 0, None, None, None) == dev
    assert lib.fp8q_swiglu_backward(P, None, 4, 7, 14, P, 7, P, 14, 0, None, 0, None, None, 0, None) == dev
    assert lib.fp8q_grouped_wgrad(P, P, P, P, P, 2, 256, 5, 7, P, 7, None) == dev


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="GPU"):
        fp8q.moe_sort(torch.zeros((2, 2), dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        fp8q.moe_sort(torch.zeros((2, 2)), 4)
    y, rows = torch.zeros((4, 8), dtype=torch.bfloat16), torch.zeros((2, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        fp8q.moe_combine(y, rows)
    with pytest.raises(ValueError, match="GPU"):
        fp8q.moe_combine_backward(y[:2], y, rows)
    with pytest.raises(ValueError, match="GPU"):
        fp8q.swiglu_backward(y, y[:, :4])
    c, s = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1))
    with pytest.raises(ValueError, match="GPU"):
        fp8q.grouped_wgrad(c, s, c, s, torch.zeros(2, dtype=torch.int32))


def test_sort_numbers_that_do_not_fit_are_refused_before_the_call(monkeypatch):
    """ctypes keeps the low bits of a number that does not fit: none gets that far."""
    class Lib:
        @staticmethod
        def fp8q_moe_sort_workspace(*_):
            raise AssertionError("called")

    monkeypatch.setattr(fp8q, "_lib", Lib)
    monkeypatch.setattr(fp8q, "_rows_of", lambda t, name, dtypes: (2, 2, 2, 4096))
    experts = torch.zeros((2, 2), dtype=torch.int32)
    for bad in (dict(first=1 << 64), dict(first=(1 << 64) + 3), dict(first=1 << 31), dict(first=-1), dict(align=1 << 31), dict(align=1 << 32),
                dict(align=0), dict(rows_cap=-1)):
        with pytest.raises(ValueError):
            fp8q.moe_sort(experts, 4, **bad)
    for hosted in (-1, 1 << 31, (1 << 32) + 4):
        with pytest.raises(ValueError):
            fp8q.moe_sort(experts, hosted)


def test_binding_refuses_what_is_no_tensor(monkeypatch):
    """Lists in the place of any tensor, next to operands that pass, are a TypeError that names the argument."""
    def rows_of(t, name, dtypes, checked=fp8q._rows_of):
        return (*t.shape, t.shape[1], 4096) if isinstance(t, torch.Tensor) else checked(t, name, dtypes)

    monkeypatch.setattr(fp8q, "_rows_of", rows_of)
    y, rows, w = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    c, s, off = torch.zeros((4, 128), dtype=torch.uint8), torch.zeros((4, 1)), torch.zeros(2, dtype=torch.int32)
    for name, call in (("row_of", lambda: fp8q.moe_combine(y, rows.tolist())), ("weights", lambda: fp8q.moe_combine(y, rows, w.tolist())),
                       ("out", lambda: fp8q.moe_combine(y, rows, out=y.tolist())),
                       ("out", lambda: fp8q.moe_combine(y, rows, out=y.tolist(), out_dtype=torch.float32)),
                       ("y", lambda: fp8q.moe_combine(y.tolist(), rows)), ("experts", lambda: fp8q.moe_sort(rows.tolist(), 4)),
                       ("dout", lambda: fp8q.moe_combine_backward(y.tolist(), y, rows)),
                       ("row_of", lambda: fp8q.moe_combine_backward(y, y, rows.tolist())),
                       ("token", lambda: fp8q.moe_combine_backward(y, y, rows, w, off.tolist())),
                       ("dy", lambda: fp8q.swiglu_backward(y, y[:, :4].tolist())),
                       ("x_scales", lambda: fp8q.swiglu_backward(torch.zeros((4, 256)), torch.zeros((4, 128)), x_scales=s.tolist())),
                       ("offsets", lambda: fp8q.grouped_wgrad(c, s, c, s, off.tolist()))):
        with pytest.raises(TypeError, match=name):
            call()


def test_calls_run_on_the_tensors_own_device(monkeypatch):
    """With another device current the call is made under the tensors' device and on that device's stream."""
    seen, current = [], [0]

    class On:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            current.append(self.dev.index)

        def __exit__(self, *_):
            current.pop()

    class Lib:
        @staticmethod
        def fp8q_moe_combine(*args):
            seen.append((current[-1], args))
            return 0

    monkeypatch.setattr(fp8q, "_lib", Lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(fp8q, "_raw_stream", lambda dev: 1000 + dev.index)
    fp8q._call(torch.device("cuda:0"), "fp8q_moe_combine", 7)
    fp8q._call(torch.device("cuda:1"), "fp8q_moe_combine", 8)
    assert seen == [(0, (7, 1000)), (1, (8, 1001))] and current == [0]


def test_host_code_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")):
        pytest.skip("g++ or the HIP headers are not available")
    exe = str(tmp_path / "host_moe_abi_check")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE,
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(CSRC, "fp8q_moe_api.cpp"), os.path.join(ROOT, "tests", "host_moe_abi_check.cpp"), "-o", exe]
    build = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "host MoE ABI checks passed" in run.stdout
