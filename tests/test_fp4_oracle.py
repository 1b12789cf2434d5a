"""CPU: the 4-bit page format's plain definition (oracle/fp4.py) pinned by
hand-picked values, and the library's own layout functions
(csrc/sp_fp4.cuh, compiled for the host) against it."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import fp4

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "..", "head_aware_paged_gb300", "csrc")


def _row(*head):
    return np.array(list(head) + [0.0] * (16 - len(head)))


def test_hand_picked_codes():
    # amax 6 -> scale 1 (code 15 << 3); every e2m1 value and its negative
    x = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6.0])
    code, sc = fp4.quantize(x)
    assert sc.tolist() == [15 << 3]
    assert code.tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 0, 9, 10, 11, 12, 13, 14, 15]
    # ties go to the even code: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    code, _ = fp4.quantize(_row(6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5))
    assert code[1:8].tolist() == [0, 2, 2, 4, 4, 6, 6]
    # scale ties: 6 * (1 + 1/16) lies between 1 and 1 + 1/8 -> the even 1; 6 * (1 + 3/16) -> 1 + 1/4
    assert fp4.quantize(_row(6 * 1.0625))[1].tolist() == [15 << 3]
    assert fp4.quantize(_row(6 * 1.1875))[1].tolist() == [(15 << 3) + 2]
    # saturation and zero
    code, sc = fp4.quantize(_row(1e9, -1e9, 3.0))
    assert sc.tolist() == [226] and code[:3].tolist() == [7, 15, 0]
    assert fp4.quantize(_row(6 * 2.0 ** -19))[1].tolist() == [0]
    assert fp4.stored(_row(6 * 2.0 ** -19)).tolist() == [0.0] * 16


def test_half_step_error_bound():
    """Each element is within half a step of its block's grid, or clipped where
    the rounded scale fell below amax / 6 (by 1/16 at most)."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((200, 128)) * np.exp2(rng.integers(-10, 10, (200, 1)))
    code, sc = fp4.quantize(x)
    s = np.repeat(fp4.SCALES[sc], 16, axis=1)
    err = np.abs(fp4.dequantize(code, sc) - x)
    y = np.abs(x) / s
    step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    assert np.all((err <= step / 2 * s * (1 + 1e-12)) | (y > 6))
    assert np.all(y <= 6 * (1 + 1 / 16))


def test_scale_rounding_error():
    a = np.exp(np.linspace(np.log(1e-3), np.log(6e4), 5000))
    sc = fp4.quantize(np.stack([a] + [0 * a] * 15, -1))[1][:, 0]
    rel = np.abs(fp4.SCALES[sc] / (a / 6) - 1)
    assert rel.max() <= 2.0 ** -4 + 1e-12        # half a step of 3 mantissa bits


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("fp4")
    src = d / "layout.cpp"
    src.write_text('#include "sp_fp4.cuh"\nusing namespace sp;\nextern "C" int place(int what, int s, int b) {\n'
                   "return what == 0 ? fp4_k_code(s, b) : what == 1 ? fp4_k_scale(s, b) :\n"
                   "what == 2 ? fp4_v_code(s, b) : fp4_v_scale(s, b); }\n"
                   'extern "C" long long group(long long page, int slot, int P) { return fp4_group_off(page, slot, P); }\n')
    so = str(d / "layout.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.group.restype = ctypes.c_longlong
    lib.group.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


def test_layout_covers_a_group_once_and_matches(layout):
    for code, scale, value in ((0, 1, False), (2, 3, True)):
        used = np.zeros(1152, int)
        rng = np.random.default_rng(5)
        codes, scales = rng.integers(0, 16, (16, 128)), rng.integers(0, 227, (16, 8))
        group = np.zeros(1152, np.uint8)
        for s in range(16):
            for b in range(8):
                at = layout.place(code, s, b)
                used[at:at + 8] += 1
                c = codes[s, 16 * b:16 * b + 16]
                group[at:at + 8] = c[0::2] | (c[1::2] << 4)
                used[layout.place(scale, s, b)] += 1
                group[layout.place(scale, s, b)] = scales[s, b]
        assert (used == 1).all()
        for s in range(16):
            c, sc = fp4.read_row(group, s, value)
            assert (c == codes[s]).all() and (sc == scales[s]).all()


def test_group_offsets_pass_32_bits(layout):
    assert layout.group(0, 17, 64) == 1152
    assert layout.group(3, 0, 16) == 3 * 1152
    assert layout.group(1 << 25, 33, 64) == (1 << 25) * 64 * 72 + 2 * 1152
