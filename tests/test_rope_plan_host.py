"""Host-side check (no GPU) of the append's ring layout: csrc/rope_plan.h, compiled for
the CPU, over the head counts, widths and rotary sizes of ordinary models."""
import ctypes
import os
import subprocess

import pytest

from s3d8_a8_linear_gb300 import _build


class Ring(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("threads", "ctas", "stages", "stage")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("plan")
    src, lib = out / "plan.cpp", out / "plan.so"
    names = ("kRopeThreads", "kRingStages", "kRingBytes", "kRingSm", "kRingFixed")
    src.write_text('#include "rope_plan.h"\n'
                   'extern "C" s3d8::RopeRing ring(int h, int d, int r, int l) { return s3d8::rope_ring(h, d, r, l); }\n'
                   'extern "C" int whole(int h, long long s, int d) { return s3d8::rope_whole(h, s, d); }\n' +
                   "".join(f'extern "C" int {n}() {{ return s3d8::{n}; }}\n' for n in names))
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", _build.CSRC, str(src), "-o", str(lib)],
                   check=True)
    L = ctypes.CDLL(os.fspath(lib))
    L.ring.restype = Ring
    L.whole.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int]
    return L, {n: getattr(L, n)() for n in names}


@pytest.mark.parametrize("dim", range(16, 257, 16))
def test_the_ring_stays_within_what_a_launch_is_allowed(lib, dim):
    L, k = lib
    log_lanes = (dim // 16 - 1).bit_length()
    fitted = 0
    for heads in range(3, 481):
        for rotary in range(0, dim + 1, 16):
            r = L.ring(heads, dim, rotary, log_lanes)
            assert r.stage == heads * dim * 2 + rotary * 4
            if 3 * r.stage > k["kRingBytes"]:
                assert r.stages == 0
                continue
            fitted += 1
            where = (heads, dim, rotary, r.threads, r.ctas, r.stages)
            assert 3 <= r.stages <= k["kRingStages"] and r.ctas >= 1, where
            assert r.stages * r.stage <= k["kRingBytes"], where
            assert r.ctas * (r.stages * r.stage + k["kRingFixed"]) <= k["kRingSm"], where
            assert r.threads % 32 == 0 and 32 <= r.threads <= k["kRopeThreads"], where
    assert fitted


@pytest.mark.parametrize("heads,dim,rotary,want", [
    (48, 128, 128, (128, 5, 3)),      # 32 / 8 heads of 128, the measured case
    (16, 64, 64, (32, 12, 7)),
    (96, 96, 96, (256, 2, 5)),        # 32 / 32 heads of 96: six stages would pass the allowance
    (112, 128, 0, (256, 2, 3)),       # 96 / 8 of 128 without rotation
])
def test_the_ring_of_some_models(lib, heads, dim, rotary, want):
    r = lib[0].ring(heads, dim, rotary, (dim // 16 - 1).bit_length())
    assert (r.threads, r.ctas, r.stages) == want


def test_heads_lie_in_one_piece(lib):
    whole = lib[0].whole
    assert whole(8, 128, 128) and not whole(8, 256, 128) and not whole(2, 0, 64) and not whole(2, 1 << 40, 64)
    for stride in (0, 64, 128, 1 << 40):      # one head is one piece, whatever its stride says
        assert whole(1, stride, 64)
