"""Host-side check (no GPU) of the arithmetic that decides which entries of a page call
find pages: csrc/page_room.h, compiled for the CPU, against Python's integers."""
import ctypes
import os
import subprocess

import pytest

from s3d8_a8_linear_gb300 import _build

MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def room(tmp_path_factory):
    out = tmp_path_factory.mktemp("room")
    src, lib = out / "room.cpp", out / "room.so"
    src.write_text('#include "page_room.h"\n'
                   'extern "C" int32_t rank(int64_t w) { return s3d8::page_rank(w); }\n'
                   'extern "C" int room(int32_t r, int32_t n, int32_t f) { return s3d8::page_room(r, n, f); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-shared", "-fPIC", "-I", _build.CSRC, str(src), "-o", str(lib)],
                   check=True)
    L = ctypes.CDLL(os.fspath(lib))
    L.rank.argtypes, L.rank.restype = [ctypes.c_int64], ctypes.c_int32
    L.room.argtypes = [ctypes.c_int32] * 3
    return L


@pytest.mark.parametrize("free", [0, 1, 7, 64, MAX - 4096])
@pytest.mark.parametrize("needs", [
    [3, 2 ** 30, 2 ** 30, 5, 0], [MAX, 1, 1, 0, 4], [2 ** 30] * 9 + [0, 1], [0, -1, 0, 7, 1], [MAX] * 5,
    [1] * 70, [MAX - 4096, 1, 0], [2 ** 31 - 1 - 7, 3, 2 ** 31 - 1, 3],
])
def test_an_entry_gets_pages_only_where_all_in_front_of_it_would(room, needs, free):
    wanted = 0
    for need in needs:
        want = need == 0 or (need > 0 and wanted + need <= free)
        assert room.room(room.rank(wanted), need, free) == int(want), (needs, need)
        wanted += max(need, 0)
