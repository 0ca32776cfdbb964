"""The launches that calls of the library make, on a machine without a GPU.

launches(calls): for each call, (entry point's name, arguments behind the handle and before the stream), the kernel's
name and its grid and block.  A child process makes the calls, on a library whose launches launch_recorder.c
records.  shape() names the kernels of the grouped and the MXFP4 products shortly; tiles_of_rows() and tiles_of_sums() tell
what the 256 x 256 kernel computes in a launch."""
import json
import os
import re
import shutil
import subprocess
import sys
import tempfile

import pytest

import lds_staged_matrix_amd as lsm

HERE = os.path.dirname(os.path.abspath(__file__))
CUS = 256


def launches(calls):
    if shutil.which("gcc") is None or shutil.which("c++filt") is None:
        pytest.skip("no gcc or c++filt")
    if not os.path.exists(lsm.library_path()):
        from lds_staged_matrix_amd import build
        build.build()
    with tempfile.TemporaryDirectory() as d:
        recorder = os.path.join(d, "launch_recorder.so")
        subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-I", "/opt/rocm/include", os.path.join(HERE, "launch_recorder.c"),
                        "-o", recorder], check=True)
        out = subprocess.run([sys.executable, os.path.abspath(__file__), recorder], input=json.dumps(calls), check=True,
                             capture_output=True, text=True, env=dict(os.environ, PYTHONPATH=os.path.dirname(HERE))).stdout
    made = json.loads(out)
    names = subprocess.run(["c++filt"], input="\n".join(m[0] for m in made), check=True, capture_output=True,
                           text=True).stdout.splitlines()
    return [(n, g, b) for n, (_, g, b) in zip(names, made)]


def shape(name):
    """Of a kernel's name: "256x256", "tile 64x128, 3 stages, K by 2" or "stream 16x64 of 4"."""
    if "lds_gemm_tile256_kernel" in name:
        return "256x256"
    m = re.search(r"lds_gemm_tile_kernel<lsm::TileShape<(\d+), (\d+), \d+, \d+, (\d+), (\d+)>", name)
    if m:
        return f"tile {m[1]}x{m[2]}, {m[3]} stages" + (f", K by {m[4]}" if m[4] != "1" else "")
    m = re.search(r"lds_gemm_stream_kernel<lsm::StreamShape<(\d+), (\d+), (\d+),", name)
    return f"stream {m[1]}x{m[2]} of {m[3]}"


# ------------------------------------------------- the 256 x 256 kernel's tiles

def cdiv(a, b):
    return -(-a // b)


def xcd_logical_id(bid, n):
    return (bid & 7) * (n >> 3) + min(bid & 7, n & 7) + (bid >> 3)


def tile_coords(lid, tiles_m, tiles_n, group_m=8):
    first = lid // (group_m * tiles_n) * group_m
    gm, at = min(tiles_m - first, group_m), lid % (group_m * tiles_n)
    return first + at % gm, at // gm


def parts_of(total, most):
    """(tiles that stay whole, parts of each other one)."""
    rest = total % CUS
    return total - rest, 4 if most == 4 and 4 * rest <= CUS else 2 if 2 * rest <= CUS else 1


def _form(rows, height, most):
    rows = min(rows, height)
    return 256 if rows > 128 else 128 if rows > 64 or most == 2 else 64


def tiles_of_rows(spans, N, align):
    """[(rows of the tile's form: 256, 128 or 64; parts that the tile was cut into)] of every workgroup that computes,
    for groups of rows at `spans`; one product is one group, from row 0."""
    tiles_n, per = cdiv(N, 256), [cdiv(l - f + f % align, 256) if l > f else 0 for f, l in spans]
    total, out = sum(per) * tiles_n, []
    whole, parts = parts_of(total, 4)
    for tile in range(total):
        n = 1 if tile < whole else parts
        lid, g = xcd_logical_id(tile, total), 0
        while lid >= per[g] * tiles_n:
            lid -= per[g] * tiles_n
            g += 1
        tm, _ = tile_coords(lid, per[g], tiles_n)
        for sub in range(n):
            first = spans[g][0] - spans[g][0] % align + 256 * tm + sub * 256 // n
            if first < spans[g][1]:
                out.append((_form(spans[g][1] - first, 256 // n, 4), n))
    return out


def tiles_of_sums(groups, M, N):
    """The same of the matrices' gradient."""
    tiles_m, tiles_n, out = cdiv(M, 256), cdiv(N, 256), []
    total = groups * tiles_m * tiles_n
    whole, parts = parts_of(total, 2)
    for tile in range(total):
        n = 1 if tile < whole else parts
        tm, _ = tile_coords(xcd_logical_id(tile % (tiles_m * tiles_n), tiles_m * tiles_n), tiles_m, tiles_n)
        for sub in range(n):
            first = 256 * tm + sub * 256 // n
            if first < M:
                out.append((_form(M - first, 256 // n, 2), n))
    return out


def _child(recorder):
    import ctypes
    rec = ctypes.CDLL(recorder, ctypes.RTLD_GLOBAL)
    rec.recorded_kernel.restype = ctypes.c_char_p
    lib = lsm.Library(lsm.library_path())
    device = ctypes.c_int(0)                       # a handle is where its device's number stands
    handle, made = ctypes.cast(ctypes.pointer(device), ctypes.c_void_p), []
    for name, args in json.load(sys.stdin):
        status = getattr(lib, name)(handle, *args)
        if status != lsm.GEMM_OK:
            raise SystemExit(f"{name}{tuple(args)}: status {status}")
        made.append((rec.recorded_kernel().decode(), rec.recorded_grid(), rec.recorded_block()))
    print(json.dumps(made))


if __name__ == "__main__":
    _child(sys.argv[1])
