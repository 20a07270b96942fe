"""The choice of a bf16 product's kernel (csrc/moe_gemm_bf16_choice.h), compiled by itself for the
host."""
import ctypes
import os
import subprocess

import pytest

import routed_grouped_gemm_topk_amd as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")
KERNELS = ["any 64x64", "any 128x128", "any stream 16x16", "stream 16x16", "stream 16x32", "32x64",
           "64x64", "64x128", "128x128", "128x256", "192x192", "192x256", "256x256"]
LAYOUTS = {"nt": (True, True), "nn": (True, False), "tn": (False, False)}
SHIM = """
#include "moe_gemm_bf16_choice.h"
using namespace moe::gb;
extern "C" int kernels() { return kKernels; }
extern "C" int choose_(int m, int n, int k, bool ka, bool kb, int cus) {
  return choose(m, n, k, ka, kb, cus);
}
extern "C" int64_t tiles(int kernel, int m, int n) { return tiles_of((Kernel)kernel, m, n); }
extern "C" int64_t whole(int64_t tiles, int cus) { return whole_tiles(tiles, cus); }
extern "C" void size_of(int kernel, int* s) {
  const TileSize& t = kTileSize[kernel];
  s[0] = t.bm, s[1] = t.bn, s[2] = t.threads;
}
"""


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    src, out = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    "-o", str(out), str(src)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.choose_.argtypes = [ctypes.c_int] * 3 + [ctypes.c_bool] * 2 + [ctypes.c_int]
    lib.tiles.restype = lib.whole.restype = ctypes.c_int64
    lib.whole.argtypes = [ctypes.c_int64, ctypes.c_int]
    assert lib.kernels() == len(KERNELS)
    return lib


def size_of(choice, kernel):
    s = (ctypes.c_int * 3)()
    choice.size_of(kernel, s)
    return list(s)


def accepted(m, n, k):
    """Whether the library takes these sizes (it looks at them before the output's type, which is
    wrong here, so that no call goes through)."""
    ok = ctypes.c_void_p(4096)
    status = moe.load().moe_gemm_bf16(m, n, k, 0, ok, ok, None, 0, None, None, ok, 99, None)
    assert status in (moe.MOE_ERR_SHAPE, moe.MOE_ERR_DTYPE)
    return status == moe.MOE_ERR_DTYPE


# the largest products that are accepted, square and narrow, of any k
LARGEST = [(2 ** 24, 8192), (8192, 2 ** 24), (2 ** 22, 2 ** 15), (2 ** 18, 2 ** 19),
           (2 ** 24 - 8, 8184), (18336, 7475544), (2423784, 56584), (2 ** 24, 16), (16, 2 ** 24),
           (1, 2 ** 24), (2 ** 24, 1), (65, 2 ** 24), (2 ** 23, 128), (128, 2 ** 23), (2 ** 23, 8)]


@pytest.mark.parametrize("k", [8, 64, 512, 4096, 2 ** 21, 2 ** 24, 7, 2 ** 24 - 1])
@pytest.mark.parametrize("m,n", LARGEST)
def test_launches_count_their_threads_in_32_bits(choice, m, n, k):
    assert accepted(m, n, k)
    for cus in (8, 64, 256, 304):
        for name, (ka, kb) in LAYOUTS.items():
            kernel = choice.choose_(m, n, k, ka, kb, cus)
            bm, bn, threads = size_of(choice, kernel)
            tiles = choice.tiles(kernel, m, n)
            assert tiles == -(-m // bm) * -(-n // bn)
            groups = -(-tiles // 8) * 8
            if kernel < 2:
                groups = min(tiles, 2 ** 21)               # the others are run by striding
            elif kernel == 2:
                groups = tiles
            elif KERNELS[kernel] == "256x256":             # whole tiles and halves
                w = choice.whole(tiles, cus)
                assert tiles < 2 ** 30
                groups = -(-w // 8) * 8 + -(-2 * (tiles - w) // 8) * 8
            assert groups * threads < 2 ** 32, (KERNELS[kernel], name, cus)


def test_offsets_of_one_tile_stay_within_31_bits(choice):
    """What the kernels of 16-byte loads address through one descriptor: a tile's rows over all of
    k, or a slice of 64 values of k over a whole row."""
    for m, n, k in [(256, 256, 2 ** 21), (256, 256, 2 ** 21 + 8), (2 ** 23, 64, 64),
                    (2 ** 23 + 8, 64, 64), (64, 2 ** 23, 64), (64, 2 ** 23 + 8, 64),
                    (2 ** 24, 8, 8), (8, 2 ** 24, 2 ** 24)]:
        for name, (ka, kb) in LAYOUTS.items():
            kernel = choice.choose_(m, n, k, ka, kb, 256)
            bm, bn, _ = size_of(choice, kernel)
            a = bm * k if ka else 64 * m
            b = bn * k if kb else 64 * n
            assert kernel < 3 or (max(a, b) * 2 < 2 ** 31), (m, n, k, name, KERNELS[kernel])


def test_just_past_the_largest_is_refused():
    for m, n, k in [(2 ** 24, 8193, 64), (2 ** 18 + 1, 2 ** 19, 64), (2 ** 24 + 1, 1, 64),
                    (1, 2 ** 24 + 1, 64), (1, 1, 2 ** 24 + 1)]:
        assert not accepted(m, n, k)


def test_rows_that_are_no_whole_blocks_take_the_kernels_of_any_alignment(choice):
    for m, n, k in [(7, 8, 8), (8, 7, 8), (8, 8, 7), (2047, 2047, 2047), (1000, 1001, 1000)]:
        for ka, kb in LAYOUTS.values():
            whole = (k if ka else m) % 8 == 0 and (k if kb else n) % 8 == 0
            assert (choice.choose_(m, n, k, ka, kb, 256) >= 3) == whole


def test_every_kernel_is_run_by_the_gpu_tests(choice):
    """The shapes of test_gpu_gemm_bf16_tiles reach every kernel that the choice can give in every
    layout, with rows of c on 16 bytes, on an even and on an odd number of values (where b's layout
    allows it), with ragged tiles, a number of slices that is no multiple of the groups of waves
    along k, and more steps than stages, so that every stage is filled again."""
    from test_gpu_gemm_bf16_tiles import TILES, UNITS
    groups = [4, 1, 16, 8, 8, 2, 2, 1, 1, 1, 1, 1, 1]          # of waves that cut k
    stages = [2, 2, 4, 4, 3, 4, 3, 3, 3, 3, 3, 4, 3]
    none = {"nt": set(), "nn": {2, 3, 4}, "tn": {2, 3, 4, 5}}    # kernels that the layout has not
    hit = set()
    for m, n, k, name in TILES:
        q = choice.choose_(m, n, k, *LAYOUTS[name], UNITS)
        bm, bn, _ = size_of(choice, q)
        slices = -(-k // 64)
        if m % bm and n % bn and k % 64 and -(-slices // groups[q]) > stages[q] + 1 and (
                groups[q] == 1 or slices % groups[q]):
            hit.add((q, name, "odd" if n % 2 else "16 bytes" if n % 8 == 0 else "even"))
    for q, kernel in enumerate(KERNELS):
        for name, (ka, kb) in LAYOUTS.items():
            if q in none[name]:
                continue
            for rows in ("odd", "16 bytes", "even") if kb or q < 3 else ("16 bytes",):
                assert (q, name, rows) in hit, (kernel, name, rows)


def test_the_halves_of_a_last_round_are_run_by_the_gpu_tests(choice):
    from test_gpu_gemm_bf16_tiles import HALVES, UNITS
    second = set()
    for m, n, k, name in HALVES:
        assert choice.choose_(m, n, k, *LAYOUTS[name], UNITS) == KERNELS.index("256x256")
        tiles = choice.tiles(KERNELS.index("256x256"), m, n)
        assert choice.whole(tiles, UNITS) < tiles
        second.add((name, m % 256 > 128))
    assert second == {(name, s) for name in LAYOUTS for s in (False, True)}
