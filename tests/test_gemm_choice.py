"""The choice of an e4m3 product's kernel (csrc/moe_gemm_e4m3_choice.h), compiled by itself for the
host."""
import ctypes
import os
import subprocess

import pytest

import routed_grouped_gemm_topk_amd as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")
KERNELS = ["16x16 stream", "16x32 stream", "16x64", "32x64", "64x64", "64x128", "128x128",
           "128x128 ring of 3", "128x256", "192x256", "256x256"]
VARIANTS = [(brow, f32) for brow in (False, True) for f32 in (False, True)]
SHIM = """
#include "moe_gemm_e4m3_choice.h"
using namespace moe::q8;
extern "C" int kernels() { return kDenseKernels; }
extern "C" int choose(int m, int n, int k, bool brow, bool f32, int cus) {
  return choose_dense(m, n, k, brow, f32, cus);
}
extern "C" int64_t tiles(int kernel, int m, int n) { return dense_tiles((DenseKernel)kernel, m, n); }
extern "C" int threads(int kernel) { return kDenseSize[kernel].threads; }
extern "C" int grouped_kernels() { return kGroupedKernels; }
extern "C" int choose_grouped_(int bm, int64_t rows, int64_t tiles, int n, bool f32, int cus) {
  return choose_grouped(bm, rows, tiles, n, f32, cus);
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
    lib.choose.argtypes = [ctypes.c_int] * 3 + [ctypes.c_bool] * 2 + [ctypes.c_int]
    lib.tiles.restype = ctypes.c_int64
    lib.choose_grouped_.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 2 + [ctypes.c_int, ctypes.c_bool,
                                                                           ctypes.c_int]
    assert lib.kernels() == len(KERNELS)
    return lib


def accepted(m, n, k):
    """Whether the library takes these sizes (it looks at them before the output's type, which is
    wrong here, so that no call goes through)."""
    ok = ctypes.c_void_p(4096)
    status = moe.load().moe_gemm_e4m3(m, n, k, ok, ok, ok, ok, 128, ok, 99, None)
    assert status in (moe.MOE_ERR_SHAPE, moe.MOE_ERR_DTYPE)
    return status == moe.MOE_ERR_DTYPE


# the largest products that are accepted, square and narrow, of any K
LARGEST = [(2 ** 24, 8192), (8192, 2 ** 24), (2 ** 22, 2 ** 15), (2 ** 18, 2 ** 19),
           (2 ** 24 - 7, 8191), (18334, 7475545), (2423788, 56589), (2 ** 24, 17), (17, 2 ** 24),
           (1, 2 ** 24), (2 ** 24, 1), (65, 2 ** 24), (193, 2 ** 24)]


@pytest.mark.parametrize("k", [128, 256, 384, 512, 4096, 2 ** 22])
@pytest.mark.parametrize("m,n", LARGEST)
def test_launches_count_their_threads_in_32_bits(choice, m, n, k):
    assert accepted(m, n, k)
    for cus in (8, 64, 256, 304):
        for brow, f32 in VARIANTS:
            kernel = choice.choose(m, n, k, brow, f32, cus)
            # rounded up to whole chunks of 32 tiles for each of 8 XCDs
            groups = -(-choice.tiles(kernel, m, n) // 256) * 256
            assert groups * choice.threads(kernel) < 2 ** 32, (KERNELS[kernel], brow, f32, cus)


def test_just_past_the_largest_is_refused():
    for m, n in [(2 ** 24, 8193), (2 ** 18 + 1, 2 ** 19), (2 ** 24 + 1, 1)]:
        assert not accepted(m, n, 128)


def test_every_kernel_is_run_by_the_gpu_tests(choice):
    """The shapes of test_gpu_gemm_tiles reach every kernel that the choice can give, in each form:
    scales of b by block and by row, both result types, rows of c on 16 bytes, on an even and on an
    odd number of values; with ragged tiles, a number of slices that is no multiple of the groups of
    waves along k, and more steps than stages, so that every stage is filled again."""
    from test_gpu_gemm_tiles import TILES, UNITS
    bm = [16, 16, 16, 32, 64, 64, 128, 128, 128, 192, 256]
    bn = [16, 32, 64, 64, 64, 128, 128, 128, 256, 256, 256]
    groups = [8, 8, 4, 2, 2, 1, 1, 1, 1, 1, 1]             # of waves that cut k
    stages = [2, 2, 3, 3, 3, 3, 2, 3, 3, 2, 2]             # streams: slices in flight, 2 a step
    only_bf16, only_blocks = {7, 9, 10}, {10}
    hit = set()
    for m, n, k in TILES:
        for brow, f32 in VARIANTS:
            q = choice.choose(m, n, k, brow, f32, UNITS)
            slices = k // 128
            ragged = q < 2 or (m % bm[q] and n % bn[q])
            if ragged and -(-slices // groups[q]) > stages[q] + 1 and (
                    groups[q] == 1 or slices % groups[q]):
                hit.add((q, brow, f32, "odd" if n % 2 else "16 bytes" if n % 8 == 0 else "even"))
    for q, name in enumerate(KERNELS):
        for brow, f32 in VARIANTS:
            if (f32 and q in only_bf16) or (brow and q in only_blocks):
                continue
            for rows in ("odd", "16 bytes", "even"):
                assert (q, brow, f32, rows) in hit, (name, brow, f32, rows)


def test_the_halves_of_a_last_round_are_run_by_the_gpu_tests(choice):
    from test_gpu_gemm_tiles import HALVES, UNITS
    second = set()
    for m, n, k in HALVES:
        assert choice.choose(m, n, k, False, False, UNITS) == KERNELS.index("256x256")
        tiles = choice.tiles(KERNELS.index("256x256"), m, n)
        assert tiles > UNITS and 0 < tiles % UNITS <= UNITS // 2      # run_large's rule
        second.add(m % 256 > 128)
    assert second == {False, True}


def test_every_grouped_kernel_is_run_by_the_gpu_tests(choice):
    """The same for the grouped product, each kernel with both result types, more steps than stages
    and ragged columns."""
    import test_gpu_gemm_tiles as small
    import test_gpu_large_outputs as large
    names = ["16x64", "16x128", "32x64", "32x128", "64x64", "64x128", "64x256", "64x256 past",
             "128x128", "128x256", "128x256 past"]
    bn = [64, 128, 64, 128, 64, 128, 256, 256, 128, 256, 256]
    groups = [4, 1, 2, 1, 2, 1, 1, 1, 1, 1, 1]
    stages = [3, 3, 3, 3, 3, 3, 3, 3, 2, 3, 3]
    assert choice.grouped_kernels() == len(names)
    hit = set()
    for T, E, k, bm, n, kk in small.GROUPED + large.PAST:
        p = moe.make_problem(T, 128, 128, E, k, "bf16", "e4m3", bm)
        for f32 in (False, True):
            q = choice.choose_grouped_(bm, moe.moe_max_padded_slots(p), moe.moe_max_tiles(p), n, f32,
                                      small.UNITS)
            if n % bn[q] and -(-(kk // 128) // groups[q]) > stages[q] + 1:
                hit.add((names[q], f32))
    assert hit == {(name, f32) for name in names for f32 in (False, True)}
