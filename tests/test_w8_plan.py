"""Which kernel the 8-bit product takes: the sizes that the GPU tests list for a kernel do go to it.  The choice
(csrc/qamw_w8_plan.hpp) is host code and is compiled here by itself."""
import ctypes
import os
import subprocess

import pytest

import test_gpu_w8
import test_gpu_w8_far
import test_gpu_w8_host
import weight_quantization_codec_amd as q
from weight_quantization_codec_amd import _build

TILES = [(256, 256), (256, 128), (128, 128), (128, 64), (64, 128), (64, 64)]
FEW = len(TILES)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text("""#include "qamw_w8_plan.hpp"
static_assert(qamw::kTileKinds == %d && qamw::kThin == %d, "");
extern "C" void plan(int M, int N, int K, int* out) {
    const qamw::Plan p = qamw::plan(M, N, K);
    out[0] = p.tile, out[1] = p.splits;
}
extern "C" int tile_rows(int i, int of_weights) { return of_weights ? qamw::kTiles[i].bn : qamw::kTiles[i].bm; }
""" % (len(TILES), FEW))
    so = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-shared", "-fPIC", "-I", _build.CSRC,
                    str(d / "plan.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    assert [(lib.tile_rows(i, 0), lib.tile_rows(i, 1)) for i in range(len(TILES))] == TILES

    def choose(M, N, K):
        out = (ctypes.c_int * 2)()
        lib.plan(M, N, K, out)
        return out[0], out[1]
    return choose


def _sizes(test):
    (mark,) = [m for m in test.pytestmark if m.name == "parametrize"]
    return mark.args[1]


def test_every_kernel_is_tested(plan):
    sizes = _sizes(test_gpu_w8.test_gemm8_every_kernel)
    got = [plan(*s) for s in sizes]
    assert [tile for tile, _ in got] == [0] * 2 + [1] * 4 + [2] * 4 + [3] * 4 + [4] * 4 + [5] * 4 + [FEW] * 5
    for tile in range(1, len(TILES)):   # k whole, and in parts
        parts = [s for t, s in got if t == tile]
        assert min(parts) == 1 and max(parts) > 1, tile
    # one size or more whose last step of k is not full, of each kind; and few rows at each of the kernel's widths
    for tile in range(len(TILES) + 1):
        assert any(k % 128 for (_, _, k), (t, _) in zip(sizes, got) if t == tile)
    few = [m for (m, _, _), (t, _) in zip(sizes, got) if t == FEW]
    assert {8 if m <= 8 else 16 if m <= 16 else 32 if m <= 32 else 64 for m in few} == {8, 16, 32, 64}


def test_far_products(plan):
    assert [plan(*s)[0] for s in test_gpu_w8_far.FAR_FEW] == [FEW] * len(test_gpu_w8_far.FAR_FEW)
    assert [plan(*s)[0] for s in test_gpu_w8_far.FAR_TILES] == [0] * len(test_gpu_w8_far.FAR_TILES)


def test_workspaces_follow_the_plan(plan):
    """The library chooses as this header does: 32-bit sums of every part, rows of whole 64 columns."""
    sizes = _sizes(test_gpu_w8.test_gemm8_every_kernel) + _sizes(test_gpu_w8.test_gemm8_large) + test_gpu_w8_host.PARTS
    for M, N, K in sizes:
        _, parts = plan(M, N, K)
        assert q.gemm8_workspace(M, N, K) == (parts * M * ((N + 63) // 64 * 64) * 4 if parts > 1 else 0), (M, N, K)
    assert all(plan(*s)[1] > 1 for s in test_gpu_w8_host.PARTS)


def test_grids_of_the_largest_products(plan):
    """A launch has at most 2^23 workgroups of 256 threads, at the limits of M, d_out and M d_out too."""
    top, out = q.w8.GEMM8_MAX_ROWS, q.w8.GEMM8_MAX_OUT
    for K in (1, 128, 5120, q.w8.GEMM8_MAX_COLS):
        for a in (1, 2, 64, 65, 257, 4097, out // top - 1, out // top, 1 << 19):
            for M, N in ((a, min(top, out // a)), (min(top, out // a), a)):
                tile, parts = plan(M, N, K)
                if tile < FEW:
                    bm, bn = TILES[tile]
                    assert -(-M // bm) * -(-N // bn) * parts <= 1 << 23, (M, N, K)
                else:
                    assert M <= 64
