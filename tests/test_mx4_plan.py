"""Which kernel the 4-bit products take: the sizes that the GPU tests list for a kernel do go to it.  The choice
(csrc/qamw_mx4_plan.hpp) is host code and is compiled here by itself."""
import ctypes
import subprocess

import pytest

import test_gpu_mx4
import weight_quantization_codec_amd as q
from weight_quantization_codec_amd import _build

TILES = [(256, 256), (128, 256), (128, 128), (64, 256), (32, 256), (64, 64)]
FEW = len(TILES)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text("""#include "qamw_mx4_plan.hpp"
static_assert(qamw::kTileKinds4 == %d && qamw::kThin4 == %d && qamw::kMaxTiles4 == 1 << 23, "");
extern "C" void plan(int M, int N, int groups, int* out) {
    const qamw::Plan4 p = qamw::plan4(M, N, groups);
    out[0] = p.tile, out[1] = p.splits;
}
extern "C" int grouped(int rows, int experts, int N, int groups) { return qamw::plan4_grouped(rows, experts, N, groups); }
extern "C" int tile_rows(int i, int of_weights) { return of_weights ? qamw::kTiles4[i].bn : qamw::kTiles4[i].bm; }
""" % (len(TILES), FEW))
    so = str(d / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-O1", "-shared", "-fPIC", "-I", _build.CSRC,
                    str(d / "plan.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    assert [(lib.tile_rows(i, 0), lib.tile_rows(i, 1)) for i in range(len(TILES))] == TILES

    class Plan:
        grouped = staticmethod(lib.grouped)

        @staticmethod
        def product(M, N, groups):
            out = (ctypes.c_int * 2)()
            lib.plan(M, N, groups, out)
            return out[0], out[1]
    return Plan


def test_every_kernel_is_tested(plan):
    sizes = test_gpu_mx4.KERNELS
    got = [plan.product(M, N, q.mx4_groups(K)) for M, N, K in sizes]
    assert [t for t, _ in got] == [0] * 5 + [1] * 3 + [2] * 5 + [3] * 4 + [4] * 3 + [5] * 6 + [FEW] * 6
    for tile in (2, 3, 4, 5):   # k whole, and in parts
        parts = [s for t, s in got if t == tile]
        assert min(parts) == 1 and max(parts) > 1, tile
    # several tiles a workgroup, of one group of columns and of more
    count = [-(-M // 256) * -(-N // 256) for (M, N, _), (t, _) in zip(sizes, got) if t == 0]
    walks = [q.mx4_groups(K) for (_, _, K), n in zip(sizes, count) if n > 256]
    assert 1 in walks and max(walks) > 2 and min(count) < 256
    few = [m for (m, _, _), (t, _) in zip(sizes, got) if t == FEW]
    assert {8 if m <= 8 else 16 if m <= 16 else 32 for m in few} == {8, 16, 32}


def test_every_kernel_of_groups_is_tested(plan):
    got = [plan.grouped(sum(sizes), len(sizes), N, q.mx4_groups(K)) for _, sizes, N, K in test_gpu_mx4.GROUP_KERNELS]
    assert got == [0] * 3 + [1] * 2 + [3] * 2 + [4] * 2 + [FEW] * 2 + [FEW + 1]


def test_workspaces_follow_the_plan(plan):
    """The library chooses as this header does: 32-bit sums of every part, rows of whole 64 columns."""
    for M, N, K in test_gpu_mx4.KERNELS + test_gpu_mx4.SMALL:
        _, parts = plan.product(M, N, q.mx4_groups(K))
        assert q.gemm4_workspace(M, N, q.mx4_groups(K)) == (parts * M * ((N + 63) // 64 * 64) * 4 if parts > 1 else 0), (M, N, K)


def test_grids_of_the_largest_products(plan):
    """A launch has at most 2^23 workgroups of 256 threads, at the limits of M, d_out, M d_out and experts too."""
    top, out = q.mx4.GEMM4_MAX_ROWS, q.mx4.GEMM4_MAX_OUT
    for groups in (1, 2, 20, q.mx4.MX4_MAX_COLS // 256):
        for a in (1, 2, 31, 32, 33, 64, 65, 257, 4097, out // top - 1, out // top, 1 << 19):
            for M, N in ((a, min(top, out // a)), (min(top, out // a), a)):
                tile, parts = plan.product(M, N, groups)
                if tile < FEW:
                    bm, bn = TILES[tile]
                    assert -(-M // bm) * -(-N // bn) * parts <= 1 << 23, (M, N, groups)
                else:
                    assert M <= 32
                for experts in (1, 3, 64, 1000, q.mx4.GEMM4_MAX_EXPERTS):
                    if experts * N > q.mx4.GEMM4_MAX_EXPERT_ROWS:
                        continue
                    kind = plan.grouped(M, experts, N, groups)
                    bm, bn = TILES[kind] if kind < FEW else (8 * (1 + kind - FEW), 32)
                    assert (M // bm + min(experts, M)) * -(-N // bn) <= 1 << 23, (M, N, groups, experts, kind)

