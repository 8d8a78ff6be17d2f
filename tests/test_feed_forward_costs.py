"""The costs by which the feed-forward calls choose a kernel and its tiles stay costs over the whole range of sizes
(host code of csrc/feed_forward.cu, compiled once more with its two estimates exported)."""

import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="nvcc not available")

LAST = 2 ** 31 - 1024  # the largest d_in


@pytest.fixture(scope="module")
def costs(tmp_path_factory):
    from token_adapter_routing_gb300 import build
    build.build()
    out = tmp_path_factory.mktemp("costs")
    here = os.path.join(os.path.dirname(os.path.abspath(__file__)), "feed_forward_costs.cu")
    obj, path = str(out / "costs.o"), str(out / "libcosts.so")
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-c", here, "-o", obj], check=True)
    others = [os.path.join(build.BUILD, os.path.basename(s)[:-3] + ".o") for s in build.sources() if not s.endswith("feed_forward.cu")]
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-o", path, obj, *others], check=True)
    lib = ctypes.CDLL(path)
    for fn in (lib.pairs_cost, lib.few_cost):
        fn.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int]
        fn.restype = ctypes.c_int64
    return lib


@pytest.mark.parametrize("gated, fp8", [(0, 1), (1, 1), (1, 0)])
@pytest.mark.parametrize("N, d_out", [(1, 1), (33, 1), (4096, 4096), (2 ** 31 - 1024, 64)])
def test_costs_grow_with_the_input(costs, gated, fp8, N, d_out):
    """A K block costs the same however many there are: from 2^20 columns of x on, where it is nearly all, twice as many cost
    nearly twice as much, up to the last."""
    for fn, tiles in ((costs.pairs_cost, (128, 192, 256)), (costs.few_cost, (16, 32, 64, 128, 256))):
        for tile in tiles:
            last = fn(gated, fp8, N, 1 << 20, d_out, tile)
            assert last > 0
            for d_in in [1 << k for k in range(21, 31)]:
                cost = fn(gated, fp8, N, d_in, d_out, tile)
                assert 1.7 * last < cost <= 2.001 * last, (tile, d_in, last, cost)
                last = cost
            assert fn(gated, fp8, N, LAST, d_out, tile) > 1.9 * last


def test_a_tile_with_a_long_sum_splits_it(costs):
    """Where there is one tile, few tokens' kernel, which splits its sum over a cluster, costs less than the pairs'."""
    for d_in in (1 << 20, 1 << 26, 1 << 29, 1 << 30, LAST):
        for gated, fp8 in ((0, 1), (1, 1), (1, 0)):
            assert min(costs.few_cost(gated, fp8, 33, d_in, 64, t) for t in (32, 64)) < \
                min(costs.pairs_cost(gated, fp8, 33, d_in, 64, t) for t in (128, 192, 256))
