"""How rows of logits and of gradients are cut, on the host: the plans of the largest and smallest
sizes, compiled into a small program that prints them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_66_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "lp_stream.cuh"
int main()
{
    long long rows, V;
    int per_vec;
    while (std::scanf("%lld %lld %d", &rows, &V, &per_vec) == 3) {
        const int tiles = svl::most_tiles(static_cast<int>(V), per_vec);
        int warps;
        const svl::GradPlan g = svl::grad_plan_of(static_cast<int>(rows), tiles, &warps);
        std::printf("%d %d %d %d", tiles, g.pieces, g.piece, warps);
        for (int w : {4, 8, 16})
            for (int ragged = 0; ragged < 2; ++ragged) {
                const svl::Cut c = svl::cut_of(rows, tiles, w, ragged != 0);
                std::printf(" %d %d %d", c.whole, c.pieces, c.piece);
            }
        std::printf("\n");
    }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    d = tmp_path_factory.mktemp("plans")
    (d / "plans.cu").write_text(PROGRAM)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a",
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", os.path.join(CSRC, "logprobs"),
                    "-o", str(d / "plans"), str(d / "plans.cu")], check=True)

    def run(sizes):
        out = subprocess.run([str(d / "plans")], input="".join("%d %d %d\n" % s for s in sizes),
                             capture_output=True, text=True, check=True).stdout
        return [[int(x) for x in line.split()] for line in out.splitlines()]
    return run


def test_all_turns_are_somebodys(plans):
    top = 2 ** 31 - 1
    vocabularies = [1, 2, 7, 8, 9, 1023, 1024, 1025, 32000, 128256, 1 << 20, top - 8, top - 7, top - 3,
                    top - 2, top - 1, top]
    counts = [1, 2, 3, 40, 304, 1216, 1217, 2304, 4863, 4864, 5000, 65536, top - 1, top]
    sizes = [(rows, V, p) for rows in counts for V in vocabularies for p in (4, 8)]
    for (rows, V, p), (tiles, pieces, piece, warps, *cuts) in zip(sizes, plans(sizes), strict=True):
        # p - 1 elements may lie in front of a row
        assert tiles == -(-(-(-V // p) + 1) // 128) >= -(-(V + p - 1) // (128 * p))
        assert 1 <= warps <= 8 and 1 <= piece < 2 ** 31 and pieces >= 1
        assert pieces * piece >= tiles and pieces * rows < 2 ** 31
        for whole, n, each in zip(cuts[::3], cuts[1::3], cuts[2::3], strict=True):
            assert 0 <= whole <= rows and n >= 1 and n * each >= tiles
            assert whole + (rows - whole) * n < 2 ** 31
            # (the pieces' counters)
            assert n == 1 or rows - whole <= 4864
