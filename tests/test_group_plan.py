"""How the stable sort cuts its slots (csrc/gsr_group_plan.hpp, the code that
host and kernels share), compiled for the host: the runs of all waves of all
blocks cover every slot once and in order, up to the largest count of slots."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tiled_dense_gemm_scale_amd", "csrc")

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "gsr_group_plan.hpp"
int main(int argc, char** argv)
{
    for (int i = 1; i + 1 < argc; i += 2) {
        const long long n = std::atoll(argv[i]), groups = std::atoll(argv[i + 1]);
        const gsr::GroupPlan plan = gsr::group_plan(n, groups);
        const int waves = plan.chunk >= 64 * gsr::kGroupWaves ? gsr::kGroupWaves : plan.chunk > 64 ? (plan.chunk + 63) / 64 : 1;
        long long next = 0;
        for (int b = 0; b < plan.blocks; ++b)
            for (int w = 0; w < waves; ++w) {
                const gsr::GroupSpan r = gsr::group_run(gsr::group_block((int)n, plan.chunk, b), w, waves);
                // a run begins where the last one ended, and all but the last of a block are whole steps
                if (r.len < 0 || r.beg != next) return std::printf("%lld slots: wave %d of block %d at %d + %d, not %lld\n", n, w, b, r.beg, r.len, next), 1;
                next += r.len;
            }
        if (next != n || plan.blocks > gsr::kGroupBlocks) return std::printf("%lld slots: %lld covered\n", n, next), 1;
    }
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("group_plan")
    src, out = d / "main.cpp", d / "main"
    src.write_text(MAIN)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover", "-I", CSRC,
                    str(src), "-o", str(out)], check=True, capture_output=True)
    return str(out)


@pytest.mark.parametrize("groups", [1, 8, 64, 1000, 1024])
def test_runs_cover_the_slots(program, groups):
    counts = [1, 63, 64, 65, 1000, 8191, 8192, 8193, 10000, 131072, 524288, 524289, 2200002, 10 ** 8 + 7, 2 ** 30, 2 ** 31 - 300000,
              2147221504, 2147221505, 2 ** 31 - 1024, 2 ** 31 - 65, 2 ** 31 - 64, 2 ** 31 - 1]  # 2147221505: 256 blocks end at 2^31
    done = subprocess.run([program, *(str(v) for n in counts for v in (n, groups))], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout + done.stderr
