"""The choice of a product's kernel is host arithmetic: the same rule over the whole range of sizes (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "linear_choice.h"
int main() {
  long long M, N, K;
  int mn, sms;
  while (scanf("%lld %lld %lld %d %d", &M, &N, &K, &mn, &sms) == 5) {
    const moe::LinearChoice c = moe::choose_linear((int)M, (int)N, (int)K, mn, sms);
    printf("%d %d\n", c.nb, c.S);
  }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cc = shutil.which("g++")
    if not cc:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("choice")
    (d / "c.cpp").write_text(PROGRAM)
    exe = str(d / "c")
    subprocess.run([cc, "-O1", "-std=c++17", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error",
                    "-I" + os.path.join(ROOT, "expert_grouped_gemm_gb300", "csrc"), str(d / "c.cpp"), "-o", exe], check=True)

    def run(cases, sms=152):
        text = "".join(f"{M} {N} {K} {mn} {sms}\n" for M, N, K, mn in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return [tuple(int(v) for v in line.split()) for line in r.stdout.splitlines()]

    return run


def test_rows_past_half_the_range_choose_as_those_before(choose):
    """M up to 2^31 - 2^20: the estimates grow with the rows, the choice between them does not change at 2^30."""
    for N, K in ((8, 8), (128, 64), (64, 512)):
        below, above, last = choose([(2 ** 30 - 64, N, K, 0), (2 ** 30 + 64, N, K, 0), (2 ** 31 - 2 ** 20, N, K, 0)])
        assert below == above == last, (N, K)


def test_choices_at_known_sizes(choose):
    """Few tokens split the weight's K over a cluster, large products run on CTA pairs; no split has an empty part."""
    got = choose([(16, 4096, 4096, 0), (2048, 4096, 4096, 0), (4096, 8192, 2048, 0), (4096, 128, 2048, 0)])
    assert got == [(16, 4), (0, 2), (0, 2), (64, 4)]
    cases = [(M, N, K, mn) for M in (1, 17, 300, 5000) for N in (1, 130, 4096) for K in (1, 64, 65, 500, 4096) for mn in (0, 1)]
    for (M, N, K, mn), (nb, S) in zip(cases, choose(cases)):
        assert nb in (0, 16, 32, 64) and (nb >= 64 or nb == 0 or not mn)
        assert S in (1, 2, 4, 8) and (S <= (K + 63) // 64 if nb else S <= 2)
