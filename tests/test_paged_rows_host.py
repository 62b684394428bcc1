"""Rows of a request in the packed rows of a paged attention call, from whatever
stands in cu_rows: the function that the kernels use, compiled for the host.
They never lie outside the call's rows, and entries that do not decrease and
stay inside are taken as they are."""
import json
import os
import subprocess

import pytest

from block_discrete_diffusion_denoise_b200 import build

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "paged_attention.cuh"

// argv: group shift, then triples: rows, cu_rows[0], cu_rows[1]
int main(int argc, char** argv) {
  std::printf("[");
  for (int i = 2; i + 2 < argc; i += 3) {
    const int32_t cu[2] = {std::atoi(argv[i + 1]), std::atoi(argv[i + 2])}, kv = 5;
    dg::PagedAttnParams p{};
    p.cu_rows = cu;
    p.kv_lens = &kv;
    p.rows = std::atoi(argv[i]);
    p.width = 1;
    p.page_shift = 4;
    p.g_shift = std::atoi(argv[1]);
    const dg::PagedRequest a = dg::paged_request<16>(p, 0), b = dg::paged_request<256>(p, 0);
    std::printf("%s[%d,%d,%d,%d,%d,%d]", i > 2 ? "," : "", a.t0, a.n, a.tiles, b.t0, b.n, b.tiles);
  }
  std::printf("]");
}
"""

LO, HI = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, exe = d / "rows.cu", d / "rows"
    src.write_text(MAIN)
    subprocess.run([build._nvcc(), "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
                    "--expt-relaxed-constexpr", "-I", build.CSRC, "-I", os.path.dirname(build.HEADER),
                    "-o", str(exe), str(src)], check=True)
    return exe


@pytest.mark.parametrize("g_shift", [0, 1, 7])
def test_rows_of_a_request_stay_inside_the_call(program, g_shift):
    ends = [LO, LO + 1, -1000, -1, 0, 1, 7, 99, 100, 101, 4000, HI - 1, HI]
    cases = [(rows, a, b) for rows in (1, 100, 2 ** 20) for a in ends for b in ends]
    out = subprocess.run([str(program), str(g_shift)] + [str(x) for c in cases for x in c], check=True,
                         capture_output=True, text=True).stdout
    for (rows, a, b), got in zip(cases, json.loads(out), strict=True):
        t0 = min(max(a, 0), rows)
        n = max(0, min(b, rows) - t0)
        want = []
        for tile in (16, 256):
            want += [t0, n, -(-(n << g_shift) // tile)]
        assert got == want, (rows, a, b)
