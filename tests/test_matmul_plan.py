"""How a block-scaled product is cut (kvp_matmul_plan.h, host code), over all sizes that the
entry point takes."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "pagedattention_decode_kvp_gb300", "csrc")
MAIN = """
#include <cstdio>
#include "kvp_matmul_plan.h"
int main() {
  const int sizes[] = {1, 2, 16, 17, 64, 127, 129, 1000, 4096, 33098, 1 << 20, (1 << 30) - 1, 1 << 30,
                       (1 << 30) + 5, 2147483647 - 255};
  const int groups[] = {1, 2, 31, 64, 1000, (2147483647 - 127) / 128};
  for (int m : sizes)
    for (int n : sizes)
      for (int g : groups) {
        const kvp::MatmulPlan p = kvp::matmul_plan(m, n, g);
        std::printf("%d %d %d %d %d\\n", m, n, g, p.tokens, p.splits);
      }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """The plans of every mix of sizes, by a program that ends at the first overflow."""
    at = tmp_path_factory.mktemp("plan")
    (at / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    f"-I{CSRC}", str(at / "main.cpp"), "-o", str(at / "main")], check=True)
    r = subprocess.run([str(at / "main")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]


def test_every_size_has_a_plan(plans):
    assert len(plans) == 15 * 15 * 6
    for m, n, groups, tokens, splits in plans:
        assert tokens in (16, 32, 64, 128, 256)
        assert 1 <= splits <= 8 and (splits == 1 or (tokens < 256 and 2 * splits <= groups))
        # no tile is twice as high as the rows that there are
        assert tokens <= 16 or tokens == 256 or tokens < 2 * m


def test_many_rows_go_to_pairs(plans):
    assert all(tokens == 256 for m, n, _, tokens, _ in plans if m >= 33098 and n >= 33098)


def test_the_entry_point(plans):
    import pagedattention_decode_kvp_gb300 as kvp
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    for m, n, groups, tokens, splits in plans:
        if n > 2 ** 31 - 256 or m * n > 2 ** 40:
            continue                     # (too many tiles are refused below)
        for k in (128 * groups - 112, 128 * groups):
            if k <= 2 ** 31 - 128:
                assert kvp.kvp_matmul_fp8_plan(m, n, k) == (tokens, splits)
    for bad in ((0, 5, 16), (-1, 5, 16), (5, 0, 16), (5, 5, 0), (5, 5, 24), (2 ** 31 - 1, 5, 16),
                (5, 2 ** 31 - 1, 16), (5, 5, 2 ** 31 - 16), (2 ** 31 - 300, 2 ** 31 - 300, 16),
                (2 ** 32 + 5, 5, 16), (5, 2 ** 32 + 5, 16), (5, 5, 2 ** 32 + 16)):
        with pytest.raises(kvp.KvpError):
            kvp.kvp_matmul_fp8_plan(*bad)
    lib = kvp.load_library()
    assert lib.kvp_matmul_fp8_plan(5, 5, 16, None, None) == kvp.KVP_ERR_INVALID_ARG
