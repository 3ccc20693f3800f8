"""How the backward's dH is cut into parts of the vocabulary (policy and preference losses), computed on the host."""
import subprocess

import pytest

from chunked_lm_head_linear_gb300 import build

CLUSTERS = 76
MAIN = r"""
#include <cstdio>
#include "lce_internal.h"
int main() {
  long long r, v, d, w;
  while (std::scanf("%lld %lld %lld %lld", &r, &v, &d, &w) == 4) std::printf("%d\n", lce::dh_parts_balanced(r, v, d, w != 0));
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    at = tmp_path_factory.mktemp("parts")
    (at / "main.cu").write_text(MAIN)
    subprocess.run([build.nvcc(), "-std=c++17", "-I" + build.CSRC, "-o", str(at / "main"), str(at / "main.cu")], check=True)

    def ask(cases):
        text = "".join(f"{r} {v} {d} {int(w)}\n" for r, v, d, w in cases)
        return [int(x) for x in subprocess.run([str(at / "main")], input=text, capture_output=True, text=True, check=True).stdout.split()]
    return ask


SHAPES = [(r, v, d) for r in (1, 32, 256, 300, 512, 768, 1024, 2560, 6144, 18432) for v in (64, 700, 32000, 151936)
          for d in (64, 256, 2048, 4096, 7168)]


def test_parts_cover_the_vocabulary(parts):
    """Each part has a k-block of 64 words at least: the launch cuts the vocabulary into ceil(kb / parts) of them."""
    cases = [(*s, w) for s in SHAPES for w in (False, True)]
    for (r, v, d, w), p in zip(cases, parts(cases)):
        kb = -(-v // 64)
        assert 1 <= p <= 32 and -(-kb // -(-kb // p)) == p, (r, v, d, w, p)


def test_without_dW_the_clusters_are_kept_busy(parts):
    """With no dW in the launch nothing else fills the clusters: the parts are taken in rounds, which leave less than half as
    much again as an even share and a part's overhead where the vocabulary is long enough to be cut."""
    cases = [(*s, False) for s in SHAPES if s[1] == 151936 and s[0] >= 256]
    for (r, v, d, w), p in zip(cases, parts(cases)):
        kb, tiles = -(-v // 64), -(-r // 256) * -(-d // 256)
        depth = -(-tiles * p // CLUSTERS) * (kb / p)
        assert depth <= 1.5 * max(tiles * kb / CLUSTERS, kb / 32), (r, v, d, p, depth, tiles * kb / CLUSTERS)
