"""What the paged forward's second kernel believes of a workspace that the first one did
not fill, because a wait gave up: csrc/gbattn_parts.h, compiled for the host."""
import itertools
import os
import shutil
import subprocess

from exact_tiled_attention_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include "gbattn_parts.h"
int main() {
  int first, n, ctas;
  while (std::scanf("%d %d %d", &first, &n, &ctas) == 3) std::printf("%d\n", gbattn::split_parts(first, n, ctas));
}
"""


def test_parts_lie_in_the_workspace(tmp_path):
    """True exactly where every part is the state of a CTA of the grid, for entries that
    a call writes and for whatever a workspace may have held."""
    src, exe = tmp_path / "parts.cpp", tmp_path / "parts"
    src.write_text(PROGRAM)
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-ftrapv", "-I", _build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    edge = [-2 ** 31, -2 ** 31 + 1, -0x01010101, -152, -1, 0, 1, 2, 3, 150, 151, 152, 153, 160, 0x7F7F7F7F, 2 ** 31 - 1]
    cases = list(itertools.product(edge, edge, [1, 2, 3, 152, 160]))
    text = "".join("%d %d %d\n" % c for c in cases)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
    want = [n >= 2 and 0 <= first and first + n <= ctas for first, n, ctas in cases]
    assert [o == "1" for o in out] == want
    assert any(want) and not all(want)


def test_the_second_kernel_asks():
    """Before it follows an entry."""
    text = open(os.path.join(_build.CSRC, "prefill_paged.cu")).read()
    kernel = text[text.index("prefill_paged_merge_kernel("):text.index("struct Shape")]
    said = kernel.index("p.parts[unit]")
    assert kernel.index("split_parts(", said) < kernel.index("load_ml", said) and "part = said" in kernel
