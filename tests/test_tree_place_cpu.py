"""Where a CTA's range begins inside a request, at the most tiles that the
limits allow: 16384 tiles x 4 blocks of rows x 65535 KV heads, 4294901760.  (A
call of that size would run for many seconds.)"""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_kv_block_gb300", "csrc")


def test_place_of_a_range(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    cases = [(in_, tiles) for tiles in (1, 2, 7, 12345, 16383, 16384) for pairs in (1, 5, 131072, 4 * 65535)
             for in_ in (0, 1, tiles - 1, tiles, pairs * tiles // 2, pairs * tiles // 152 * 151, pairs * tiles - 1)
             if in_ < pairs * tiles]
    assert max(c[0] for c in cases) > 1 << 31 and max(c[0] for c in cases) < 1 << 32
    main = tmp_path / "place.cpp"
    main.write_text('#include "tree_place.h"\n#include <cstdio>\nint main() {\n'
                    + "".join(f"  {{ auto p = oasis::tree_place({i}ll, {t}); std::printf(\"%d %d\\n\", p.pair, p.tile); }}\n" for i, t in cases)
                    + "}\n")
    exe = str(tmp_path / "place")
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(main), "-o", exe], check=True)
    got = [tuple(map(int, line.split())) for line in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines()]
    assert got == [divmod(i, t) for i, t in cases]


def test_the_offset_is_not_narrowed_before():
    text = open(os.path.join(CSRC, "tree.cu")).read()
    assert "tree_place(__shfl_sync(0xffffffffu, u0 - (incl - t), from), walk.q.tiles)" in text
    assert "static_cast<int>(u0" not in text
