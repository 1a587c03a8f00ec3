"""The tiled products' choice of a tile, evaluated on the host: choose_tiles and its
measured costs as w4_internal.h has them, compiled with g++ (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_bit_weight_awq_amd", "csrc")

MAIN = """
int main(int n, char** v) {
  for (int i = 1; i + 3 < n; i += 4) {
    const int64_t tokens = atoll(v[i + 1]), in = atoll(v[i + 2]), out = atoll(v[i + 3]);
    int mt = 0;
    TileSplit s{};
    if (v[i][0] == 'b')
      choose_tiles(tokens, (int)((in + 255) / 256), (int)((out + 63) / 64), kDxCosts, 1.0f, &mt, &s);
    else
      choose_tiles(tokens, (int)((out + 255) / 256), (int)(in / 128), kGemmCosts, SCALE, &mt, &s);
    printf("%d %d %d %d\\n", mt, s.full, s.left, s.parts);
  }
}
"""


def choices(folder, shapes, scale="1.0f"):
    """(32-token units of a tile, whole tiles, split tiles, their parts) of each ("f" or "b", tokens, in, out)."""
    cxx = next((shutil.which(c) for c in ("g++", "c++", "clang++") if shutil.which(c)), None)
    if cxx is None:
        pytest.skip("no host C++ compiler")
    text = open(os.path.join(CSRC, "w4_internal.h")).read()
    body = re.search(r"struct TileSplit \{.*?constexpr TileCosts kDxCosts = .*?;\n", text, re.S).group(0)
    src, exe = os.path.join(str(folder), "choice.cpp"), os.path.join(str(folder), "choice")
    with open(src, "w") as f:
        f.write("#include <cstdint>\n#include <cstdio>\n#include <cstdlib>\n" + body + MAIN.replace("SCALE", scale))
    subprocess.run([cxx, "-std=c++17", "-O1", src, "-o", exe], check=True)
    out = subprocess.run([exe, *(str(i) for s in shapes for i in s)], check=True, stdout=subprocess.PIPE, text=True).stdout
    return [tuple(int(i) for i in line.split()) for line in out.splitlines()]
