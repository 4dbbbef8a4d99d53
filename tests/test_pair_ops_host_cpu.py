"""Host arithmetic of the operators around the layer, compiled from its source with the C++ compiler."""

import os
import shutil
import subprocess

from co_folding_pair_gb300 import _lib


def compiled(tmp_path, text, *sources):
    """Builds a program of `text` and `sources` (names under csrc/) and returns what it prints; it has to exit 0."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_lib._nvcc()))), "include")
    main, exe = tmp_path / "main.cpp", tmp_path / "main"
    main.write_text(text)
    flags = ["-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + _lib.CSRC, "-I" + _lib.INCLUDE, "-I" + cuda]
    r = subprocess.run([shutil.which("g++") or "g++", *flags, "-x", "c++", str(main), *[os.path.join(_lib.CSRC, s) for s in sources],
                        "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


PLANES = r"""
#include <cstdio>
#include "pair_ops.h"
using trimul::HeadPlane;
int main() {
  long long looked = 0;
  for (int V : {4, 8})
    for (uint32_t n : {1u, 2u, 3u, 4u, 5u, 6u, 7u, 8u, 9u, 15u, 16u, 17u, 1000u, 2147483647u})
      for (long long planes = 1; planes <= 20; ++planes)
        for (long long q = 0; q < planes; ++q) {
          const HeadPlane p(q * n, n, planes * n, V);
          if (p.at % V || p.at + p.early != q * n || p.early >= static_cast<uint32_t>(V) || p.end != p.early + n) return 1;
          // the first groups and the last ones
          for (uint32_t k = 0; k < p.end; k = k < 64 || k + 256 > p.end ? k + V : p.end / V * V - 64) {
            const bool whole = k + V <= p.whole, inside = p.at + k + V <= planes * n;
            if (whole != inside) return std::printf("V %d n %u plane %lld of %lld: group %u\n", V, n, q, planes, k), 2;
            ++looked;
          }
        }
  std::printf("%lld groups\n", looked);
}
"""


def test_head_planes_are_read_within_their_tensor(tmp_path):
    """A group of 16 bytes is read whole if, and only if, all of it is in the tensor, planes smaller than a group
    among others."""
    assert "groups" in compiled(tmp_path, PLANES)
