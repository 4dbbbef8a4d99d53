"""Host arithmetic of the operators around the layer, compiled from its source with the C++ compiler."""

import os
import shutil
import subprocess

import pytest

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
      for (int B : {1, 2, 3, 5, 9, 20}) for (int H : {1, 2, 3, 4, 7, 8, 9, 256})
        for (long long q = 0, planes = B * H; q < planes; ++q) {
          const HeadPlane p(static_cast<uint32_t>(q / H), static_cast<int>(q % H), B, H, n, V);
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


# A CUDA runtime that only writes down what it is called for, so that the entry points' host code runs without a GPU.
RUNTIME = r"""
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include "api_status.h"
#include "pair_ops.h"

extern "C" {
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetDeviceCount(int* n) { return *n = 1, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  return *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152, cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) { return std::puts("malloc"), *p = std::malloc(n), cudaSuccess; }
cudaError_t cudaFree(void* p) { return std::puts("free"), std::free(p), cudaSuccess; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return std::puts("copy"), cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return std::puts("synchronize device"), cudaSuccess; }
cudaError_t cudaStreamSynchronize(cudaStream_t s) { return std::printf("synchronize %s\n", s ? "a stream" : "stream 0"), cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
}
namespace trimul {
trimul_status fail(trimul_status s, const char* fmt, ...) {
  std::va_list a;
  va_start(a, fmt), std::vprintf(fmt, a), va_end(a);
  return std::puts(""), s;
}
trimul_status cuda_fail(cudaError_t, const char* what) { return std::puts(what), TRIMUL_ERR_CUDA; }
cudaError_t launch_relpos_forward(const RelposArgs&, const void*, bool, const void*, void*, bool, trimul_layout, int, cudaStream_t) { return std::puts("forward"), cudaSuccess; }
size_t relpos_backward_workspace(int, int, int, int, int, trimul_layout, bool, int) { return 64; }
cudaError_t launch_relpos_backward(const RelposArgs&, const void*, bool, trimul_layout, float*, bool, float*, int, cudaStream_t) { return std::puts("backward"), cudaSuccess; }
cudaError_t launch_residual_forward(const ResidualArgs&, int, cudaStream_t) { return cudaSuccess; }
size_t residual_backward_workspace(int, long long, int) { return 64; }
cudaError_t launch_residual_backward(const ResidualArgs&, int, cudaStream_t) { return cudaSuccess; }
size_t grad_workspace(int, int) { return 64; }
cudaError_t launch_grad_norm(const trimul_grad_tensor*, int, trimul_norm_kind, float*, void*, bool, float, int, cudaStream_t) { return cudaSuccess; }
}  // namespace trimul
"""


@pytest.mark.parametrize("kind,buckets,want", [
    (0, 0, ["made", "gone"]),
    (1, 32, ["malloc", "copy", "synchronize stream 0", "made", "synchronize device", "free", "gone"]),
])
def test_a_plan_is_made_once_its_table_has_arrived(tmp_path, kind, buckets, want):
    """A copy from pageable memory may return before its data is on the device, and other streams do not wait for it."""
    main = RUNTIME + r"""
int main() {
  const trimul_relpos_params p{static_cast<trimul_bucket_kind>(KIND), 128, BUCKETS, 1, 0};
  trimul_relpos r = nullptr;
  if (trimul_relpos_create(&r, &p, 0) != TRIMUL_OK) return 1;
  std::puts("made");
  if (trimul_relpos_destroy(r) != TRIMUL_OK) return 1;
  std::puts("gone");
}
""".replace("KIND", str(kind)).replace("BUCKETS", str(buckets))
    assert compiled(tmp_path, main, "pair_ops_api.cu").split("\n")[:-1] == want


def test_alignment_is_asked_for_where_it_is_needed(tmp_path):
    """dtable is written, and the HEADS layout's table read, one element at a time; all else 16 bytes at a time."""
    main = RUNTIME + r"""
int main() {
  const trimul_relpos_params p{TRIMUL_BUCKETS_LINEAR, 4, 0, 1, 0};
  trimul_relpos r = nullptr;
  if (trimul_relpos_create(&r, &p, 0) != TRIMUL_OK) return 1;
  auto at = [](long mb, long off) { return reinterpret_cast<char*>((mb << 20) + off); };
  const int32_t* const pos = reinterpret_cast<int32_t*>(at(1, 4));
  auto forward = [&](trimul_layout lay, long table, trimul_dtype type, long out) {
    return trimul_relpos_forward(r, at(2, table), type, pos, pos, nullptr, nullptr, nullptr, 1, 8, 8, 16, lay, at(3, out), TRIMUL_BF16, nullptr, 0);
  };
  auto backward = [&](trimul_layout lay, long dout, long dtable) {
    return trimul_relpos_backward(r, at(2, dout), TRIMUL_BF16, pos, pos, nullptr, nullptr, 1, 8, 8, 16, lay,
                                  reinterpret_cast<float*>(at(3, dtable)), at(4, 0), 64, nullptr, 0);
  };
  const trimul_layout P = TRIMUL_LAYOUT_PAIR, H = TRIMUL_LAYOUT_HEADS;
  std::printf("%d %d %d\n", forward(P, 16, TRIMUL_BF16, 16), forward(H, 2, TRIMUL_BF16, 16), forward(H, 4, TRIMUL_F32, 16));
  std::printf("%d %d %d\n", backward(P, 16, 4), backward(H, 16, 12), backward(P, 0, 0));
  std::puts("refused");
  std::printf("%d %d %d %d\n", forward(P, 8, TRIMUL_F32, 16), forward(H, 2, TRIMUL_F32, 16), forward(H, 1, TRIMUL_BF16, 16), forward(H, 0, TRIMUL_F32, 8));
  std::printf("%d %d %d\n", backward(P, 8, 0), backward(H, 2, 0), backward(P, 0, 2));
  return trimul_relpos_destroy(r) != TRIMUL_OK;
}
"""
    fine, refused = compiled(tmp_path, main, "pair_ops_api.cu").split("refused\n")
    assert sorted(fine.split()) == sorted(["0"] * 6 + ["forward"] * 3 + ["backward"] * 3)
    lines = refused.strip().split("\n")
    assert [v for v in lines if v[0].isdigit()] == ["1 1 1 1", "1 1 1"]
    assert sorted(v for v in lines if not v[0].isdigit()) == sorted(
        ["table must be 16-byte aligned", "table must be 4-byte aligned", "table must be 2-byte aligned",
         "base and out must be 16-byte aligned", "dout must be 16-byte aligned", "dout must be 16-byte aligned",
         "dtable must be 4-byte aligned"])
