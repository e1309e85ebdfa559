"""Index arithmetic that the 4-bit products share with the host, compiled for the host and run there (no GPU)."""

import os
import shutil
import subprocess

import pytest

from ragged_grouped_gemm_histogram_amd import build as B

pytestmark = pytest.mark.skipif(not shutil.which("hipcc") and not os.path.exists("/opt/rocm/bin/hipcc"), reason="no hipcc")


def run_on_host(tmp_path, body):
    """Builds and runs a host program around `body`; a check that fails ends it with its line."""
    src, exe = tmp_path / "check.hip", tmp_path / "check"
    src.write_text("""#include <cstdio>
#include <cstdlib>
#include "int4.h"
#define CHECK(c, ...) do { if (!(c)) { std::printf("line %d: %s ", __LINE__, #c); std::printf(__VA_ARGS__); std::exit(1); } } while (0)
using namespace moe;
int main() {
""" + body + "\n  std::puts(\"ok\");\n  return 0;\n}\n")
    flags = [f"-I{B.INCLUDE}", f"-I{B.CSRC}", "-std=c++17", "-O1", "--offload-host-only",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]
    made = subprocess.run([B.hipcc(), *flags, str(src), "-o", str(exe)], stdout=subprocess.PIPE,
                          stderr=subprocess.STDOUT, text=True, timeout=300)
    assert made.returncode == 0, made.stdout[-3000:]
    res = subprocess.run([str(exe)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=120)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stdout[-2000:]


def test_scalar_offsets_stay_inside_the_weights(tmp_path):
    """The range check of a load compares the lane's offset with the resource's size less the scalar offset, so no scalar
    offset may reach the size. A wave loads 64 weight rows (gated: 32 gate rows and 32 up rows); the waves of a wide tile
    stand next to each other, and where N is no multiple of the tile's width the last ones stand behind column N - 1."""
    run_on_host(tmp_path, """
  const int64_t widths[] = {8, 16, 40, 64, 128, 136, 264, 520, 768, 1032, 2048, 2056, 2880, 4104, int64_t(1) << 20};
  const int64_t lengths[] = {8, 32, 40, 128, 136, 264, 392, 768, 2048, 2880, 4104, int64_t(1) << 20};
  for (int gated = 0; gated < 2; ++gated)
    for (int64_t N : widths)
      for (int64_t K : lengths) {
        const int64_t w_rows = gated ? 2 * N : N, row_bytes = int4_row_bytes(K), units = (K + kInt4Unit - 1) / kInt4Unit;
        const int cols = gated ? 32 : 64;
        for (int waves : {1, 4}) {
          const int64_t tiles = (N + waves * cols - 1) / (waves * cols);
          for (int64_t tile : {int64_t(0), tiles - 1})
            for (int wave = 0; wave < waves; ++wave) {
              const int64_t n0 = (tile * waves + wave) * cols, at = int4_first_column(n0, N);
              CHECK(at >= 0 && at < N && (n0 >= N || at == n0), "N %lld from %lld: %lld", (long long)N, (long long)n0, (long long)at);
              for (int b = 0; b < kInt4Blocks; ++b)
                for (int64_t u : {int64_t(0), units - 1}) {
                  const int64_t range = int4_bytes_left(w_rows, at + (gated ? b >> 1 : 0) * N, row_bytes);
                  const uint32_t off = int4_block_at(gated != 0, b, (int)u, (uint32_t)row_bytes);
                  CHECK((int64_t)off < range, "gated %d N %lld K %lld from %lld, load %d of unit %lld: %u of %lld", gated,
                        (long long)N, (long long)K, (long long)n0, b, (long long)u, off, (long long)range);
                }
            }
        }
      }""")
