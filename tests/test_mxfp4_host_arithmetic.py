"""Index arithmetic that the MXFP4 kernels share with the host, compiled for the host and run there (no GPU).

The programs below include the kernels' own header, so what they check is what the kernels compute with. They are built
with the undefined-behaviour sanitizer, which ends them at a signed overflow.
"""

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
#include "mxfp4.h"
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


def test_scalar_offsets_of_stages_stay_inside_the_row(tmp_path):
    """A buffer resource of the products ends with its last row. The range check of a load compares the lane's offset
    with the resource's size less the scalar offset, so the scalar offset may not pass the shortest range, one row: of
    8 values (16 bytes) four stages are loaded, whose plain offsets would be 0, 64, 128 and 192."""
    run_on_host(tmp_path, """
  for (int64_t K = 8; K <= (1 << 20); K += K < 8192 ? 8 : 8 * 1021) {
    const int blocks = (int)mx_blocks(K), real = (blocks + 3) / 4;
    for (int stage = 0; stage < real + 8; ++stage) {
      const uint32_t off = mx_stage_offset(stage, blocks);
      CHECK((int64_t)off < mx_row_bytes(K), "K %lld stage %d: %u", (long long)K, stage, off);
      if (stage < real) CHECK(off == (uint32_t)stage * 64u, "K %lld stage %d: %u", (long long)K, stage, off);
    }
  }""")


def test_row_tiles_of_the_largest_blocks(tmp_path):
    """Tiles of a block that ends at the largest capacity, 2^31 - 1 rows."""
    run_on_host(tmp_path, """
  const int top = 0x7FFFFFFF;
  for (int height : {32, 256})
    for (int64_t lo : {0ll, 1ll, 30ll, 31ll, 255ll, (long long)top - 300, (long long)top - 1, (long long)top})
      for (int64_t hi : {0ll, 1ll, 32ll, 33ll, 257ll, (long long)top - 257, (long long)top - 31, (long long)top}) {
        const int64_t want = hi > lo ? (hi - lo + height - 1) / height : 0;
        CHECK((int64_t)mx_row_tiles((int)lo, (int)hi, height) == want, "[%lld, %lld) by %d: %u", (long long)lo,
              (long long)hi, height, mx_row_tiles((int)lo, (int)hi, height));
      }""")
