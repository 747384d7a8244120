"""The blocks and stages the kernels ask for fit the device, swept over every size on the host.

csrc/layout.h holds that arithmetic without any CUDA, so a small C++ program can
run it for a device whose blocks may opt in to 227 KB.  A launch that asks for
more dynamic shared memory than the limit its kernel was given is refused.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "invariant_token_log_gb300", "csrc")

HEAD = r"""
#include <cstdio>
#include "layout.h"
using namespace bil_layout;
static const int kOptin = 227 * 1024;
static int bad = 0;
// `blocks` resident blocks of `stages` stages: within the launch limit, and together within the SM
static void check(const char *what, int size, int form, int blocks, size_t statics, size_t stages, size_t stage_bytes) {
  const size_t bytes = stages * stage_bytes;
  const bool fits = bytes <= dynamic_limit(kOptin) && bytes + statics <= kOptin &&
                    blocks * (bytes + statics + kReserved) <= kSmBytes;
  if (!fits && bad++ < 10) printf("%s: size %d form %d: %d blocks of %zu x %zu\n", what, size, form, blocks, stages, stage_bytes);
}
"""

NORM = HEAD + r"""
int main() {
  const size_t limit = dynamic_limit(kOptin);
  int widest[2][2] = {{0, 0}, {0, 0}};  // the widest row of the backward's ring, by element size and dh
  for (int eb = 2; eb <= 4; eb += 2)
    for (int operands = 1; operands <= 3; ++operands)
      for (int width = 1; width <= kMaxRowThreads * kMaxGroups * kVec; ++width) {
        const size_t stage = size_t(slot_bytes(width * eb)) * operands;
        const int form = 10 * eb + operands;
        int threads = 0, groups = 0, per_sm = 0, stages = 0;
        if (operands <= 2) {
          row_shape(width, 4, &threads, &groups);
          fwd_ring(stage, threads, eb, limit, &per_sm, &stages);
          if (stages < 1 || per_sm < 1) ++bad, printf("forward: no ring at width %d\n", width);
          check("forward", width, form, per_sm, kNormStatics, stages, stage);
        }
        if (operands >= 2) {
          row_shape(width, 2, &threads, &groups);
          if (threads == kWarp) continue;
          per_sm = bwd_per_sm(threads, groups);
          bwd_ring(stage, limit, &per_sm, &stages);
          if (stages == 0) {
            if (eb == 2) ++bad, printf("backward: no ring at width %d of a 16-bit type\n", width);
            continue;
          }
          if (stages < 2 || per_sm < 1) ++bad, printf("backward: %d stages at width %d\n", stages, width);
          widest[eb == 4][operands == 3] = width;
          check("backward", width, form, per_sm, kNormStatics, stages, stage);
        }
      }
  printf("widest %d %d\n", widest[1][0], widest[1][1]);
  return bad != 0;
}
"""


def run(tmp_path, program):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.fail("no C++ compiler on PATH")
    src, exe = tmp_path / "sweep.cpp", tmp_path / "sweep"
    src.write_text(program)
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


def test_norm_rings_fit(tmp_path):
    out = run(tmp_path, NORM)
    assert out.returncode == 0, out.stdout
    # where float32 rows leave the backward's ring, without and with dh: four slots of two stages, six of two
    assert out.stdout.split() == ["widest", "14460", "9636"]


TOPK = HEAD + r"""
int main() {
  for (int eb = 2; eb <= 4; eb += 2)
    for (int tile = 8; tile * eb <= 64 * 1024; tile += 8)
      for (int pad = 0; pad <= 16; pad += 16) {  // rows off 16-byte boundaries
        const size_t stage = (size_t(tile) * eb + pad + 127) / 128 * 128;
        int warps = 0, blocks = 0;
        topk_stream(stage, dynamic_limit(kOptin), &warps, &blocks);
        if (warps < 1 || warps > kTopkMaxWarps || blocks < 1) ++bad, printf("no warps at tile %d\n", tile);
        check("pass", tile, 10 * eb + pad / 16, blocks, kTopkStatics, warps, stage);
      }
  return bad != 0;
}
"""


def test_topk_stages_fit(tmp_path):
    out = run(tmp_path, TOPK)
    assert out.returncode == 0, out.stdout
