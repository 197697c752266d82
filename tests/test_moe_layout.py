"""CPU test of the mixture-of-experts kernel's layout: for every number of tokens, experts and choices that rocmfp4_moe accepts,
both block layouts, aligned rows or not, nothing in shared memory or in the workspace passes the end of its room.

csrc/moe_layout.h is plain C++; the walk below is compiled with it by the host compiler.  It restates what the kernel uses of
each array: the selection's 4 bytes an expert in the first 8 E bytes of a warp's room and up to E candidates of 8 bytes behind
them, for one warp a token and at most 16; the outputs of a tile, 16 rows x tokens for each of 16 warps; a warp's sums, 128
floats for every four tokens; and the ring, whose unaligned rows are read up to 24 bytes behind the word of their last block."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
WALK = r"""
#include "moe_layout.h"
using namespace rocmfp4;
// 0, or the number of the first rule that does not hold; at[]: the sizes.
static int rule(int v, bool al, int64_t M, int64_t E, int64_t k, int64_t K, int64_t I) {
  MoeLayout l;
  if (!moe_layout(v, al, M, E, k, K, I, &l)) return 1;
  const int64_t W = 16, block = v == 0 ? 18 : 17, span = v == 0 ? 144 : 272, blocks = v == 0 ? 8 : 16;
  const int64_t limit = 227 * 1024 - 15744;  // a CTA's shared memory but the static arrays
  if (l.bytes > limit || l.stages < 1 || l.stages > 6) return 2;
  // one after the other, each with its room
  if (M * k * 4 > l.off_mask || l.off_mask + E * 4 > l.off_list || l.off_list + E * 2 > l.off_slot || l.off_slot + M * E > l.off_unscale ||
      l.off_unscale + M * 4 > l.off_y || l.off_y + W * 16 * M * 4 > l.off_acc || l.acc_floats < (M + 3) / 4 * 128 ||
      l.off_acc + W * l.acc_floats * 4 > l.off_ring || l.off_ring + W * l.stages * l.stage_bytes > l.bytes) return 3;
  if (l.off_mask % 4 || l.off_list % 4 || l.off_unscale % 4 || l.off_y % 16 || l.off_acc % 16 || l.off_ring % 128 || l.stage_bytes % 128) return 4;
  // the selection: behind what lasts, inside the launch's shared memory
  const int64_t warps = M < W ? M : W;
  if (l.off_select < l.off_y || l.off_select % 8 || l.select_bytes % 8 || l.select_bytes < 8 * E + 8 * E ||
      l.off_select + warps * l.select_bytes > l.bytes) return 5;
  // a stage: ns spans of 16 rows
  if (al) {
    if (l.ns * 16 * span > l.stage_bytes) return 6;
  } else {
    const int64_t pitch = l.ns * span + 32;
    if (16 * pitch > l.stage_bytes) return 7;
    // a row's copy of up to ns spans from and to 16-byte boundaries, and the reads of its last block: six words
    const int64_t last = 15 + (l.ns - 1) * span + 3 * (blocks / 4 * block) + (blocks / 4 - 1) * block / 4 * 4 + 24;
    if ((15 + l.ns * span + 15) / 16 * 16 > pitch || 15 * pitch + last > l.stage_bytes + 32) return 8;
  }
  // the workspace: logits, scales, largest values, h, activations, two halves of h, and 512 bytes read ahead
  const int64_t sk = (K / 32 + blocks - 1) / blocks, si = (I / 32 + blocks - 1) / blocks, x = 16 * blocks;  // floats of a span's activations
  if (l.ws_logits + M * E > l.ws_unscale || l.ws_unscale + M > l.ws_amax || l.ws_amax + M * k > l.ws_h || l.ws_h + M * k * I > l.ws_x ||
      l.ws_x + M * sk * x > l.ws_hi || l.ws_hi + M * k * si * x > l.ws_lo || l.ws_lo + M * k * si * x > l.ws_end ||
      l.ws_end + 128 > (int64_t)kMoeWsFloats) return 9;
  if (l.ws_x % 4 || l.ws_hi % 4 || l.ws_lo % 4) return 10;
  return 0;
}
extern "C" int walk(int v, int al, int64_t* at) {
  const int64_t widths[][2] = {{32, 32}, {256, 256}, {512, 512}, {5120, 1536}, {2048, 768}, {1056, 352}, {7168, 2048}, {32768, 32768}, {32736, 32736}};
  for (int64_t M = 1; M <= 32; ++M)
    for (int64_t E = 1; E <= 512; ++E)
      for (int64_t k = 1; k <= 16 && k <= E; ++k)
        for (const auto& w : widths) {
          if (M * k * w[1] > (1 << 22)) continue;
          if (al && (w[0] % (v == 0 ? 256 : 512) || w[1] % (v == 0 ? 256 : 512))) continue;
          if (const int r = rule(v, al, M, E, k, w[0], w[1])) {
            at[0] = M, at[1] = E, at[2] = k, at[3] = w[0], at[4] = w[1];
            return r;
          }
        }
  return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("moe_layout")
    src, so = d / "walk.cpp", d / "walk.so"
    src.write_text(WALK)
    cxx = shutil.which("g++") or "g++"
    subprocess.run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I", os.path.join(ROOT, "gemm_rocmfp4_dequant_gb300", "csrc"), str(src), "-o", str(so)],
                   check=True)
    return ctypes.CDLL(str(so))


@pytest.mark.parametrize("aligned", [0, 1])
@pytest.mark.parametrize("variant", [0, 1])
def test_nothing_passes_its_room(lib, variant, aligned):
    at = (ctypes.c_int64 * 5)()
    rule = lib.walk(variant, aligned, at)
    assert rule == 0, f"rule {rule} at M, E, top_k, K, I = {list(at)}"
