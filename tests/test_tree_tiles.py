"""Which tiles a batch's trees get, compiled and run on the CPU (no GPU needed)."""
import os
import subprocess

from test_batch_host import PKG, _nvcc

TILES = r"""
#include <cstdio>
#include "chunk_attn.cuh"
using namespace sub;

int bad = 0;
void is(int tile, int group, int n_seqs, int n_rows, int heads, long long keys, bool codes, const char* what) {
  const int t = tree_rows(group, n_seqs, n_rows, heads, keys, codes, 152);
  if (t != tile) bad += printf("%s: %d seqs, %d rows, group %d, %lld keys, codes %d: %d, not %d\n", what, n_seqs,
                               n_rows, group, keys, codes, t, tile) > 0;
}

int main() {
  // half the sequences with 5 nodes and half with 9, in 4 heads: two tiles of 32, or one of 64
  for (int n : {16, 48})
    for (int pad : {0, 1, 2, 3}) is(64, 4, n, 7 * n + pad, 8, 8128, false, "5 and 9 nodes");
  is(32, 4, 16, 7 * 16, 8, 8128, true, "5 and 9 nodes");
  is(32, 4, 4, 7 * 4, 8, 2128, false, "5 and 9 nodes, few keys");
  // a level of 8 nodes
  is(32, 4, 16, 8 * 16, 8, 16416, true, "8 nodes");
  is(32, 4, 16, 8 * 16 + 1, 8, 16416, true, "8 nodes and a row of no sequence");
  is(32, 4, 4, 8 * 4 + 1, 8, 2128, false, "8 nodes and a row of no sequence, few keys");
  is(64, 7, 32, 8 * 32, 4, 8240, false, "8 nodes of 7 heads");
  is(64, 8, 16, 8 * 16 + 1, 8, 8192, false, "64 rows each and a row of no sequence");
  // fewer rows of no sequence than sequences change nothing, whatever the batch
  for (int group : {1, 2, 4, 5, 7, 8, 16, 64})
    for (int n : {2, 3, 8, 16, 64})
      for (int nodes : {1, 2, 5, 8, 9, 16, 33, 65, 129})
        for (long long keys : {100, 1000, 8192, 65536})
          for (int codes = 0; codes < 2; ++codes) {
            const int t = tree_rows(group, n, n * nodes, 8, keys, codes, 152);
            for (int pad = 1; pad < n; ++pad) is(t, group, n, n * nodes + pad, 8, keys, codes, "padded");
            if (t != 0 && t != 32 && t != 64) bad += puts("another tile") >= 0;
          }
  // the workspace is as large as tiles of 64 need from 17 rows on average on
  for (int group : {1, 3, 4, 7, 16, 33, 64})
    for (int n = 1; n < 40; ++n)
      for (int rows = 1; rows < 40 * n; rows += 1 + rows / 7)
        for (long long keys : {100, 8192, 100000})
          for (int codes = 0; codes < 2; ++codes)
            if (rows * group <= 16 * n) is(0, group, n, rows, 8, keys, codes, "few rows");
  return bad != 0;
}
"""


def test_tiles_of_trees(tmp_path):
    src = tmp_path / "tiles.cu"
    src.write_text(TILES)
    exe = tmp_path / "tiles"
    subprocess.run([_nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-I", os.path.join(PKG, "csrc"),
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
