"""Host-side parts of the batched calls, compiled and run on the CPU (no GPU
needed): the guard that the join of cut work puts before its list of cuts."""
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "substitute_speculative_decoding_gb300")


def _nvcc():
    spec = importlib.util.spec_from_file_location("subspec_build", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    try:
        return mod.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")


CUTS = r"""
#include <climits>
#include <cstdio>
#include <cstring>
#include <random>
#include "chunk_attn.cuh"
using namespace sub;

int main() {
  const int n_ctas = 152, n_rows = 1000, heads = 8, group = 4, tile = 256;
  auto stands = [&](const ChunkCut& c, int part) {
    return cut_stands(c, part, n_ctas, n_rows, heads, group, tile);
  };
  const ChunkCut good{0, 1000, 15, 7, 3, 2 * 20 + 1, {0, 0}};
  if (!stands(good, 20)) return puts("a cut that is one is refused"), 1;
  ChunkCut c = good;
  c.pieces = 132;
  if (!stands(c, 20)) return puts("pieces up to the last CTA are refused"), 1;
  // each field out of its range, one at a time
  int bad = 0;
  auto no = [&](int ChunkCut::*f, int v) {
    ChunkCut x = good;
    x.*f = v;
    if (stands(x, 20)) bad += printf("taken: field value %d\n", v) > 0;
  };
  for (int v : {-1, 1, 1001, 1 << 30, INT_MIN, INT_MAX}) no(&ChunkCut::row0, v);
  for (int v : {-5, 0, 1001, INT_MAX, INT_MIN, 950 / 64}) no(&ChunkCut::rows, v);   // too few for tile 15
  for (int v : {-1, 16, 1 << 24, INT_MAX, INT_MIN}) no(&ChunkCut::tile, v);
  for (int v : {-1, 8, INT_MAX, INT_MIN}) no(&ChunkCut::head, v);
  for (int v : {0, 1, -1, 133, INT_MAX, INT_MIN}) no(&ChunkCut::pieces, v);
  for (int v : {-1, 39, 42, INT_MAX, INT_MIN}) no(&ChunkCut::first, v);
  // whatever memory holds: an entry that is taken names what there is
  std::mt19937 rng(1);
  for (int i = 0; i < 2000000; ++i) {
    ChunkCut x;
    int w[8];
    for (int& y : w) y = (int)(rng() >> (rng() % 32)) * (rng() % 8 ? 1 : -1);
    memcpy(&x, w, sizeof(x));
    const int part = rng() % n_ctas;
    if (!stands(x, part)) continue;
    const long long last_slot = 2ll * (part + x.pieces - 1);
    if (x.first < 0 || x.first >= 2 * n_ctas || last_slot >= 2 * n_ctas || x.row0 < 0 ||
        (long long)x.row0 + x.rows > n_rows || x.head >= heads || (long long)x.tile * tile >= (long long)x.rows * group)
      bad += printf("taken: random entry %d\n", i) > 0;
  }
  for (int fill : {0, 0xff, 0x7f, 0x80, 0x55}) {
    memset(&c, fill, sizeof(c));
    for (int part = 0; part < n_ctas; ++part)
      if (stands(c, part)) bad += printf("taken: fill %d\n", fill) > 0;
  }
  return bad != 0;
}
"""


def test_the_join_takes_no_entry_that_names_what_is_not_there(tmp_path):
    src = tmp_path / "cuts.cu"
    src.write_text(CUTS)
    exe = tmp_path / "cuts"
    subprocess.run([_nvcc(), "-std=c++17", "--expt-relaxed-constexpr", "-I", os.path.join(PKG, "csrc"),
                    str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
