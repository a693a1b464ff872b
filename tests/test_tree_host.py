"""What the tree attention's kernels count with, run on the host: the functions of
csrc/tree_parts.cuh, compiled into a program of its own (no GPU needed)."""

import glob
import os
import re
import subprocess

import pytest

from mla_latent_kv_03_gb300 import build as B

HEAD = '#include <cstdio>\n#include <cstdlib>\n#include <cstdint>\n#include "tree_parts.cuh"\nusing namespace mla;\n'


def run(tmp_path, body):
    src, exe = tmp_path / "host.cu", tmp_path / "host"
    src.write_text(HEAD + body)
    subprocess.run([B._nvcc(), *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, "-o", str(exe), str(src)],
                   check=True, cwd=tmp_path, env=dict(os.environ, TMPDIR=str(tmp_path)))
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout


RING = """
int main() {
  // Readers as early as they can be: a segment's query is read as soon as it is there.
  // A wait for a phase returns only while no phase follows the one that is waited for.
  unsigned rng = 1;
  int waits = 0, lapped = 0, early = 0;
  for (int run = 0; run < 200; ++run) {
    QuerySlots q;
    int done[QuerySlots::kBars] = {}, ri = 0;      // phases completed
    int held[4][2];                                // per slot: the barrier, its phase
    for (int seg = 0; seg < 40; ++seg) {
      rng = rng * 1664525u + 1013904223u;
      const int tiles = run == 0 ? 1 : 1 + (rng >> 16) % 4;
      for (int k = 0; k < 2 + tiles; ++k, ++ri) {
        const int slot = ri % 4;
        if (ri >= 4 && q.held(slot)) {
          ++waits;
          const int bar = q.bar(slot);
          if (bar != held[slot][0] || q.parity(slot) != (uint32_t)(held[slot][1] & 1)) ++early;
          if (done[bar] < held[slot][1] + 1) ++early;
          if (done[bar] > held[slot][1] + 1) ++lapped;
        }
        if (k < 2) {
          q.put(slot, seg, k);
          const int bar = QuerySlots::bar_of(seg, k);
          held[slot][0] = bar;
          held[slot][1] = done[bar]++;
        } else {
          q.clear(slot);
        }
      }
    }
  }
  printf("%d %d %d", waits > 1000, lapped, early);
}
"""


def test_the_wait_for_a_query_is_never_lapped(tmp_path):
    """Also with a tile a segment, where a slot is taken again after the same half of
    the next segment's query was copied."""
    assert run(tmp_path, RING) == "1 0 0"


UNITS = """
int main() {
  const int sizes[][3] = {{1, 2, 1}, {7, 3, 2}, {100, 5, 9}, {33, 4, 33}, {33, 4, 500},      // n, m, share
                          {2048, 1024, 2048 * 1024}, {2050, 1024, 1 << 21}, {16384, 1024, 16384 * 1024 / 7},
                          {1 << 19, 1024, 1 << 21}, {1 << 19, 1024, 1 << 29}, {1 << 19, 1023, 6900000}};
  long long wrong = 0, seen = 0;
  for (auto& z : sizes) {
    const long long n = z[0], m = z[1], share = z[2], step = n * m > 4000 ? n * m / 4001 : 1;
    for (long long off = 0; off < n * m; off += step, ++seen) {
      const TreeUnit x = tree_unit((int)off, (int)n, (int)m, (int)share);
      const long long strip = off / (share * m), rem = off - strip * share * m;
      const long long tiles = share < n - strip * share ? share : n - strip * share;
      wrong += x.strip != strip || x.tiles != tiles || x.j != rem / tiles || x.k != rem % tiles || x.j >= m;
    }
  }
  printf("%d %lld", seen > 20000, wrong);
}
"""


def test_units_of_many_q_blocks(tmp_path):
    """Also where a share times the q-blocks passes 32 bits."""
    assert run(tmp_path, UNITS) == "1 0"


@pytest.mark.parametrize("path", [p for p in sorted(glob.glob(os.path.join(B.CSRC, "*.cu"))) if "cl::map(" in open(p).read()],
                         ids=os.path.basename)
def test_a_cluster_meets_before_its_shared_memory_is_written(path):
    """A CTA of the cluster may not have started when another has. Each kernel that uses an
    address in a peer's shared memory waits at a barrier of the cluster before that. (By
    the order in the source: a late CTA can not be made to happen.)"""
    for kernel in re.split(r"__global__", open(path).read())[1:]:
        use = kernel.find("cl::map(")
        if use >= 0:
            met = re.search(r"cl::sync\(\);|cl::wait_started\(\);  //|barrier\.cluster\.wait", kernel[:use])
            assert met, (os.path.basename(path), kernel[:120])
