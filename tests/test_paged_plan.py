"""The paged cache's plan of a call, its host-callable functions compiled into
a program that runs on the CPU: how two lists of work share the CTAs, and which words about a
unit's parts are followed."""
import os
import subprocess

import pytest

from io_aware_exact_02_gb300 import build

MAIN = r"""
#include <cstdio>
#include "fa_paged.cuh"
using namespace fa;

static int bad(const char* what, long long a, long long b, int c, int g, int got) {
  printf("%s: wa %lld wb %lld ctas %d groups %d -> %d\n", what, a, b, c, g, got);
  return 1;
}

// Every pair of weights 1, 1.4, 2, ... 10^12 on every even number of CTAs.
static int split() {
  long long w[96];
  int n = 0;
  for (double x = 1; x < 1e12; x *= 1.4)
    if (n == 0 || (long long)x != w[n - 1]) w[n++] = (long long)x;
  for (int ctas = 4; ctas <= kPagedMaxCtas; ctas += 2)
    for (int groups = 1; groups <= ctas - 2; groups += groups < 12 ? 1 : 7) {
      if (paged_duo_split(0, 7, ctas, groups) != 0) return bad("no first", 0, 7, ctas, groups, 0);
      if (paged_duo_split(7, 0, ctas, groups) != ctas) return bad("no second", 7, 0, ctas, groups, 0);
      for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
          const int na = paged_duo_split(w[i], w[j], ctas, groups);
          if (na < 2 || na > ctas - 2 || na % 2 != 0) return bad("share", w[i], w[j], ctas, groups, na);
          if (na < groups) return bad("groups", w[i], w[j], ctas, groups, na);
          // A multiple of the groups, or one more CTA, which makes it even.
          if (na % groups > 1) return bad("multiple", w[i], w[j], ctas, groups, na);
          // In proportion, to half a group and the rounding to clusters.
          const double want = (double)w[i] / ((double)w[i] + (double)w[j]) * ctas;
          const double off = na > want ? na - want : want - na;
          if (off > groups + 2.0) return bad("proportion", w[i], w[j], ctas, groups, na);
        }
    }
  return 0;
}

// A word is taken for one exactly when it has slots and they lie in the
// workspace of the CTAs: all values of its 16-bit halves, as garbage may hold.
static int parts() {
  const int all[] = {0, 2, 76, 150, 152, kPagedMaxCtas};
  for (int ctas : all)
    for (int slot = 0; slot < 65536; slot += slot < 700 ? 1 : 97)
      for (int n = 0; n < 65536; n += n < 700 ? 1 : 97) {
        // Where the join reads: the first slot, then the next CTAs' slots 0.
        long long last = n > 1 ? (slot & ~1) + 2ll * (n - 1) : slot;
        if (last < slot) last = slot;
        const bool inside = n >= 1 && slot < 2 * ctas && last < 2 * ctas;
        if (paged_parts_ok(slot, n, 0, ctas, 8) != inside) return bad("parts", slot, n, ctas, 8, !inside);
      }
  const int rows[] = {-2147483647 - 1, -1, 0, 7, 8, 255, 256, 2147483647};
  for (int row : rows)
    for (int slot_rows : {8, 16, 256})
      if (paged_parts_ok(3, 2, row, 152, slot_rows) != (row >= 0 && row < slot_rows))
        return bad("row", 3, 2, row, slot_rows, 0);
  return 0;
}

int main(int argc, char** argv) { return argv[1][0] == 's' ? split() : parts(); }
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cu").write_text(MAIN)
    out = str(d / "plan")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O2", "-cudart", "static", "-I",
                    build.INCLUDE, "-I", build.CSRC, str(d / "plan.cu"), "-o", out], check=True)
    assert os.path.exists(out)
    return out


@pytest.mark.parametrize("what", ["split", "parts"])
def test_plan(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
