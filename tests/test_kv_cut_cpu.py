"""How the split attention kernel cuts its line of tiles among the CTAs: the
header's arithmetic, compiled for the host.  Every tile's owner has to be the
CTA whose piece holds it, for lines of a few tiles and of more than 2^32."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "gdn_kv_cut.h"

struct Even { static constexpr int kCtas = 3; static constexpr int kShare(int) { return 1; } };
struct Skewed { static constexpr int kCtas = 3; static constexpr int kShare(int o) { return 13 - o; } };

template <typename Cfg>
int check(int64_t total, int ctas, int segments) {
  const gdn::Cut<Cfg> cut{total, ctas / segments, segments};
  if (cut.begin(0) != 0 || cut.begin(ctas) != total) return printf("ends %lld\n", (long long)total);
  for (int i = 0; i < ctas; ++i) {
    const int64_t a = cut.begin(i), b = cut.begin(i + 1);
    if (b < a) return printf("pieces %lld %d\n", (long long)total, i);
    if (b == a) continue;
    const int64_t places[] = {a, a + (b - a) / 3, a + (b - a) / 2, b - 1};
    for (int64_t x : places)
      if (cut.owner(x) != i)
        return printf("total %lld ctas %d segments %d: tile %lld is CTA %d's, not %d's\n",
                      (long long)total, ctas, segments, (long long)x, i, cut.owner(x));
  }
  return 0;
}

int main() {
  std::vector<int64_t> totals = {1824, 2000, 4567, 179900, 1000003};
  const int64_t one = 1;
  for (int64_t t : {one << 31, one << 32, 3 * (one << 32), one << 35, one << 40})
    for (int64_t d : {-1000, -1, 0, 1, 12345}) totals.push_back(t + d);
  int bad = 0;
  for (int64_t t : totals)
    for (int ctas : {456, 608, 760, 3 * 148}) {
      if (ctas > t) continue;
      bad |= check<Even>(t, ctas, 1);
      if (ctas % 3 == 0) bad |= check<Skewed>(t, ctas, 3);
    }
  for (int64_t t : {1, 2, 7, 100}) bad |= check<Even>(t, (int)t, 1);
  return bad != 0;
}
"""


def test_owners_of_tiles(tmp_path):
    src = tmp_path / "cut.cc"
    src.write_text(SOURCE)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    # (a division by zero ends the program)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", os.path.join(ROOT, "gated_deltanet_recurrent_gb300", "csrc"),
                    "-I", os.path.join(cuda, "include"), str(src), "-o", str(tmp_path / "cut")],
                   check=True)
    r = subprocess.run([str(tmp_path / "cut")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
