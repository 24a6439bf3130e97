"""How moe_kv_append shares its rows out, on the CPU: the kernel's own
arithmetic, up to the largest number of rows that a call takes."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include <climits>
#include <cstdio>
#include <initializer_list>
#include "kv_append_shape.h"
using namespace moe;
int main() {
  for (unsigned sms : {1u, 16u, 148u, 152u, 200u})
    for (int N : {1, 2, 31, 32, 1215, 1216, 9727, 9728, 9729, 20000, 311295, 311296, 311297, 1 << 20, 1 << 30,
                  INT_MAX - 320000, INT_MAX - 9728, INT_MAX - 9000, INT_MAX - 1, INT_MAX}) {
      const AppendShape a = append_shape(N, sms);
      const unsigned step = append_step(a);
      if (a.per < 1 || a.per > 32 || a.ctas < 1 || a.ctas > 8 * sms) return std::printf("%u %d: %u %u\n", sms, N, a.per, a.ctas), 1;
      unsigned long long rows = 0;
      for (unsigned c = 0; c < a.ctas; ++c)
        for (unsigned w = 0; w < kAppendWarps; ++w) {
          const unsigned first = append_first(a, c, w);
          if (first >= (unsigned)N) continue;
          const unsigned turns = ((unsigned)N - first + step - 1) / step, last = first + (turns - 1) * step;
          if (last >= (unsigned)N || last + step < (unsigned)N || last + step < last)
            return std::printf("%u %d: a warp's last turn at %u, step %u\n", sms, N, last, step), 1;
          rows += (unsigned long long)(turns - 1) * a.per + ((unsigned)N - last < a.per ? (unsigned)N - last : a.per);
        }
      if (rows != (unsigned long long)N) return std::printf("%u %d: %llu rows\n", sms, N, rows), 1;
    }
  return 0;
}
"""


def test_every_row_is_taken_once(tmp_path):
    (tmp_path / "h.cpp").write_text(HARNESS)
    exe = str(tmp_path / "h")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "edge_moe_serving_gb300", "csrc"),
                    str(tmp_path / "h.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
