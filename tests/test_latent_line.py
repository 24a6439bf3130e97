"""The absorbed attention's division of work, on the CPU: the arithmetic that
its kernels index partial results with, compiled as host code and asked about
random batches with empty sequences (an id out of range counts as one); and
the order of its probabilities' barriers, over every interleaving."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HARNESS = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "latent_line.h"
using namespace moe;
#define REQUIRE(x) do { if (!(x)) { std::printf("line %d: %s (B %d Q %d heads %d shared %d ctas %d row %d n %d k %d at %zu)\n", \
    __LINE__, #x, p.B, p.Q, p.heads, p.shared, p.ctas, row, q.n, k, at); std::exit(1); } } while (0)
int main(int argc, char** argv) {
  std::mt19937 g(std::atoi(argv[1]));
  auto pick = [&](int lo, int hi) { return lo + (int)(g() % (unsigned)(hi - lo + 1)); };
  long long empty = 0, cut = 0;
  for (int trial = 0; trial < 400; ++trial) {
    LineShape p;
    const int heads[] = {1, 5, 8, 16, 20, 37, 64, 96, 128};
    const int shared = pick(0, 2) ? 0 : 16 * pick(1, 300);
    set_line(p, pick(1, 90), pick(1, 4), heads[pick(0, 8)], shared, pick(0, 3) ? 152 : pick(16, 200));
    std::vector<int> at_b(1, 0);
    const int longest = pick(0, 1) ? 300 : 20000;
    for (int b = 0; b < p.B; ++b) {
      const int len = pick(0, 2) ? pick(0, longest) : 0;
      at_b.push_back(at_b.back() + (len > shared ? (len - shared + kTok - 1) / kTok + kHead : 0));
    }
    for (int row = 0; row < p.B * p.Q * p.heads; ++row) {
      const int b = row / (p.Q * p.heads);
      const Pieces q(p, row, LineSums{at_b[p.B], at_b[b], at_b[b + 1]});
      size_t at = 0, last = ~(size_t)0;
      int k = 0;
      REQUIRE(q.n >= 0 && q.n_p >= 0 && q.n >= q.n_p);
      REQUIRE((q.n_p > 0) == (shared > 0));
      REQUIRE((q.n > q.n_p) == (at_b[b + 1] > at_b[b]));
      empty += q.n == 0;
      cut += q.n > 1;
      // what a row that decode_kernel did not write itself may be asked for: places inside the regions, one a piece
      for (k = -2; !q.direct() && k < q.n + 40; ++k) {
        const bool there = q.find(k, at);
        REQUIRE(there == (k >= 0 && k < q.n));
        if (!there) continue;
        REQUIRE(at < (k < q.n_p ? prefix_rows(p) : suffix_rows(p)));
        REQUIRE(k == 0 || k == q.n_p || at != last);
        last = at;
      }
    }
  }
  std::printf("%lld %lld\n", empty, cut);
  return 0;
}
"""

# All states (tiles the softmax warps arrived for, tiles the product's warp saw, value products that ended) that can be
# reached: a wait on a phase's parity passes once that phase is over and until the next one is.
BARRIERS = r"""
#include <cstdio>
#include <set>
#include <tuple>
#include <vector>
#include "latent_line.h"
using namespace moe;
int main() {
  const int N = 9;
  typedef std::tuple<int, int, int> State;
  std::set<State> seen;
  std::vector<State> todo(1, State(0, 0, 0));
  while (!todo.empty()) {
    const State st = todo.back();
    todo.pop_back();
    if (!seen.insert(st).second) continue;
    const int soft = std::get<0>(st), product = std::get<1>(st), ended = std::get<2>(st);
    const size_t before = todo.size();
    if (soft < N && (soft < 2 || ended >= soft - 1)) todo.push_back(State(soft + 1, product, ended));
    if (product < N) {
      unsigned over = 0;                                     // phases of this tile's barrier that are over
      for (int t = 0; t < soft; ++t) over += p_bar(t) == p_bar(product);
      if ((over & 1u) != p_phase(product)) {
        if (soft <= product) return std::printf("tile %d's product starts before its probabilities\n", product), 1;
        todo.push_back(State(soft, product + 1, ended));
      }
    }
    if (ended < product) todo.push_back(State(soft, product, ended + 1));
    if (todo.size() == before && st != State(N, N, N)) return std::printf("stuck at %d %d %d\n", soft, product, ended), 1;
  }
  return seen.count(State(N, N, N)) ? 0 : 1;
}
"""


def compiled(d, source):
    (d / "h.cpp").write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "edge_moe_serving_gb300", "csrc"),
                    str(d / "h.cpp"), "-o", str(d / "h")], check=True)
    return str(d / "h")


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("line"), HARNESS)


@pytest.mark.parametrize("seed", range(4))
def test_pieces_lie_inside_the_workspace(harness, seed):
    r = subprocess.run([harness, str(seed)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    empty, cut = (int(x) for x in r.stdout.split())
    assert empty > 1000 and cut > 1000            # rows without pieces, and cut ones, were among them


def test_probability_barriers_never_stick(tmp_path):
    r = subprocess.run([compiled(tmp_path, BARRIERS)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
