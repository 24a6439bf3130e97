// The absorbed latent attention's division of work, as integer arithmetic that
// the kernels and the host share (no CUDA header needed): how query rows and
// tokens are cut, where a cut sequence's partial results lie, and how much room
// they take.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HD __host__ __device__
#else
#define MOE_HD
#endif

namespace moe {

constexpr int kTok = 64;                 // tokens of a tile
constexpr int kRows = 64;                // query rows of a tile at most
constexpr int kHead = 2;                 // tiles' worth of time that a piece costs beside its tiles

MOE_HD inline int up16(int v) { return (v + 15) & ~15; }
MOE_HD inline int per_cta(unsigned tiles, unsigned parts) { return (int)((tiles + parts - 1) / parts); }

struct RowTiles {
  int n, rows;   // row tiles and their rows
};
// rows split into tiles of at most 64, evenly, in multiples of 16
MOE_HD inline RowTiles row_tiles(long long rows) {
  RowTiles t;
  t.n = (int)((rows + kRows - 1) / kRows);
  t.rows = up16((int)((rows + t.n - 1) / t.n));
  t.n = (int)((rows + t.rows - 1) / t.rows);
  return t;
}

// One launch's sequences, query rows and CTAs.
struct LineShape {
  int B, Q, heads, shared;
  int G, NR, teams;          // row tiles of a sequence, their rows, and CTA teams
  int Gp, NRp, np, ctas;     // row tiles of the prefix, their rows, prefix tiles; CTAs of the grid
  int per_p;                 // tiles of the prefix line that a CTA takes
};

MOE_HD inline void set_line(LineShape& p, int B, int Q, int heads, int shared, int ctas) {
  p.B = B;
  p.Q = Q;
  p.heads = heads;
  p.shared = shared;
  p.ctas = ctas;
  const RowTiles s = row_tiles((long long)Q * heads), f = row_tiles((long long)B * Q * heads);
  p.G = s.n;
  p.NR = s.rows;
  p.teams = p.ctas / s.n;
  p.np = shared / kTok + (shared % kTok != 0);    // no sum that could pass an int
  p.Gp = p.np ? f.n : 0;
  p.NRp = f.rows;
  p.per_p = (int)(((long long)p.Gp * p.np + p.ctas - 1) / p.ctas);
}

// Room for partial results, in query rows: at least what a launch uses, and never less for more sequences, queries or
// heads (an even split's tiles can be smaller for more rows), so that a workspace serves every smaller call.
MOE_HD inline size_t tiles_at_most(long long rows) { return (size_t)((rows + kRows - 1) / kRows); }
MOE_HD inline size_t tile_rows_at_most(long long rows) { return rows < kRows ? (size_t)up16((int)rows) : (size_t)kRows; }
// The sequences' line: two pieces a CTA, and with a prefix the whole sequences too.
MOE_HD inline size_t suffix_rows(const LineShape& p) {
  const long long rows = (long long)p.Q * p.heads;
  return ((size_t)2 * p.ctas + (p.np ? p.B * tiles_at_most(rows) : 0)) * tile_rows_at_most(rows);
}
// The prefix line: two pieces a CTA, and the whole row tiles.
MOE_HD inline size_t prefix_rows(const LineShape& p) {
  const long long rows = (long long)p.B * p.Q * p.heads;
  return p.np ? ((size_t)2 * p.ctas + tiles_at_most(rows)) * tile_rows_at_most(rows) : 0;
}

// The barrier that says tile t's probabilities are written, and the phase of it.  The softmax warps wait for the value
// product of two tiles ago only, so they may have arrived for two tiles that the product's warp has not looked at yet:
// on one barrier the second arrival would hide the first.
constexpr int kPBars = 2;
MOE_HD inline int p_bar(int tile) { return tile % kPBars; }
MOE_HD inline uint32_t p_phase(int tile) { return (uint32_t)(tile / kPBars) & 1u; }

// The units of the sequences' line: all, and those before and through sequence b.
struct LineSums {
  int total, x0, x1;
};

// Where a query row's pieces lie: the prefix's first, then the sequence's.  A
// row of an empty sequence (or a bad id) has none.
class Pieces {
 public:
  int n_p, n;   // pieces of the prefix, and all

  MOE_HD Pieces(const LineShape& p_, int row_, const LineSums& line) : p(p_), row(row_) {
    const int per_seq = p.Q * p.heads;
    b = row / per_seq;
    in_seq = row - b * per_seq;
    g = in_seq / p.NR;
    const int total = line.total;
    x0 = line.x0;
    x1 = line.x1;
    per = per_cta(total, p.teams);
    t0 = x1 > x0 ? (x0 + kHead) / per : 0;                    // from its first tile on
    const int n_s = (x1 > x0 ? (x1 - 1) / per : -1) - t0 + 1;
    n_p = c0 = pr = 0;
    pa = 0;
    if (p.np) {
      pr = row / p.NRp;
      pa = (long long)pr * p.np;
      c0 = (int)(pa / p.per_p);
      n_p = (int)((pa + p.np - 1) / p.per_p) - c0 + 1;
    }
    n = n_p + n_s;
  }
  MOE_HD bool direct() const { return n_p == 0 && n == 1; }   // written by decode_kernel
  // Piece k's index among all rows of its line's pieces; false, and no index, where the row has no such piece.
  MOE_HD bool find(int k, size_t& at) const {
    if (k < 0 || k >= n) return false;
    if (k < n_p) {
      const long long from = (long long)(c0 + k) * p.per_p;
      const int slot = (pa >= from && pa + p.np <= from + p.per_p) ? 2 * p.ctas + pr : 2 * (c0 + k) + (pa > from ? 1 : 0);
      at = (size_t)slot * p.NRp + (row - pr * p.NRp);
      return true;
    }
    const int t = t0 + k - n_p;
    const long long from = (long long)t * per;
    const int slot = (x0 + kHead >= from && x1 <= from + per) ? 2 * p.teams * p.G + b * p.G + g
                                                              : 2 * (t * p.G + g) + (x0 > from ? 1 : 0);
    at = (size_t)slot * p.NR + (in_seq - g * p.NR);
    return true;
  }

 private:
  const LineShape& p;
  int row, b, in_seq, g, x0, x1, per, t0, c0, pr;
  long long pa;
};

}  // namespace moe
