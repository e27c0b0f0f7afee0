// The work list of pa_chunk_fp8, shared by the kernel and a host test.
//
// An item is bt = 256 / G whole tokens of one request and KV head; it costs a
// unit per 128-key tile and ITEM_COST units to begin (its query operand, the
// first tile's way through the pipeline, its result). The units in order:
// heads, then requests, then items, then the beginning and the key tiles. How
// many a request has is known in closed form, so nobody has to list them.
#pragma once
#ifndef __CUDACC__
#include <algorithm>
#define QPA_HD
namespace qpa { namespace chunk { using std::max; using std::min; } }
#else
#define QPA_HD __host__ __device__
#endif
#ifdef __CUDACC__
#define QPA_HD_CALL __host__ __device__ __noinline__   // cold code, once per kernel
#else
#define QPA_HD_CALL
#endif

namespace qpa {
namespace chunk {

constexpr int TILE = 128;            // keys per unit, rows per row tile
constexpr int ITEM_COST = 4;
constexpr int MIN_UNITS = 4;         // per CTA: fewer CTAs take part rather than smaller ranges

// sum_{i < n} floor((a i + b) / m) for a, b >= 0 (the lattice points under a
// line, by a Euclid-like reduction). T: 32 bits where a n + b and m fit (the
// divisions are most of the work), else 64.
template <typename T>
QPA_HD inline long long floor_sum_t(T n, T m, T a, T b) {
  long long s = 0;
  while (n > 0) {
    if (a >= m) {
      s += (long long)n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += (long long)n * (b / m);
      b %= m;
    }
    const T y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const T t = m;
    m = a;
    a = t;
  }
  return s;
}
QPA_HD_CALL inline long long floor_sum(long long n, long long m, long long a, long long b) {
  if (a * n + b <= 0x7fffffffLL) return floor_sum_t<unsigned>((unsigned)n, (unsigned)m, (unsigned)a, (unsigned)b);
  return floor_sum_t<long long>(n, m, a, b);
}

// sum_{i < n} floor((bt i + b) / TILE) for b >= 0. Group sizes are powers of two
// as a rule, so bt is one too and no division is left: with bt <= TILE, q = TILE
// / bt and c = floor(b / bt) the terms are floor((c + i) / q), a difference of
// F(x) = sum_{y < x} floor(y / q) = q k (k - 1) / 2 + k (x - q k), k = floor(x / q).
// (The general reduction took 1.7 us of a launch.)
QPA_HD inline long long tile_sum(int n, int bt, long long b) {
  if (n <= 0) return 0;
  if ((bt & (bt - 1)) != 0) return floor_sum(n, TILE, bt, b);
  if (bt > TILE) return (b / TILE) * n + (long long)(bt / TILE) * n * (n - 1) / 2;   // constants: shifts
  int lb = 0;
  while ((1 << lb) < bt) ++lb;
  const int lq = 7 - lb;
  static_assert(TILE == 128, "2^7");
  const long long c = b >> lb, x = c + n, kc = c >> lq, kx = x >> lq;
  return (((kx * (kx - 1)) << lq) >> 1) + kx * (x - (kx << lq)) - (((kc * (kc - 1)) << lq) >> 1) - kc * (c - (kc << lq));
}

// One request as the schedule sees it: first query row, rows, cached tokens
// (the rows' own included), items.
struct Req {
  int q0, ql, L, nt;
  // key tiles of item j: those its last row sees, at least one
  QPA_HD int tiles(int j, int bt) const {
    const int last = min((j + 1) * bt, ql) - 1;
    return max(L - ql + last, 0) / TILE + 1;
  }
  // units of items 0 .. j-1 (j < nt: all of them have bt tokens)
  QPA_HD_CALL long long before(int j, int bt) const {
    const int d = L - ql;
    // items whose last row sees nothing, d + (i + 1) bt - 1 < 0: one unit each
    const int i0 = d >= 1 - bt ? 0 : min(j, -d / bt);
    return (long long)j * (1 + ITEM_COST) + tile_sum(j - i0, bt, d + (long long)(i0 + 1) * bt - 1);
  }
  QPA_HD long long units(int bt) const { return nt ? before(nt - 1, bt) + tiles(nt - 1, bt) + ITEM_COST : 0; }
  // first key tile at offset o into an item's units
  QPA_HD static int tile_at(long long o) { return o > ITEM_COST ? (int)(o - ITEM_COST) : 0; }
  // One step of the search for the item that holds unit off, which lies in
  // [lo, hi): whether probe i of 32 splits it at or before off, and where that is
  QPA_HD static int split(int lo, int hi, int i) { return lo + (int)((long long)(hi - lo) * (i + 1) / 33); }
};

QPA_HD inline Req make_req(int start, int next, int len, int num_tokens, int max_len, int bt) {
  Req q;
  q.q0 = max(0, min(start, num_tokens));
  q.ql = max(0, max(0, min(next, num_tokens)) - q.q0);
  q.L = max(0, min(len, max_len));
  q.nt = q.ql / bt + (q.ql % bt != 0);
  return q;
}

// CTAs that take part in U units
QPA_HD inline int active_ctas(long long U, int grid) {
  const long long n = (U + MIN_UNITS - 1) / MIN_UNITS;
  return n < grid ? (int)n : grid;
}

}  // namespace chunk
}  // namespace qpa
