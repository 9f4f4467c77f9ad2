// qmv_attn_geom.h -- which keys a query, or a block of query rows, sees, and the tiles they
// make: integer arithmetic alone, so that a host compiler can build it for tests too.
//
// A sequence has n cached tokens, the last c of them new; its query i stands at position
// n - c + i, which is negative for the first ones when c > n. window is 0 (none) or any
// positive int.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define QMV_HD __host__ __device__ __forceinline__
#else
#define QMV_HD inline
#endif

namespace qmv {

// first key that the query at position pos sees. pos - window is formed only where it
// cannot leave 32 bits: window may be the largest int, and pos negative.
QMV_HD int window_first(int pos, int window) { return window == 0 || pos < window ? 0 : pos - window + 1; }

// tiles of TILE tokens from the one that holds token `first` to the one that holds token n - 1
// (n > 0, up to 2^31 - 16: n + TILE - 1 may leave 32 bits)
template <int TILE>
QMV_HD int tiles_of(int n, int first) {
  return (n - 1) / TILE + 1 - first / TILE;
}

// Rows qb QB .. (qb + 1) QB - 1 of a sequence (row = token * G + query head), as far as it has them
struct BlockRange {
  int first_pos, last_pos;   // positions of its first and last token
  int tile0, nt, last;       // first key tile of KT tokens, key tiles, last key that a row sees
};
template <int KT, int QB>
QMV_HD BlockRange block_range(int n, int c, int G, int qb, bool causal, int window) {
  const int R = c * G;
  const int r1 = (qb + 1) * QB < R ? (qb + 1) * QB : R;
  BlockRange b;
  b.first_pos = n - c + qb * QB / G;
  b.last_pos = n - c + (r1 - 1) / G;
  b.last = causal ? b.last_pos : n - 1;
  const int lo = window_first(b.first_pos, window);
  b.tile0 = lo / KT;
  b.nt = b.last < lo ? 0 : b.last / KT - lo / KT + 1;
  return b;
}


// What a block adds to the numbered tiles: its key tiles and `overhead`; 0 without a key tile
template <int KT, int QB>
QMV_HD int block_cost(int n, int c, int G, int qb, bool causal, int window, int overhead) {
  const int nt = block_range<KT, QB>(n, c, G, qb, causal, window).nt;
  return nt ? nt + overhead : 0;
}
// Blocks lane, lane + 32, ... of a sequence's nqb. A sequence's sum can pass 32 bits: 2^20
// queries of 16 heads over 2^20 keys are 2^17 blocks of 2^14 tiles.
template <int KT, int QB>
QMV_HD int64_t blocks_cost(int n, int c, int G, int nqb, int lane, bool causal, int window, int overhead) {
  int64_t sum = 0;
  for (int qb = lane; qb < nqb; qb += 32) sum += block_cost<KT, QB>(n, c, G, qb, causal, window, overhead);
  return sum;
}

}  // namespace qmv
