/*
 * mk_attn_cut.h -- the arithmetic of mk_attn.cu's cut: items of work on a line, their costs,
 * and the workers that own its places.  Plain integer code, which also compiles for the host.
 */
#ifndef MK_ATTN_CUT_H
#define MK_ATTN_CUT_H

#include <cstdint>

#ifdef __CUDACC__
#define MK_HD __host__ __device__ __forceinline__
#else
#define MK_HD inline
#endif

namespace mk_cut {

constexpr int kTile = 128;         /* keys per tile; rows per row tile */
/* The line's unit is about 1100 cycles.  A tile takes 4000 of a CTA in a pair (its products
 * and softmaxes, partly hidden under one another) and 2300 in a single (64 KB at the SM's
 * share of HBM); an item's beginning and end take 12000 and 4000 on top. */
constexpr int kPairTile = 3, kSingleTile = 2, kPairItem = 11, kSingleItem = 4;
constexpr int kShare = 6; /* a CTA's share at least: each of its streams meets a tile of a long item */

MK_HD int lesser(int a, int b) { return a < b ? a : b; }
MK_HD int greater(int a, int b) { return a > b ? a : b; }

/* Query tokens come in blocks of two row tiles of TB tokens.  T tokens: this many blocks have
 * more than one row tile (pairs); a last one may have one (a single). */
MK_HD int pair_blocks(int T, int TB) {
  if (T <= TB) return 0;
  const int n = T / (2 * TB);
  return n + (T - n * 2 * TB > TB);
}
MK_HD bool has_single(int T, int TB, int pairs) {
  return T > pairs * 2 * TB; /* else the last pair holds the rest */
}
/* Keys that the last token of block j of a sequence sees. */
MK_HD int block_end(int len, int T, int TB, int j) {
  return lesser(len, len - T + lesser(T, (j + 1) * 2 * TB));
}
MK_HD int key_tiles(int begin, int end) {
  return end > begin ? (end - begin + kTile - 1) / kTile : 0;
}
/* An item begins with its fixed cost; tile t then begins t tile costs further on, and
 * belongs to the worker that owns its first place. */
MK_HD int fixed_cost(int line) { return line ? kSingleItem : kPairItem; }
MK_HD int tile_cost(int line) { return line ? kSingleTile : kPairTile; }
MK_HD int item_cost(int line, int tiles) {
  return tiles ? tiles * tile_cost(line) + fixed_cost(line) : 0;
}

/* sum of floor((a k + b) / m) over k = 0 .. n - 1, by Euclid's algorithm on (m, a).
 * a n + b below 2^32; a, n >= 0, m >= 1. */
MK_HD uint64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  uint64_t sum = 0;
  while (n) {
    sum += (uint64_t)n * (n - 1) / 2 * (a / m) + (uint64_t)n * (b / m);
    a %= m;
    b %= m;
    const uint32_t y = a * n + b;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}
/* Cost of the pairs of a sequence's blocks 0 .. j - 1, j <= pair_blocks(T, TB), over the keys
 * from `start`: without a walk over the blocks, of which a call can have 2^18. */
MK_HD int pairs_before(int start, int len, int T, int TB, int j) {
  const int B = 2 * TB, full = lesser(j, T / B); /* blocks whose tokens all exist: B keys apart */
  const int e0 = len - T + B - start;            /* keys of block 0 */
  const int i0 = e0 > 0 ? 0 : -e0 / B + 1;       /* the first block with keys */
  int cost = 0;
  if (full > i0) {
    const int n = full - i0;
    cost = (int)floor_sum(n, kTile, B, e0 + i0 * B + kTile - 1) * kPairTile + n * kPairItem;
  }
  if (j > full) cost += item_cost(0, key_tiles(start, len)); /* the last block, partly filled */
  return cost;
}

/* CTAs that take part.  With kShare places each, every worker whose share lies between an
 * item's first tile and its last has a tile of it: a CTA's 6 places hold one of a pair's
 * tiles, a stream's 3 one of a single's.  (The CTA whose share holds the last pairs may have
 * fewer singles, but those begin with an item's fixed cost: with up to 4 of them no tile, with
 * up to 8 the first tile in stream 1, with 9 or more tiles in both.) */
MK_HD int active_ctas(int total, int n_cta) { return greater(1, lesser(n_cta, total / kShare)); }
/* Where CTA c's share of the line begins. */
MK_HD int share_begin(int c, int total, int n) {
  return (int)((unsigned long long)c * (unsigned)total / (unsigned)n);
}
/* Of CTA c's share: the pairs, for both streams, and the singles (behind all pairs), of which
 * each stream has its half. */
struct Share {
  int x, end, x1, end1;
};
MK_HD Share share_of(int c, int s, int total, int pairs, int n) {
  const int lo = share_begin(c, total, n), hi = share_begin(c + 1, total, n);
  const int s0 = greater(lo, pairs) - pairs, s1 = greater(hi, pairs) - pairs, mid = (s0 + s1 + 1) >> 1;
  return {lesser(lo, pairs), lesser(hi, pairs), s ? mid : s0, s ? s1 : mid};
}
/* The CTA that owns place x: the largest c with c total < (x + 1) n.  An estimate in
 * 32 bits is off by less than one. */
MK_HD int cta_of(int x, int total, int n) {
  const long long y = ((long long)x + 1) * n;
#ifdef __CUDA_ARCH__
  int c = (int)__fdividef((float)y, (float)total);
#else
  int c = (int)((float)y / (float)total);
#endif
  while ((long long)c * total >= y) --c;
  while (((long long)c + 1) * total < y) ++c;
  return c;
}
/* The worker that owns place x of the pairs (a CTA) or of the singles (two streams a CTA). */
MK_HD int worker_of(int line, int x, int total, int pairs, int n) {
  if (line == 0) return cta_of(x, total, n);
  const int c = cta_of(x + pairs, total, n);
  return 2 * c + (x >= share_of(c, 1, total, pairs, n).x1);
}
/* Of an item of nt tiles at `begin`, a share from place x (inside the item) to `end` has n
 * tiles from t0; `next` is the place behind them.  n is 0 where the share ends within the
 * item's fixed cost. */
struct Range {
  int t0, n, next;
};
MK_HD Range piece_range(int line, int begin, int nt, int x, int end) {
  const int at = begin + fixed_cost(line);
  const int a = greater(0, x - at), b = greater(0, end - at);
  const int t0 = line ? (a + kSingleTile - 1) / kSingleTile : (a + kPairTile - 1) / kPairTile;
  const int t1 = line ? (b + kSingleTile - 1) / kSingleTile : (b + kPairTile - 1) / kPairTile;
  return {t0, greater(0, lesser(nt, t1) - t0), lesser(end, at + nt * tile_cost(line))};
}

}  // namespace mk_cut

#endif /* MK_ATTN_CUT_H */
