// Work partition of the grouped-head (GQA) attention: blocks of query rows,
// their key tiles, and an equal share of all key tiles for every CTA.
//
// Sequence s brings nq new rows and holds L tokens with them; row i stands at
// position L - nq + i.  The G query heads of a kv head are packed into tile
// rows: row r of a 128-row tile is token r / G, head r % G, so `tpt` = 128 / G
// tokens share a tile and one K/V tile serves all heads of the group.  An item
// is (sequence, kv head, block of tpb tokens); it needs the key tiles of 128
// up to its last row's position.  Items are ordered by sequence, kv head and
// block; CTA c takes the tiles [T c / C, T (c + 1) / C) of the whole list of T,
// so every CTA has the same number of tiles whatever the lengths are, and an
// item that straddles a border leaves partial softmax states that a second
// kernel merges.  The lengths live in device memory (a captured call can be
// replayed with others), so the kernel computes the partition itself: a closed
// form counts the tiles of a sequence, and a block-wide sum finds the CTA's
// first item.
#pragma once

#include "common.cuh"

namespace csa {
namespace gqa {

constexpr int kTile = 128;  // keys per tile, and rows per tile

struct Geometry {
  const int32_t* cu_q;       // [n_seqs + 1]
  const int32_t* cache_len;  // [n_seqs]; null: L = nq (whole prompts)
  int n_seqs;
  int max_len;               // what a row of the block table can hold
  int64_t total_q;
  int Hkv, G;
  int tpt;                   // tokens per 128-row tile
  int tpb;                   // tokens per item (one or two tiles)
};

// sum_{t < n} floor((a t + b) / m) for n, a, b >= 0, m > 0, in O(log) steps:
// whole parts come out, and what is left is the same sum with the roles of
// the axes exchanged (lattice points under the line).
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t ans = 0;
  while (n > 0) {
    if (a >= m) {
      ans += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      ans += n * (b / m);
      b %= m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return ans;
}

// One sequence's rows and keys (offsets are clamped: bad ones cost wrong
// results, never an access out of range).
struct Seq {
  int row0;  // first packed row
  int nq, L, nblk;

  __device__ __forceinline__ void load(const Geometry& g, int s) {
    int64_t a = __ldg(g.cu_q + s), b = __ldg(g.cu_q + s + 1);
    a = a < 0 ? 0 : (a > g.total_q ? g.total_q : a);
    b = b < a ? a : (b > g.total_q ? g.total_q : b);
    row0 = static_cast<int>(a);
    nq = static_cast<int>(b - a);
    L = nq;
    if (g.cache_len != nullptr) {
      L = __ldg(g.cache_len + s);
      L = L < 0 ? 0 : (L > g.max_len ? g.max_len : L);
    }
    nblk = (nq + g.tpb - 1) / g.tpb;
  }
  // key tiles of block blk (at least one, so that rows without a key are written too)
  __device__ __forceinline__ int tiles(const Geometry& g, int blk) const {
    const int last = min((blk + 1) * g.tpb, nq);
    const int e = L - nq + last;  // keys its last row sees
    return e <= kTile ? 1 : (e + kTile - 1) / kTile;
  }
  // tiles of blocks 0 .. n-1
  __device__ __forceinline__ int64_t tiles_before(const Geometry& g, int n) const {
    int64_t sum = 0;
    if (n == nblk && n > 0) {
      sum = tiles(g, n - 1);
      --n;
    }
    if (n <= 0) return sum;
    const int off = L - nq;
    int z = off >= kTile ? 0 : (kTile - off) / g.tpb;  // blocks that need one tile
    z = z < n ? z : n;
    sum += z;
    // block z + t: floor((off + 127 + (z + 1) tpb + t tpb) / 128)
    if (n > z)
      sum += floor_sum(n - z, kTile, g.tpb, static_cast<int64_t>(off) + kTile - 1 + static_cast<int64_t>(z + 1) * g.tpb);
    return sum;
  }
};

// What one CTA does: tiles [start, start + left) of the list, beginning in
// sequence s at tile `within` of that sequence's Hkv * tiles_before(nblk).
struct Share {
  int64_t left, within;
  int s;
  int ctas;  // CTAs that have work
};

// All threads of the block call this (blockDim.x a multiple of 32, at most
// 1024); `scratch` holds 40 int64 words.
__device__ __forceinline__ Share find_share(const Geometry& g, int cta, int n_ctas, int64_t* scratch) {
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nthr >> 5;
  const int chunk = (g.n_seqs + nthr - 1) / nthr;
  const int s0 = tid * chunk, s1 = min(s0 + chunk, g.n_seqs);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    Seq q;
    q.load(g, s);
    mine += q.tiles_before(g, q.nblk) * g.Hkv;
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  if (tid == 0) {
    scratch[32] = -1;
    scratch[33] = 0;
  }
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    const int64_t v = scratch[w];
    if (w < warp) before += v;
    total += v;
  }
  before += inc - mine;
  Share sh;
  sh.ctas = static_cast<int>(total < n_ctas ? total : n_ctas);
  sh.left = 0;
  sh.within = 0;
  sh.s = 0;
  if (cta >= sh.ctas) return sh;  // the same for every thread of the block
  const int64_t start = total * cta / sh.ctas, end = total * (cta + 1) / sh.ctas;
  sh.left = end - start;
  if (start >= before && start < before + mine) {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      Seq q;
      q.load(g, s);
      const int64_t n = q.tiles_before(g, q.nblk) * g.Hkv;
      if (start < at + n) {
        scratch[32] = s;
        scratch[33] = start - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  sh.s = static_cast<int>(scratch[32]);
  sh.within = scratch[33];
  return sh;
}

// Walks a share item by item.
struct Walk {
  Seq q;
  int s, h, blk;
  int t0, t1, n;  // this piece's key tiles [t0, t1) of the item's n
  int left;       // tiles of the share from this piece on
  bool one;       // the block's rows fit one 128-row tile

  __device__ __forceinline__ void set(const Geometry& g, int ta) {
    n = q.tiles(g, blk);
    t0 = ta;
    t1 = ta + min(n - ta, left);
    one = g.tpb <= g.tpt || q.nq - blk * g.tpb <= g.tpt;
  }
  __device__ __forceinline__ bool begin(const Geometry& g, const Share& sh) {
    left = static_cast<int>(sh.left);
    if (left <= 0) return false;
    s = sh.s;
    q.load(g, s);
    const int64_t per = q.tiles_before(g, q.nblk);
    h = static_cast<int>(sh.within / per);
    const int64_t r = sh.within - h * per;
    int lo = 0, hi = q.nblk - 1;  // the last block with tiles_before <= r
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (q.tiles_before(g, mid) <= r) lo = mid; else hi = mid - 1;
    }
    blk = lo;
    set(g, static_cast<int>(r - q.tiles_before(g, lo)));
    return true;
  }
  __device__ __forceinline__ bool next(const Geometry& g) {
    left -= t1 - t0;
    if (left <= 0) return false;
    if (++blk >= q.nblk) {
      blk = 0;
      if (++h >= g.Hkv) {
        h = 0;
        do {
          if (++s >= g.n_seqs) return false;
          q.load(g, s);
        } while (q.nblk == 0);
      }
    }
    set(g, 0);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n; }
};

}  // namespace gqa
}  // namespace csa
