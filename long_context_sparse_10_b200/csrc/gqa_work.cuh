// Work partition of the grouped-head (GQA) attention: blocks of query rows,
// their key tiles, and an equal share of all key tiles for every CTA.
//
// Sequence s brings nq new rows and holds L tokens with them; row i stands at
// position L - nq + i.  The G query heads of a kv head are packed into tile
// rows: row r of a 128-row tile is token r / G, head r % G, so `tpt` = 128 / G
// tokens share a tile and one K/V tile serves all heads of the group.  An item
// is (sequence, kv head, block of tpb tokens); it needs the key tiles of 128
// up to its last row's position.  Items are ordered by sequence, kv head and
// block, and each is worth its tiles plus kItemCost for its queries, its
// read-out and the pipeline's refill (measured at two tiles' time: without it
// the CTAs whose share was 29 short items of a prompt's first blocks ended 120
// of 670 us after the others).  CTA c takes the units [U c / C, U (c + 1) / C)
// of the whole list of U; an item that straddles a border leaves partial
// softmax states that a second kernel merges.  The lengths live in device
// memory (a captured call can be replayed with others), so the kernel computes
// the partition itself: a closed form counts the tiles of a sequence, a
// block-wide sum finds the sequence of the CTA's first unit, and a warp its
// block.
#pragma once

#include "common.cuh"

namespace csa {
namespace gqa {

// The partition's arithmetic runs on the host too, where a test walks it at sizes that no GPU run reaches.
#define CSA_HD __host__ __device__ __forceinline__

CSA_HD int32_t load_word(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}

constexpr int kTile = 128;  // keys per tile, and rows per tile
constexpr int kItemCost = 2;

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

// sum_{t < n} floor((a t + b) / m) for a n + b < 2^32, in O(log) steps: whole
// parts come out, and what is left is the same sum with the roles of the axes
// exchanged: lattice points under a line, counted by the steps of the Euclidean
// algorithm.
CSA_HD int64_t floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  int64_t ans = 0;
  while (n > 0) {
    if (a >= m) {
      const uint32_t q = a / m;
      ans += static_cast<int64_t>(n) * (n - 1) / 2 * q;
      a -= q * m;
    }
    if (b >= m) {
      const uint32_t q = b / m;
      ans += static_cast<int64_t>(n) * q;
      b -= q * m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
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

  CSA_HD void load(const Geometry& g, int s) {
    int64_t a = load_word(g.cu_q + s), b = load_word(g.cu_q + s + 1);
    a = a < 0 ? 0 : (a > g.total_q ? g.total_q : a);
    b = b < a ? a : (b > g.total_q ? g.total_q : b);
    row0 = static_cast<int>(a);
    nq = static_cast<int>(b - a);
    L = nq;
    if (g.cache_len != nullptr) {
      L = load_word(g.cache_len + s);
      L = L < 0 ? 0 : (L > g.max_len ? g.max_len : L);
    }
    nblk = (nq + g.tpb - 1) / g.tpb;
  }
  // key tiles of block blk (at least one, so that rows without a key are written too)
  CSA_HD int tiles(const Geometry& g, int blk) const {
    const int last = min((blk + 1) * g.tpb, nq);
    const int e = L - nq + last;  // keys its last row sees
    return e <= kTile ? 1 : (e + kTile - 1) / kTile;
  }
  // tiles of blocks 0 .. n-1
  CSA_HD int64_t tiles_before(const Geometry& g, int n) const {
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
      sum += floor_sum(static_cast<uint32_t>(n - z), kTile, static_cast<uint32_t>(g.tpb),
                       static_cast<uint32_t>(off + kTile - 1 + (z + 1) * g.tpb));
    return sum;
  }
};

// What one CTA does: `left` units of the list, beginning at unit `unit` of an
// item.
struct Share {
  int64_t left;  // 2^31 and more for a prompt of 150 million tokens
  int s, h, blk, unit;
};

// The attention's items of a sequence: its row blocks.
struct Blocks {
  static CSA_HD int count(const Seq& q) { return q.nblk; }
  static CSA_HD int64_t units_before(const Geometry& g, const Seq& q, int n) {
    return q.tiles_before(g, n) + static_cast<int64_t>(n) * kItemCost;
  }
};

// The accumulated weight's items: pairs of key tiles, each worth kItemCost and
// the row blocks (of tpb = tpt tokens) with a row that sees the pair's first key.
struct KeyPairs {
  static CSA_HD int count(const Seq& q) { return q.nq > 0 ? (q.L + 2 * kTile - 1) / (2 * kTile) : 0; }
  static CSA_HD int first_block(const Geometry& g, const Seq& q, int pair) {
    const int t = pair * 2 * kTile - (q.L - q.nq);  // the first row that sees the key
    return t <= 0 ? 0 : t / g.tpb;
  }
  static CSA_HD int64_t units_before(const Geometry& g, const Seq& q, int n) {
    const int off = q.L - q.nq;
    int z = off < 0 ? 0 : off / (2 * kTile) + 1;  // pairs that every block sees
    z = z < n ? z : n;
    int64_t units = static_cast<int64_t>(n) * (q.nblk + kItemCost);
    if (n > z)
      units -= floor_sum(static_cast<uint32_t>(n - z), static_cast<uint32_t>(g.tpb), 2 * kTile,
                         static_cast<uint32_t>(z * 2 * kTile - off));
    return units;
  }
};

// CTA cta's run of `total` units over ctas CTAs (the first ones take one more): its length, and where it begins.
CSA_HD int64_t share_range(int64_t total, int ctas, int cta, int64_t* left) {
  const int64_t per = total / ctas, more = total - per * ctas;
  *left = per + (cta < more ? 1 : 0);
  return per * cta + (cta < more ? cta : more);
}

// The kv head of unit `at` of a sequence whose heads have `seq` units each: in 32 bits where both fit (a 64-bit
// division is a subroutine); 1,500,000 tokens with 128 heads on one kv head are 2^32 units.
CSA_HD int head_of(int64_t at, int64_t seq) {
  return static_cast<int>(((at | seq) >> 32) ? at / seq : static_cast<uint32_t>(at) / static_cast<uint32_t>(seq));
}

// All threads of the block call this (blockDim.x a multiple of 32, at most
// 1024); `scratch` holds 40 int64 words.
template <typename Items>
__device__ __forceinline__ Share find_share(const Geometry& g, int cta, int n_ctas, int64_t* scratch) {
  const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nthr >> 5;
  const int chunk = (g.n_seqs + nthr - 1) / nthr;
  const int s0 = tid * chunk, s1 = min(s0 + chunk, g.n_seqs);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    Seq q;
    q.load(g, s);
    mine += Items::units_before(g, q, Items::count(q)) * g.Hkv;
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < nw; ++w) {
    const int64_t v = scratch[w];
    if (w < warp) before += v;
    total += v;
  }
  before += inc - mine;
  const int ctas = static_cast<int>(total < n_ctas ? total : n_ctas);
  Share sh = {0, 0, 0, 0, 0};
  if (cta >= ctas) return sh;  // the same for every thread of the block
  const int64_t start = share_range(total, ctas, cta, &sh.left);
  if (start >= before && start < before + mine) {
    int64_t at = start - before;
    int s = s0;
    Seq q;
    q.load(g, s);
    int64_t seq = Items::units_before(g, q, Items::count(q));
    while (at >= seq * g.Hkv) {
      at -= seq * g.Hkv;
      q.load(g, ++s);
      seq = Items::units_before(g, q, Items::count(q));
    }
    const int h = head_of(at, seq);
    at -= h * seq;
    scratch[34] = at;
    int32_t* out = reinterpret_cast<int32_t*>(scratch + 32);
    out[0] = s;
    out[1] = h;
  }
  __syncthreads();
  if (warp == 0) {  // the last item of the head with units_before <= at, 32 candidates at a time
    int32_t* out = reinterpret_cast<int32_t*>(scratch + 32);
    const int64_t at = scratch[34];
    Seq q;
    q.load(g, out[0]);
    int lo = 0, n = Items::count(q);  // it is in [lo, lo + n)
    while (n > 1) {
      const int gap = (n + 31) / 32;
      const bool here = lane * gap < n && Items::units_before(g, q, lo + lane * gap) <= at;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, here));
      n = min(gap, n - k * gap);
      lo += k * gap;
    }
    if (lane == 0) {
      out[2] = lo;
      out[3] = static_cast<int>(at - Items::units_before(g, q, lo));
    }
  }
  __syncthreads();
  const int32_t* out = reinterpret_cast<const int32_t*>(scratch + 32);
  sh.s = out[0];
  sh.h = out[1];
  sh.blk = out[2];
  sh.unit = out[3];
  if (!CSA_INBOUNDS(sh.s >= 0 && sh.s < g.n_seqs && sh.h >= 0 && sh.h < g.Hkv && sh.blk >= 0 && sh.unit >= 0)) sh.left = 0;
  return sh;
}

// Walks a share item by item, over the pieces that have a tile.
struct Walk {
  Seq q;
  int s, h, blk;
  int t0, t1, n;  // this piece's key tiles [t0, t1) of the item's n
  int64_t left;   // units of the share behind this piece
  bool one;       // the block's rows fit one 128-row tile

  // the piece from unit u of the current item; false where it has no tile
  CSA_HD bool set(const Geometry& g, int u) {
    n = q.tiles(g, blk);
    const int end = left < kItemCost + n - u ? u + static_cast<int>(left) : kItemCost + n;
    left -= end - u;
    t0 = max(u - kItemCost, 0);
    t1 = max(end - kItemCost, 0);
    one = g.tpb <= g.tpt || q.nq - blk * g.tpb <= g.tpt;
    return t1 > t0;
  }
  CSA_HD bool begin(const Geometry& g, const Share& sh) {
    left = sh.left;
    if (left <= 0) return false;
    s = sh.s;
    h = sh.h;
    blk = sh.blk;
    q.load(g, s);
    return set(g, sh.unit) || next(g);
  }
  CSA_HD bool next(const Geometry& g) {
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
    return set(g, 0);  // without a tile only where the share ends in the item's cost
  }
  CSA_HD bool whole() const { return t0 == 0 && t1 == n; }
};

// Walks a share of key pairs.
struct MassWalk {
  Seq q;
  int64_t left;
  int s, h, pair, count;

  CSA_HD int cost(const Geometry& g) const {
    return kItemCost + q.nblk - KeyPairs::first_block(g, q, pair);
  }
  // an item belongs to the CTA in whose share its first unit lies
  CSA_HD bool begin(const Geometry& g, const Share& sh) {
    left = sh.left;
    if (left <= 0) return false;
    s = sh.s;
    h = sh.h;
    pair = sh.blk;
    q.load(g, s);
    count = KeyPairs::count(q);
    if (sh.unit == 0) return true;
    left += sh.unit;
    return next(g);
  }
  CSA_HD bool next(const Geometry& g) {
    left -= cost(g);
    if (left <= 0) return false;
    if (++pair >= count) {
      pair = 0;
      if (++h >= g.Hkv) {
        h = 0;
        do {
          if (++s >= g.n_seqs) return false;
          q.load(g, s);
          count = KeyPairs::count(q);
        } while (count == 0);
      }
    }
    return true;
  }
  // whether block b has a row that sees key tile 2 * pair + t
  CSA_HD bool active(const Geometry& g, int t, int b) const {
    const int k0 = (2 * pair + t) * kTile, last = min((b + 1) * g.tpb, q.nq) - 1;
    return k0 < q.L && q.L - q.nq + last >= k0;
  }
};

}  // namespace gqa
}  // namespace csa
